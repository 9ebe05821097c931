"""Refusals of dsa_head_norm_rope, dsa_cache_append and dsa_prefix_attn_decode:
the C ABI before it launches, the binding before it reaches the C ABI."""
import ctypes

import pytest
import torch

from gpu_common import lib

dsa = lib()
BF = torch.bfloat16
FAKE = 0x100000                        # never dereferenced: every call below fails validation


def _lay(**kw):
    f = dict(block_size=64, num_blocks=16, max_blocks_per_seq=4, batch=2, max_seq_len=200,
             block_table=0x10000, seq_lens=0x20000)
    f.update(kw)
    return dsa.PagedLayoutC(**f)


def _part(**kw):
    f = dict(in_=FAKE, in_token_stride=512, in_head_stride=128, out=FAKE, out_token_stride=512,
             out_head_stride=128, out_dtype=0, heads=4, dim=128, norm=1, norm_dim=128, eps=1e-6,
             weight=FAKE, bias=None, rope_offset=0, rope_dim=64, interleaved=0, inv_freq=FAKE)
    f.update(kw)
    return dsa.HeadPartC(**f)


def _heads(part, n=1, pos=FAKE, N=3):
    arr = (dsa.HeadPartC * max(1, len(part) if isinstance(part, list) else 1))(
        *(part if isinstance(part, list) else [part]))
    return dsa.lib().dsa_head_norm_rope(arr, n, pos, N, None)


BAD_PARTS = [
    (dict(in_=None), -1), (dict(out=None), -1), (dict(dim=0), -2), (dict(dim=12), -2),
    (dict(dim=1032), -2), (dict(heads=0), -2), (dict(out_dtype=5), -2), (dict(norm=3), -2),
    (dict(in_=FAKE + 8), -1), (dict(out=FAKE + 8), -1), (dict(out=FAKE + 4, out_dtype=1), -1),
    (dict(in_token_stride=513), -1), (dict(in_head_stride=-128), -1),
    (dict(out_token_stride=1 << 40), -1),
    (dict(out_head_stride=120), -1),               # heads overlap
    (dict(out_token_stride=504), -1),              # tokens overlap
    (dict(norm_dim=0), -1), (dict(norm_dim=129), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(weight=FAKE + 4), -1),
    (dict(rope_dim=63), -1), (dict(rope_offset=1), -1), (dict(rope_offset=66), -1),
    (dict(rope_dim=-2), -1), (dict(inv_freq=None), -1), (dict(rope_dim=1 << 30), -1),
]


@pytest.mark.parametrize("bad,code", BAD_PARTS, ids=lambda v: str(v) if isinstance(v, dict) else "")
def test_a_bad_part_is_refused_by_both_calls(bad, code):
    n0 = dsa.launch_count()
    assert _heads(_part(**bad)) == code
    arr = (dsa.HeadPartC * 1)(_part(**bad))
    rc = dsa.lib().dsa_cache_append(ctypes.byref(_lay()), None, None, 2, arr, 1, None, 0, FAKE, 256, None)
    assert rc == code
    assert dsa.launch_count() == n0


def test_head_norm_rope_refuses_bad_calls():
    assert dsa.lib().dsa_head_norm_rope(None, 1, FAKE, 1, None) == -1
    assert _heads(_part(), n=0) == -1
    assert _heads([_part()] * 5, n=5) == -1
    assert _heads(_part(), N=-1) == -1
    assert _heads(_part(), pos=None) == -1                       # a rotated part needs positions
    assert _heads(_part(), N=1 << 30) == -2                      # 2^32 rows
    assert _heads(_part(), N=0) == 0                             # nothing to do


def test_cache_append_refuses_bad_calls():
    arr = (dsa.HeadPartC * 1)(_part())

    def call(lay=None, seq=None, pos=None, N=2, cache=arr, nc=1, heads=None, nh=0, ws=FAKE, wsb=256):
        return dsa.lib().dsa_cache_append(ctypes.byref(lay or _lay()), seq, pos, N, cache, nc, heads,
                                          nh, ws, wsb, None)
    assert call(cache=None) == -1 and call(nc=0) == -1 and call(nc=5) == -1
    assert call(nh=1) == -1                                      # heads missing
    assert call(seq=FAKE) == -1 and call(pos=FAKE) == -1
    assert call(N=3) == -1                                       # append form: N <= batch
    assert call(N=-1) == -1
    assert call(ws=None) == -3 and call(wsb=8) == -3 and call(ws=FAKE + 16) == -3
    assert call(lay=_lay(block_size=0)) == -1
    head_major = (dsa.HeadPartC * 1)(_part(out_head_stride=4096, out_token_stride=128))
    assert call(cache=head_major) == -1                          # a pool's rows are token-major


def test_prefix_attn_refuses_bad_calls():
    ok = dsa.prefix_attn_decode_workspace_size(2, 4, 64, 64, 100)
    assert ok >= 256

    def call(lay=None, q=FAKE, k=FAKE, ks=64, v=FAKE, vs=64, Hq=4, Dqk=64, Dv=64, prefix=100, sc=0.1,
             out=FAKE, lse=None, ws=FAKE, wsb=ok):
        return dsa.lib().dsa_prefix_attn_decode(ctypes.byref(lay or _lay()), q, k, ks, v, vs, Hq, Dqk,
                                                Dv, prefix, sc, out, lse, ws, wsb, None)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(prefix=-1),
                dict(prefix=201), dict(ks=56), dict(vs=56), dict(ks=68), dict(sc=0.0), dict(sc=-1.0),
                dict(sc=float("nan")), dict(sc=float("inf")), dict(sc=2e38), dict(q=FAKE + 8), dict(k=FAKE + 8),
                dict(out=FAKE + 8), dict(lay=_lay(max_seq_len=257)), dict(lay=_lay(batch=0))):
        assert call(**bad) == -1, bad
    for bad in (dict(Hq=0), dict(Hq=129), dict(Dqk=60), dict(Dqk=584, ks=584), dict(Dv=520, vs=520),
                dict(Dv=4), dict(lay=_lay(batch=70000)),
                dict(lay=_lay(num_blocks=1 << 25, block_size=64))):
        assert call(**bad) == -2, bad
    assert call(ws=None) == -3 and call(wsb=128) == -3


def test_the_binding_checks_parts_before_the_c_abi():
    x = torch.zeros((3, 4, 64), dtype=BF)
    f = torch.zeros(32)
    with pytest.raises(TypeError, match="x"):
        dsa.HeadPart(x.float(), x)
    with pytest.raises(ValueError, match="x"):
        dsa.HeadPart(x[0], x)
    with pytest.raises(ValueError, match="x"):
        dsa.HeadPart(x.transpose(1, 2), x)
    with pytest.raises(TypeError, match="out"):
        dsa.HeadPart(x, x.half())
    with pytest.raises(TypeError, match="out"):
        dsa.HeadPart(x, x.to(torch.float8_e5m2))
    with pytest.raises(ValueError, match="norm"):
        dsa.HeadPart(x, x, norm="batch")
    with pytest.raises(TypeError, match="weight"):
        dsa.HeadPart(x, x, norm="rms", weight=torch.zeros(64, dtype=BF))
    with pytest.raises(ValueError, match="weight"):
        dsa.HeadPart(x, x, norm="rms", weight=torch.zeros(63))
    with pytest.raises(ValueError, match="inv_freq"):
        dsa.HeadPart(x, x, rope_dim=64)
    with pytest.raises(ValueError, match="inv_freq"):
        dsa.HeadPart(x, x, rope_dim=66, inv_freq=f)
    with pytest.raises(ValueError, match="parts"):
        dsa.HeadParts([])
    with pytest.raises(ValueError, match="parts"):
        dsa.HeadParts([dsa.HeadPart(x, x)] * 5)
    with pytest.raises(ValueError, match="tokens"):
        dsa.HeadParts([dsa.HeadPart(x, x), dsa.HeadPart(x[:2], x[:2])])
    part = dsa.HeadPart(x, x, rope_dim=64, inv_freq=f)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="pos"):
        dsa.head_norm_rope([part])
    with pytest.raises(ValueError, match="out"):
        dsa.head_norm_rope([dsa.HeadPart(x, x[:, :3])], pos)
    with pytest.raises(ValueError, match="pos"):
        dsa.head_norm_rope([part], pos[:2])
    with pytest.raises(TypeError, match="pos"):
        dsa.head_norm_rope([part], pos.long())
    with pytest.raises(ValueError, match="CUDA"):
        dsa.head_norm_rope([part], pos)


def test_the_binding_checks_pools_and_attention_operands():
    bt = torch.arange(4, dtype=torch.int32).reshape(2, 2)
    lay = dsa.PagedLayout(bt, torch.full((2,), 100, dtype=torch.int32), 64, 4, 128)
    x = torch.zeros((2, 1, 64), dtype=BF)
    ws = torch.zeros(4096, dtype=torch.uint8)
    pool = torch.zeros((4, 64, 64), dtype=BF)
    with pytest.raises(ValueError, match="pool"):
        dsa.cache_append(lay, None, None, [dsa.HeadPart(x, pool[:3])], ws)
    with pytest.raises(ValueError, match="out"):
        dsa.cache_append(lay, None, None, [dsa.HeadPart(x, pool[:, :, :56])], ws)
    with pytest.raises(ValueError, match="rows"):
        dsa.cache_append(lay, None, None,
                         [dsa.HeadPart(x, torch.zeros((4, 64, 56), dtype=BF))], ws)
    with pytest.raises(ValueError, match="heads"):
        dsa.cache_append(lay, None, None, [dsa.HeadPart(x, pool)], ws,
                         heads=[dsa.HeadPart(x[:1], x[:1])])
    with pytest.raises(ValueError, match="CUDA"):
        dsa.cache_append(lay, None, None, [dsa.HeadPart(x, pool)], ws)
    q = torch.zeros((2, 4, 64), dtype=BF)
    out = torch.zeros((2, 4, 64), dtype=BF)
    lse = torch.zeros((2, 4))
    with pytest.raises(ValueError, match="sequences"):
        dsa.prefix_attn_decode(lay, q[:1], pool, pool, 0, 0.1, out, lse, ws)
    with pytest.raises(TypeError, match="q"):
        dsa.prefix_attn_decode(lay, q.float(), pool, pool, 0, 0.1, out, lse, ws)
    with pytest.raises(ValueError, match="k_pool"):
        dsa.prefix_attn_decode(lay, q, pool[:3], pool, 0, 0.1, out, lse, ws)
    with pytest.raises(ValueError, match="out"):
        dsa.prefix_attn_decode(lay, q, pool, pool, 0, 0.1, out[:1], lse, ws)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.prefix_attn_decode(lay, q, pool, pool, 0, 0.1, out, lse, ws)
