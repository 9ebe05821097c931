"""Refusals of dsa_prompt_attn and the 4-bit cache's calls: the C ABI before it launches, the
binding before it reaches the C ABI."""
import ctypes

import pytest
import torch

from gpu_common import lib
from prompt_reference import LEVELS, MIDS, quantise64, values64, pack_rows

dsa = lib()
BF = torch.bfloat16
FAKE = 0x100000                        # never dereferenced: every call below fails validation


def _lay(**kw):
    f = dict(block_size=64, num_blocks=16, max_blocks_per_seq=4, batch=2, max_seq_len=200,
             block_table=0x10000, seq_lens=0x20000)
    f.update(kw)
    return dsa.PagedLayoutC(**f)


def test_prompt_attn_refuses_bad_calls():
    n0 = dsa.launch_count()
    need = dsa.prompt_attn_workspace_size(2, 100, 8, 2, 64, 64)
    assert need >= 256

    def call(q=FAKE, qt=512, qh=64, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, cq=FAKE, ck=FAKE, B=2, Nq=100,
             Nk=100, Hq=8, Hk=2, Dk=64, Dv=64, sc=0.1, out=FAKE, ot=512, oh=64, lse=None, ws=FAKE, wsb=need):
        return dsa.lib().dsa_prompt_attn(q, qt, qh, k, kt, kh, v, vt, vh, cq, ck, B, Nq, Nk, Hq, Hk, Dk, Dv, sc,
                                         out, ot, oh, lse, ws, wsb, None)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=FAKE + 8), dict(k=FAKE + 2),
                dict(v=FAKE + 8), dict(out=FAKE + 4), dict(B=0), dict(Nq=-1), dict(Nk=-1), dict(cq=None),
                dict(ck=None), dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")), dict(sc=2e38), dict(qt=513),
                dict(qt=0), dict(qh=0), dict(qh=56), dict(kt=-128), dict(kh=60), dict(vt=1 << 40), dict(oh=8),
                dict(ot=56)):
        assert call(**bad) == -1, bad
    for bad in (dict(Hq=0), dict(Hk=0), dict(Hq=7), dict(Dk=60), dict(Dk=264), dict(Dk=0), dict(Dv=4),
                dict(Dv=264),
                # 2^22 pairs of tiles of 1024 heads
                dict(Nq=1 << 30, Hq=1024, Hk=1024, B=1, qt=64 * 1024, ot=64 * 1024, kt=64 * 1024, vt=64 * 1024)):
        assert call(**bad) == -2, bad
    assert call(ws=None) == -3 and call(wsb=128) == -3 and call(ws=FAKE + 16) == -3
    # strides of a single token or head are not looked at
    assert call(B=1, Nq=1, qt=3, ot=5, ws=None) == -3
    assert call(Nq=0, q=None, out=None) == 0                       # nothing to do
    assert dsa.launch_count() == n0


def test_cache4_calls_refuse_bad_calls():
    n0 = dsa.launch_count()
    L = dsa.lib()
    assert dsa.cache4_row_bytes(128, 128) == 144 and dsa.cache4_row_bytes(80, 80) == 96
    assert [L.dsa_cache4_row_bytes(a, b) for a, b in ((0, 16), (8, 16), (24, 16), (272, 16), (16, 264), (-16, 16))] == [0] * 6

    def write(lay=None, seq=FAKE, pos=FAKE, N=2, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, Hk=2, Dk=64, Dv=64,
              pool=FAKE, ko=None, vo=None, ws=FAKE, wsb=256):
        return L.dsa_cache4_write(ctypes.byref(lay or _lay()), seq, pos, N, k, kt, kh, v, vt, vh, Hk, Dk, Dv, None,
                                  None, pool, ko, vo, ws, wsb, None)

    def read(lay=None, seq=FAKE, pos=FAKE, N=2, Hk=2, Dk=64, Dv=64, pool=FAKE, ko=FAKE, vo=FAKE, ws=FAKE, wsb=256):
        return L.dsa_cache4_read(ctypes.byref(lay or _lay()), seq, pos, N, Hk, Dk, Dv, None, None, pool, ko, vo, ws,
                                 wsb, None)
    for bad in (dict(k=None), dict(v=None), dict(pool=None), dict(seq=None), dict(pos=None), dict(N=-1),
                dict(seq=None, pos=None, N=3), dict(ko=FAKE), dict(vo=FAKE), dict(k=FAKE + 8), dict(v=FAKE + 2),
                dict(pool=FAKE + 8), dict(ko=FAKE + 8, vo=FAKE), dict(kt=12), dict(kh=-8), dict(vt=1 << 60),
                dict(vh=3), dict(lay=_lay(block_size=0)), dict(lay=_lay(max_seq_len=257))):
        assert write(**bad) == -1, bad
    for bad in (dict(seq=None), dict(pos=None), dict(ko=None), dict(vo=None), dict(pool=None), dict(N=-1),
                dict(ko=FAKE + 8), dict(lay=_lay(batch=0))):
        assert read(**bad) == -1, bad
    for call in (write, read):
        for bad in (dict(Hk=0), dict(Dk=0), dict(Dk=72), dict(Dk=272), dict(Dv=8), dict(N=1 << 30)):
            assert call(**bad) == -2, bad
        assert call(ws=None) == -3 and call(wsb=8) == -3 and call(ws=FAKE + 16) == -3
        assert call(N=0) == 0
    need = dsa.cache4_attn_decode_workspace_size(2, 8, 2, 64, 64)

    def attn(lay=None, q=FAKE, pool=FAKE, Hq=8, Hk=2, Dk=64, Dv=64, sc=0.1, out=FAKE, ws=FAKE, wsb=need):
        return L.dsa_cache4_attn_decode(ctypes.byref(lay or _lay()), q, pool, Hq, Hk, Dk, Dv, None, None, sc, out, None,
                                        ws, wsb, None)
    for bad in (dict(q=None), dict(pool=None), dict(out=None), dict(q=FAKE + 8), dict(pool=FAKE + 4), dict(out=FAKE + 8),
                dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")), dict(sc=2e38), dict(lay=_lay(num_blocks=0)),
                dict(lay=_lay(max_seq_len=-1))):
        assert attn(**bad) == -1, bad
    for bad in (dict(Hq=0), dict(Hk=0), dict(Hq=7), dict(Dk=24), dict(Dk=288), dict(Dv=0), dict(Dv=300)):
        assert attn(**bad) == -2, bad
    assert attn(ws=None) == -3 and attn(wsb=255) == -3
    assert dsa.launch_count() == n0


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_the_binding_checks_the_prompt_s_operands():
    q, k, v, out, lse, ws = _z(10, 8, 64), _z(12, 2, 64), _z(12, 2, 32), _z(10, 8, 32), _z(10, 8, dtype=torch.float32), \
        _z(4096, dtype=torch.uint8)
    cq, ck = torch.tensor([0, 4, 10], dtype=torch.int32), torch.tensor([0, 6, 12], dtype=torch.int32)

    def call(q=q, k=k, v=v, out=out, lse=lse, ws=ws, cu_q=cq, cu_k=ck):
        dsa.prompt_attn(q, k, v, 0.1, out, lse, ws, cu_q=cu_q, cu_k=cu_k)
    for kind, name, bad in ((TypeError, "q", dict(q=q.float())), (ValueError, "q", dict(q=q[0])),
                            (TypeError, "k", dict(k=k.half())), (ValueError, "k", dict(k=_z(12, 2, 32))),
                            (ValueError, "k", dict(k=_z(12, 64, 2).transpose(1, 2))),
                            (ValueError, "v", dict(v=v[:11])), (ValueError, "v", dict(v=v[:, :1])),
                            (ValueError, "out", dict(out=out[:9])), (ValueError, "out", dict(out=_z(10, 8, 64))),
                            (TypeError, "lse", dict(lse=_z(10, 8))), (ValueError, "lse", dict(lse=lse[:9])),
                            (TypeError, "ws", dict(ws=_z(64))), (TypeError, "cu_q", dict(cu_q=cq.long())),
                            (ValueError, "cu_q", dict(cu_q=cq[:1])), (ValueError, "cu_q", dict(cu_q=None)),
                            (ValueError, "cu_k", dict(cu_k=ck[:2])), (ValueError, "cu_k", dict(cu_k=None)),
                            (ValueError, "CUDA", dict())):
        with pytest.raises(kind, match=name):
            call(**bad)


def test_the_binding_checks_the_4_bit_cache_s_operands():
    bt = torch.arange(4, dtype=torch.int32).reshape(2, 2)
    lay = dsa.PagedLayout(bt, torch.full((2,), 100, dtype=torch.int32), 64, 4, 128)
    pool = torch.zeros((4, 2, 64, dsa.cache4_row_bytes(64, 32)), dtype=torch.uint8)
    k, v, ws = _z(3, 2, 64), _z(3, 2, 32), _z(256, dtype=torch.uint8)
    seq = pos = torch.zeros(3, dtype=torch.int32)
    hs = torch.ones(2)
    with pytest.raises(ValueError, match="multiples"):
        dsa.cache4_row_bytes(64, 40)

    def write(lay=lay, seq=seq, pos=pos, k=k, v=v, pool=pool, ws=ws, **kw):
        dsa.cache4_write(lay, seq, pos, k, v, pool, ws, **kw)

    def read(ko=k, vo=v, pool=pool, seq=seq, pos=pos, **kw):
        dsa.cache4_read(lay, seq, pos, pool, ko, vo, ws, **kw)
    bad_pools = (pool[:3], pool[:, :1], pool[:, :, :63], pool[..., :-1], pool[0])
    for p in bad_pools:
        with pytest.raises(ValueError, match="pool|contiguous"):
            write(pool=p)
        with pytest.raises(ValueError, match="pool|contiguous"):
            read(pool=p)
    for kind, name, bad in ((TypeError, "k", dict(k=k.float())), (ValueError, "v", dict(v=v[:2])),
                            (TypeError, "pool", dict(pool=pool.char())), (TypeError, "seq", dict(seq=seq.long())),
                            (ValueError, "pos", dict(pos=pos[:2])), (TypeError, "k_scale", dict(k_scale=hs.double())),
                            (ValueError, "v_scale", dict(v_scale=hs[:1])), (ValueError, "k_out", dict(k_out=k[:2], v_out=v)),
                            (ValueError, "CUDA", dict())):
        with pytest.raises(kind, match=name):
            write(**bad)
    for kind, name, bad in ((TypeError, "k_out", dict(ko=k.float())), (ValueError, "out", dict(vo=v[:2])),
                            (ValueError, "seq", dict(seq=seq[:2])), (ValueError, "CUDA", dict())):
        with pytest.raises(kind, match=name):
            read(**bad)
    q, out, lse = _z(2, 8, 64), _z(2, 8, 32), torch.zeros((2, 8))

    def attn(q=q, pool=pool, out=out, lse=lse, ws=ws, **kw):
        dsa.cache4_attn_decode(lay, q, pool, 0.1, out, lse, ws, **kw)
    for kind, name, bad in ((ValueError, "q", dict(q=q[:1], out=out[:1])), (TypeError, "q", dict(q=q.float())),
                            (ValueError, "out", dict(out=out[:, :4])), (ValueError, "pool", dict(pool=pool[:3])),
                            (ValueError, "pool", dict(pool=pool[..., :-16])), (ValueError, "lse", dict(lse=lse[:1])),
                            (ValueError, "k_scale", dict(k_scale=hs[:1])), (ValueError, "contiguous", dict(q=_z(2, 8, 128)[..., :64])),
                            (ValueError, "CUDA", dict())):
        with pytest.raises(kind, match=name):
            attn(**bad)


def test_the_reference_quantiser_takes_the_nearest_value():
    """quantise64 by brute force on one group per amplitude, ties to the even code."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((500, 1, 32), generator=g).to(BF)
    x[0, 0, :7] = torch.tensor(MIDS)
    x[0, 0, 7] = 6.0
    c, s = quantise64(x)
    t = s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    val = torch.tensor(LEVELS, dtype=torch.float64)[(c & 7).long()] * t
    far = (x.double().abs()[..., None] - torch.tensor(LEVELS, dtype=torch.float64) * t[..., None]).abs()
    assert torch.equal((x.double().abs() - val).abs(), far.amin(-1))
    assert (c[0, 0, :8] & 7).tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    rows = pack_rows((c, s), (c, s), 64)
    k, v = values64(rows, 32, 32)
    sign = 1 - 2 * torch.signbit(x).double()
    assert torch.equal(k, val * sign) and torch.equal(v, k)
