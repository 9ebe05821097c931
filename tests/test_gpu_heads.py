"""GPU tests of dsa_head_norm_rope and dsa_cache_append against plain 64-bit
forms.  Tolerances: one rounding to the stored type plus the fp32 bound that
heads_reference derives; rows no token names keep every byte."""
import numpy as np
import pytest
import torch

from gpu_common import lib, need_gpu
from heads_reference import assert_heads_close, transform64

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def _randn(g, *shape):
    return torch.randn(shape, generator=g).to(BF).cuda()


def _freq(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()


def _spec(g, dim, norm="rms", norm_dim=None, roff=0, rdim=0, inter=False, weight=True, bias=False):
    nd = dim if norm_dim is None else norm_dim
    s = dict(norm=norm, norm_dim=nd if norm != "none" else None, eps=1e-6, rope_offset=roff,
             rope_dim=rdim, interleaved=inter, inv_freq=_freq(rdim) if rdim else None)
    if norm != "none" and weight:
        s["weight"] = (1 + 0.2 * torch.randn(nd, generator=g)).cuda()
    if norm != "none" and bias:
        s["bias"] = (0.3 * torch.randn(nd, generator=g)).cuda()
    return s


# dim, norm, norm_dim, rope offset, rope dim, interleaved, bias, out type
SHAPES = [
    (128, "rms", None, 0, 128, False, False, BF), (128, "layer", None, 0, 64, False, True, F8),
    (64, "none", None, 0, 64, True, False, BF), (64, "rms", None, 0, 64, False, False, F8),
    (576, "rms", 512, 512, 64, True, False, BF), (576, "rms", 512, 512, 64, False, False, F8),
    (8, "rms", None, 0, 8, False, False, BF), (8, "layer", 3, 6, 2, True, True, BF),
    (16, "none", None, 0, 0, False, False, F8), (24, "rms", 17, 2, 22, False, True, BF),
    (72, "layer", 70, 10, 34, False, False, BF), (80, "rms", None, 0, 48, True, False, BF),
    (120, "rms", None, 0, 84, False, False, BF), (136, "rms", 130, 6, 102, False, True, F8),
    (256, "layer", None, 0, 182, False, True, BF), (264, "rms", None, 100, 10, True, False, BF),
    (768, "rms", None, 0, 768, False, False, BF), (1024, "layer", 1000, 24, 1000, False, True, BF),
    (1024, "rms", None, 0, 1024, True, False, F8),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[1]}-{s[4]}")
@pytest.mark.parametrize("N,heads", [(1, 1), (5, 3), (67, 13)])
def test_head_norm_rope_matches_64_bits(shape, N, heads):
    need_gpu()
    dsa = lib()
    dim, norm, nd, roff, rdim, inter, bias, ot = shape
    g = torch.Generator().manual_seed(dim * 7 + N)
    x = _randn(g, N, heads, dim)
    pos = torch.randint(0, 1 << 21, (N,), generator=g, dtype=torch.int32)
    pos[0] = 0
    s = _spec(g, dim, norm, nd, roff, rdim, inter, bias=bias)
    out = torch.zeros((N, heads, dim), dtype=ot, device="cuda")
    n0 = dsa.launch_count()
    dsa.head_norm_rope([dsa.HeadPart(x, out, **s)], pos.cuda())
    assert dsa.launch_count() == n0 + 1
    assert_heads_close(out, *transform64(x, pos, **s))


def test_one_launch_takes_strided_slices_and_leaves_their_neighbours():
    """Query and key slices of one fused projection, the rotated part of latent
    queries into the tail of their buffer, an FP8 tensor: four parts at once."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(5)
    N = 33
    qkv = _randn(g, N, 9, 72)
    proj = _randn(g, N, 6, 192)
    qi = _randn(g, 4, N, 128).transpose(0, 1)              # head-major input
    pos = torch.randint(0, 1 << 20, (N,), generator=g, dtype=torch.int32)
    buf = torch.full((N, 6, 576), 3.0, dtype=BF, device="cuda")
    wide = torch.full((5, N, 80), 7.0, dtype=BF, device="cuda")
    parts = [(qkv[:, :5], wide[:, :, 8:].transpose(0, 1), _spec(g, 72, rdim=40)),   # head-major out
             (qkv[:, 5:7], torch.empty((N, 2, 72), dtype=BF, device="cuda"), _spec(g, 72, rdim=72)),
             (proj[:, :, 128:], buf[:, :, 512:], _spec(g, 64, "none", rdim=64, inter=True)),
             (qi, torch.empty((N, 4, 128), dtype=F8, device="cuda"), _spec(g, 128, rdim=64))]
    plan = dsa.HeadParts([dsa.HeadPart(x, o, **s) for x, o, s in parts])
    n0 = dsa.launch_count()
    dsa.head_norm_rope(plan, pos.cuda())
    assert dsa.launch_count() == n0 + 1
    for k, (x, o, s) in enumerate(parts):
        assert_heads_close(o, *transform64(x, pos, **s), what=f"part {k}")
    assert bool((buf[:, :, :512] == 3.0).all()) and bool((wide[:, :, :8] == 7.0).all())


def test_in_place_and_repeated_calls():
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(6)
    x = _randn(g, 19, 3, 96)
    pos = torch.arange(100, 119, dtype=torch.int32)
    s = _spec(g, 96, rdim=50)
    want = transform64(x, pos, **s)
    out = torch.empty_like(x)
    dsa.head_norm_rope([dsa.HeadPart(x, out, **s)], pos.cuda())
    dsa.head_norm_rope([dsa.HeadPart(x, x, **s)], pos.cuda())
    assert torch.equal(x, out)
    assert_heads_close(out, *want)


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e30])
def test_zeros_specials_and_far_positions(scale):
    """A zero head stays zero; infinities and NaN stay inside their own head;
    the rotation holds at negative and at the largest positions."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(8)
    x = (torch.randn((6, 2, 64), generator=g) * scale).to(BF)
    x[1, 0] = 0.0
    x[2, 1, 5] = float("nan")
    x[3, 0, 9] = float("inf")
    pos = torch.tensor([-1, 0, 7, 1 << 21, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32)
    s = _spec(g, 64, "none", rdim=64)
    out = torch.empty((6, 2, 64), dtype=BF, device="cuda")
    dsa.head_norm_rope([dsa.HeadPart(x.cuda(), out, **s)], pos.cuda())
    o = out.cpu()
    assert bool((o[1, 0] == 0).all())
    assert int(torch.isnan(o[2, 1]).sum()) == 2            # the NaN's pair
    assert bool(torch.isfinite(o[2, 0]).all()) and bool(torch.isfinite(o[3, 1]).all())
    keep = [0, 1, 4, 5]
    w, e = transform64(x[keep], pos[keep], **s)
    assert_heads_close(out[keep], w, e)
    # NaN and overflow in E4M3: NaN stays NaN, the rest saturates
    f8 = torch.empty((6, 2, 64), dtype=F8, device="cuda")
    dsa.head_norm_rope([dsa.HeadPart(x.cuda(), f8)], None)
    w, e = transform64(x, pos)
    assert_heads_close(f8, w, e)


def test_dimensions_of_one_may_carry_any_stride():
    """One token of one head out of odd places: the strides of its unit
    dimensions say nothing."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(12)
    base = _randn(g, 4096)
    x = base.as_strided((1, 1, 64), (3, 5, 1), 64)
    room = torch.zeros(512, dtype=BF, device="cuda")
    out = room.as_strided((1, 1, 64), (7, 1, 1), 128)
    s = _spec(g, 64, rdim=64)
    pos = torch.tensor([77], dtype=torch.int32)
    dsa.head_norm_rope([dsa.HeadPart(x, out, **s)], pos.cuda())
    assert_heads_close(out, *transform64(x, pos, **s))
    assert bool((room[:128] == 0).all()) and bool((room[192:] == 0).all())


def test_many_tokens_of_every_kind_of_part():
    """Enough tokens for the long items: groups of 16 rounds, loops over four
    tokens, wide heads, and a last item that is not full."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(13)
    N = 9001
    pos = torch.randint(0, 1 << 20, (N,), generator=g, dtype=torch.int32)
    parts = []
    for heads, dim, ot, s in ((37, 128, F8, _spec(g, 128, rdim=64)),
                              (1, 576, BF, _spec(g, 576, norm_dim=512, roff=512, rdim=64, inter=True)),
                              (1, 64, BF, _spec(g, 64, "layer", rdim=64, bias=True)),
                              (2, 320, BF, _spec(g, 320, rdim=128))):
        x = _randn(g, N, heads, dim)
        parts.append((x, torch.empty((N, heads, dim), dtype=ot, device="cuda"), s))
    dsa.head_norm_rope([dsa.HeadPart(x, o, **s) for x, o, s in parts], pos.cuda())
    for k, (x, o, s) in enumerate(parts):
        assert_heads_close(o, *transform64(x, pos, **s), what=f"part {k}")


# dim, norm, rope offset, rope dim, interleaved, bias: rotations that begin or
# end inside 8 elements, halves of odd and even length, up to the whole head
LOOSE = [(40, "rms", 0, 26, False, False), (64, "layer", 2, 60, False, True),
         (104, "none", 6, 98, False, False), (128, "rms", 0, 72, False, True),
         (128, "layer", 10, 20, True, False), (200, "rms", 0, 200, False, False),
         (256, "layer", 0, 250, False, True), (256, "none", 4, 252, True, False)]


@pytest.mark.parametrize("shape", LOOSE, ids=lambda s: f"{s[0]}-{s[1]}-{s[3]}")
@pytest.mark.parametrize("N,heads", [(1, 9), (301, 1), (2003, 21)])
def test_rotations_that_end_inside_eight_elements(shape, N, heads):
    """Together, in one launch, with a rotation in whole eights and a part that
    is not rotated; values outside the rotation meet nothing of it."""
    need_gpu()
    dsa = lib()
    dim, norm, roff, rdim, inter, bias = shape
    g = torch.Generator().manual_seed(dim + rdim + N)
    pos = torch.randint(0, 1 << 21, (N,), generator=g, dtype=torch.int32)
    parts = []
    for h, d, ot, s in ((heads, dim, BF, _spec(g, dim, norm, None, roff, rdim, inter, bias=bias)),
                        (2, 64, F8, _spec(g, 64, rdim=64)), (1, 128, F8, _spec(g, 128, "layer"))):
        x = _randn(g, N, h, d)
        parts.append((x, torch.empty((N, h, d), dtype=ot, device="cuda"), s))
    if norm == "none" and roff:
        parts[0][0][0, 0, 0] = float("inf")
    dsa.head_norm_rope([dsa.HeadPart(x, o, **s) for x, o, s in parts], pos.cuda())
    for k, (x, o, s) in enumerate(parts):
        if k == 0 and norm == "none" and roff:
            assert float(o[0, 0, 0]) == float("inf")
            o[0, 0, 0] = x[0, 0, 0] = 0.0
        assert_heads_close(o, *transform64(x, pos, **s), what=f"part {k}")


def test_zero_tokens_launch_nothing():
    need_gpu()
    dsa = lib()
    x = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    n0 = dsa.launch_count()
    dsa.head_norm_rope([dsa.HeadPart(x, torch.empty_like(x))], None)
    assert dsa.launch_count() == n0


# ------------------------------------------------------------------ cache append --
def _paged(g, starts, T, bs, dims, extra=3):
    """Pools of random rows and a table with pages only where tokens go."""
    ends = [s + T for s in starts]
    maxb = max((e + bs - 1) // bs for e in ends)
    slots = [(b, s) for b, a in enumerate(starts) for s in range(a // bs, (ends[b] - 1) // bs + 1)]
    nb = len(slots) + extra
    perm = torch.randperm(nb, generator=g).tolist()
    bt = np.full((len(starts), maxb), -1, np.int32)
    for k, (b, s) in enumerate(slots):
        bt[b, s] = perm[k]
    pools = []
    for width, dt in dims:
        t = _randn(g, nb, bs, width)
        pools.append(t if dt == BF else t.to(F8))
    return bt, nb, ends, pools


def _check_pool(pool, before, bt, bs, seq, pos, want, fp32, width, what):
    rows = torch.from_numpy(bt[seq, pos // bs].astype(np.int64) * bs + pos % bs)
    u8 = lambda t: t.contiguous().view(torch.uint8).cpu().view(-1, t.shape[-1] * t.element_size())  # noqa: E731
    now, old = u8(pool), u8(before)
    e = pool.element_size()
    rest = torch.ones(now.shape, dtype=torch.bool)
    rest[rows, :width * e] = False
    assert torch.equal(now[rest], old[rest]), f"{what}: bytes no token names have changed"
    got = pool.reshape(-1, pool.shape[-1])[rows.to(pool.device)] if pool.dtype == BF else \
        pool.view(torch.uint8).reshape(-1, pool.shape[-1])[rows.to(pool.device)].view(F8)
    assert_heads_close(got[:, :width].reshape(want.shape), want, fp32, what)


@pytest.mark.parametrize("bs", [1, 16, 48, 64, 1024])
@pytest.mark.parametrize("form", ["append", "rows"])
def test_cache_append_latent_rows_and_fp8_keys(bs, form):
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(bs)
    starts = [0, 63, 64, 1000, 70001]
    T = 1 if form == "append" else 70
    bt, nb, ends, (kv, ki) = _paged(g, starts, T, bs, [(640, BF), (128, F8)])
    seq = np.repeat(np.arange(len(starts), dtype=np.int32), T)
    pos = np.concatenate([np.arange(s, s + T, dtype=np.int32) for s in starts])
    if form == "rows":
        order = torch.randperm(len(seq), generator=g).numpy()
        seq, pos = seq[order], pos[order]
    N = len(seq)
    x, xi = _randn(g, N, 1, 576), _randn(g, N, 1, 128)
    q = _randn(g, N, 5, 192)
    qo = torch.empty((N, 5, 64), dtype=BF, device="cuda")
    sk = _spec(g, 576, norm_dim=512, roff=512, rdim=64, inter=True)
    si = _spec(g, 128, "layer", rdim=64, bias=True)
    sq = _spec(g, 64, "none", rdim=64, inter=True)
    kv0, ki0 = kv.clone(), ki.clone()
    lay = dsa.PagedLayout(torch.from_numpy(bt).cuda(), torch.tensor(ends, dtype=torch.int32).cuda(),
                          bs, nb, max(ends))
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    args = (torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()) if form == "rows" else (None, None)
    n0 = dsa.launch_count()
    dsa.cache_append(lay, *args, [dsa.HeadPart(x, kv, **sk), dsa.HeadPart(xi, ki, **si)], ws,
                     heads=[dsa.HeadPart(q[:, :, 128:], qo, **sq)])
    assert dsa.launch_count() == n0 + 1
    p = torch.from_numpy(pos)
    _check_pool(kv, kv0, bt, bs, seq, pos, *transform64(x, p, **sk), 576, "latent rows")
    _check_pool(ki, ki0, bt, bs, seq, pos, *transform64(xi, p, **si), 128, "indexer keys")
    assert_heads_close(qo, *transform64(q[:, :, 128:], p, **sq), what="queries")
    assert dsa.get_status(ws) == 0


def test_cache_append_grouped_heads_into_separate_pools():
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(3)
    bs, starts, T = 32, [5, 31, 200], 3
    bt, nb, ends, (kp, vp, ki) = _paged(g, starts, T, bs, [(4 * 80, BF), (4 * 80, BF), (64, BF)])
    N = len(starts) * T
    seq = np.repeat(np.arange(3, dtype=np.int32), T)
    pos = np.concatenate([np.arange(s, s + T, dtype=np.int32) for s in starts])
    qkv, xi = _randn(g, N, 16, 80), _randn(g, N, 1, 64)
    sk, si = _spec(g, 80, rdim=48), _spec(g, 64, "layer", rdim=32, bias=True)
    before = [t.clone() for t in (kp, vp, ki)]
    lay = dsa.PagedLayout(torch.from_numpy(bt).cuda(), torch.tensor(ends, dtype=torch.int32).cuda(),
                          bs, nb, max(ends))
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    dsa.cache_append(lay, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                     [dsa.HeadPart(qkv[:, 8:12], kp.view(nb, bs, 4, 80), **sk),
                      dsa.HeadPart(qkv[:, 12:], vp), dsa.HeadPart(xi, ki, **si)], ws)
    p = torch.from_numpy(pos)
    for pool, old, x, s, w in ((kp, before[0], qkv[:, 8:12], sk, 320), (vp, before[1], qkv[:, 12:], {}, 320),
                               (ki, before[2], xi, si, 64)):
        want, e = transform64(x, p, **s)
        _check_pool(pool, old, bt, bs, seq, pos, want.reshape(N, 1, w), e.reshape(N, 1, w), w, "pool")


def test_cache_append_skips_and_flags_rows_out_of_range():
    """A sequence outside the batch, a negative position, a position past the
    table, a page id outside the pool: those rows are skipped, the others and
    every query written."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(4)
    bs, nb = 16, 4
    bt = np.array([[0, 9], [2, -5]], np.int32)
    pool = _randn(g, nb, bs, 64)
    before = pool.clone()
    seq = np.array([0, 0, 1, 1, 7, -1, 0, 1, 0], np.int32)
    pos = np.array([3, 16, 5, 20, 1, 1, -1, 32, 2147483647], np.int32)
    good = np.array([0, 2])
    x, q = _randn(g, 9, 1, 64), _randn(g, 9, 2, 64)
    qo = torch.empty_like(q)
    s = _spec(g, 64, rdim=64)
    lay = dsa.PagedLayout(torch.from_numpy(bt).cuda(),
                          torch.tensor([20, 20], dtype=torch.int32).cuda(), bs, nb, 32)
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    dsa.cache_append(lay, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                     [dsa.HeadPart(x, pool, **s)], ws, heads=[dsa.HeadPart(q, qo, **s)])
    p = torch.from_numpy(pos)
    want, e = transform64(x, p, **s)
    _check_pool(pool, before, bt, bs, seq[good], pos[good], want[good], e[good], 64, "good rows")
    near = np.arange(8)                                    # the last position is past 2^21
    wq, eq = transform64(q, p, **s)
    assert_heads_close(qo[:8], wq[near], eq[near], "queries")
    assert dsa.get_status(ws) == dsa.STATUS_BAD_BLOCK
    # the append form: sequences of length 0 have no row to write
    pool.copy_(before)
    lay0 = dsa.PagedLayout(torch.from_numpy(bt).cuda(),
                           torch.tensor([0, 6], dtype=torch.int32).cuda(), bs, nb, 32)
    dsa.cache_append(lay0, None, None, [dsa.HeadPart(x[:2], pool, **s)], ws)
    want, e = transform64(x[:2], torch.tensor([-1, 5]), **s)
    _check_pool(pool, before, bt, bs, np.array([1]), np.array([5]), want[1:], e[1:], 64, "append")
    assert dsa.get_status(ws) == dsa.STATUS_BAD_BLOCK and dsa.get_status(ws) == 0


def test_append_is_captured_and_replayed_with_new_lengths_on_a_side_stream():
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(9)
    bs, nb, B = 64, 9, 3
    bt = np.arange(9, dtype=np.int32).reshape(3, 3)
    lens = torch.tensor([1, 60, 129], dtype=torch.int32, device="cuda")
    lay = dsa.PagedLayout(torch.from_numpy(bt).cuda(), lens, bs, nb, 192)
    pool = _randn(g, nb, bs, 576)
    x = _randn(g, B, 1, 576)
    s = _spec(g, 576, norm_dim=512, roff=512, rdim=64, inter=True)
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    plan = dsa.HeadParts([dsa.HeadPart(x, pool, **s)])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        dsa.cache_append(lay, None, None, plan, ws)
    for step in range(3):
        x.copy_(_randn(g, B, 1, 576))
        lens.add_(1)
        before = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        pos = lens.cpu().numpy() - 1
        w, e = transform64(x, torch.from_numpy(pos), **s)
        _check_pool(pool, before, bt, bs, np.arange(3), pos, w, e, 576, f"step {step}")
