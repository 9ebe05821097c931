"""GPU tests of the 4-bit cache's decode attention at the edges of its ranges."""
import math

import pytest
import torch

from gpu_common import lib, need_gpu
from prompt_reference import assert_rows_close, attend_cache64, pack_rows, quantise64, values64
from test_gpu_cache4 import FP16, Attn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# Sums over 2^31 positions: a warp has 2^31 / 2432 of them, its lane 110,000 fp32 additions (each off
# by half a step, 2^-25, of a sum that is half of the last on average: together 2^-24 * 55,000) and its
# products 55,000 accumulations (each cut off, 2^-23, likewise: 2^-23 * 27,500); beside these 2^-11 for
# a weight as fp16 and 2^-11 for its score.
LONG = 55000 * 2.0 ** -24 + 27500 * 2.0 ** -23 + 2.0 ** -10


@pytest.mark.parametrize("D,bs", [(64, 64), (64, 48), (128, 32), (256, 16)])
def test_whole_tiles_in_the_place_of_partial_ones(D, bs):
    """Tiles that a sequence's end or a bad page leaves partly unused have V's scales patched in place;
    the rows that come into their stage next keep all of theirs, call after call."""
    need_gpu()
    dsa = lib()
    p = Attn(40 + D, [(1 + 37 * i) % 300 if i % 2 else 512 for i in range(400)], Hq=4, Hk=2, Dk=D, bs=bs)
    p.bt[3::40, 0] = -1
    p.run(dsa)
    assert dsa.get_status(p.ws) == dsa.STATUS_BAD_BLOCK
    p.check(f"{D}, pages of {bs}")
    first, lse = p.out.clone(), p.lse.clone()
    for _ in range(50):
        p.out.fill_(3.0)
        p.call(dsa)
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("ks", [1e-7, 1e-8, 1e-30, 1e-45])
@pytest.mark.parametrize("bs", [64, 48])
def test_a_vanishing_score_factor_leaves_the_mean(ks, bs):
    """Queries of zeros or next to it behind head scales next to it: every weight is 1 / n, also in
    tiles that the sequence's end or a bad page leaves partly unused."""
    need_gpu()
    dsa = lib()
    for q_amp in (0.0, 1e-30):
        p = Attn(41, [70, 300, 1, 513, 0], Hq=12, Hk=2, Dk=64, bs=bs, scaled=True, q_amp=q_amp)
        p.ks = torch.full((2,), ks, device="cuda")
        p.bt[1, 1] = -1
        p.run(dsa)
        assert dsa.get_status(p.ws) == dsa.STATUS_BAD_BLOCK
        p.check(f"{q_amp} x {ks}")


@pytest.mark.parametrize("short", [0, 1, 510, 511, 700])
def test_lengths_next_to_the_largest(short):
    """2^31 - 1 positions and somewhat fewer, over the same three pages again and again but for the
    table's last; queries along the last position's key, which decides heads 0 and 2 where it is long."""
    need_gpu()
    dsa = lib()
    L, bs, D = (1 << 31) - 1 - short, 1024, 16
    p = Attn(42, [4 * bs], Hq=4, Hk=2, Dk=D, bs=bs)
    p.lay = p.layout(dsa)
    pages = p.bt[0].long()
    slots = torch.arange((L + bs - 1) // bs) % 3
    slots[-1] = 3
    p.lay = dsa.PagedLayout(pages[slots].to(torch.int32)[None].cuda(), torch.tensor([L], dtype=torch.int32).cuda(), bs,
                            p.nb, L)
    rows = p.pool.cpu()[pages].permute(1, 0, 2, 3)                       # [Hk][4 pages][bs][row]
    k, v = values64(rows.flatten(0, 2), D, D)                            # [2 * 4 * bs][D]
    k, v = k.view(2, 4, bs, D), v.view(2, 4, bs, D)
    last = (L - 1) % bs
    p.q[0, 0], p.q[0, 2] = (k[0, 3, last] * 256).to(BF), (k[1, 3, last] * 256).to(BF)
    p.ws = dsa.workspace(dsa.cache4_attn_decode_workspace_size(1, 4, 2, D, D))
    p.call(dsa)
    assert dsa.get_status(p.ws) == 0
    count = torch.bincount(slots, minlength=4).double()[:, None].expand(4, bs).clone()
    count[3] = (torch.arange(bs) <= last).double()
    for h in range(4):
        z = (k[h // 2] @ p.q[0, h].double().cpu()) * p.scale
        z = torch.where(count > 0, z + count.log(), -math.inf)
        l = torch.logsumexp(z.flatten(), 0)
        w = torch.exp(z - l)
        # a single position's weight that is small beside the largest is lost below fp16's range: off by
        # itself at most, and by 2^-32 of the largest (which stands at 2^7, and half a step is 2^-25)
        one = torch.where(count > 0, w / count.clamp(min=1), 0.0)
        lost = count * torch.minimum(one, 2.0 ** -32 * one.max())
        want, mag = (w[..., None] * v[h // 2]).sum((0, 1)), (w[..., None] * v[h // 2].abs()).sum((0, 1))
        tol = 2.0 ** -8 * want.abs() + LONG * mag + (lost[..., None] * v[h // 2].abs()).sum((0, 1))
        assert abs(float(p.lse[0, h]) - float(l)) <= LONG, h
        assert bool(((p.out[0, h].double().cpu() - want).abs() <= tol).all()), h


@pytest.mark.parametrize("Hk,G,D,bs,L", [(1, 16, 64, 64, 6000), (2, 8, 64, 48, 2500), (1, 16, 128, 128, 4000),
                                         (1, 4, 256, 32, 1500), (1, 24, 80, 1, 700)])
def test_every_position_counts_once(Hk, G, D, bs, L):
    """Keys of +-1 behind 16 sequences of about the same positions: every row asks for a position by its
    key's signs, next to the borders of tiles, units and CTAs and all others in turn."""
    need_gpu()
    dsa = lib()
    B = 16
    one = Attn(43, [L], Hq=Hk * G, Hk=Hk, Dk=D, bs=bs, fill=False)
    k = torch.where(torch.randn((L, Hk, D), generator=one.g) > 0, 1.0, -1.0).to(BF)
    v = torch.randn((L, Hk, D), generator=one.g).to(BF)
    rows = pack_rows(quantise64(k), quantise64(v), one.row)
    i = torch.arange(L)
    pool = one.pool.cpu()
    pool[one.bt[0].long()[i // bs], :, i % bs] = rows
    k, v = (x.cuda() for x in values64(rows, D, D))                     # [L][Hk][D]
    lens = torch.tensor([L - b for b in range(B)], dtype=torch.int32).cuda()
    lay = dsa.PagedLayout(one.bt.expand(B, -1).contiguous().cuda(), lens, bs, one.nb, L)
    pool, out = pool.cuda(), torch.empty((B, Hk * G, D), dtype=BF, device="cuda")
    lse = torch.empty((B, Hk * G), device="cuda")
    ws = dsa.workspace(dsa.cache4_attn_decode_workspace_size(B, Hk * G, Hk, D, D))
    heads = torch.arange(Hk * G, device="cuda") // G
    hidden = torch.arange(L, device="cuda") >= lens[:, None, None]
    for r in range(-(-L // (B * G))):
        target = (torch.arange(B * G, device="cuda").view(B, 1, G) + r * B * G).expand(B, Hk, G).reshape(B, -1)
        target = torch.minimum(target, lens[:, None] - 1).long()
        q = torch.sign(k[target, heads.expand_as(target)]).to(BF)
        out.fill_(5.0)
        dsa.cache4_attn_decode(lay, q, pool, 1.0, out, lse, ws)
        z = torch.einsum("bhd,lhd->bhl", q.double(), k[:, heads]).masked_fill_(hidden, -math.inf)
        l = torch.logsumexp(z, -1)
        w = torch.exp(z - l[..., None])
        o, m = torch.einsum("bhl,lhd->bhd", w, v[:, heads]), torch.einsum("bhl,lhd->bhd", w, v[:, heads].abs())
        # (keys are of one size, so scores have few bits; a weight is off by 2^-11, or by 2^-32 of the largest)
        tol = 2.0 ** -8 * o.abs() + 2.0 ** -10 * m + 2.0 ** -32 * v[:, heads].abs().sum(0)
        d = (out.double() - o).abs()
        assert bool((d <= tol).all()), (d > tol).any(-1).nonzero()[0].tolist()
        # (a score below 264 is 2^8.6 in log2 units, and rounded at most four times)
        assert float((lse.double() - l).abs().max()) <= 2.0 ** -13
    assert dsa.get_status(ws) == 0


@pytest.mark.parametrize("power", [0, 5, 10, 12, 14, 16, 18, 20, 25, 30, 60, 115])
def test_scores_of_any_size(power):
    """Scores of up to 64 * 2^power, up to where fp32 ends, every position of a tile's pattern 40 times over:
    the places of the key that a head asks for share the row evenly."""
    need_gpu()
    dsa = lib()
    D, n, times, Hq = 64, 100, 40, 16
    p = Attn(44, [n * times, n * times - 33], Hq=Hq, Hk=1, Dk=D, fill=False)
    k = torch.where(torch.randn((n, 1, D), generator=p.g) > 0, 1.0, -1.0).to(BF)
    v = torch.randn((n * times, 1, D), generator=p.g).to(BF)
    rows = pack_rows(quantise64(k.repeat(times, 1, 1)), quantise64(v), p.row)
    pool = p.pool.cpu()
    for b in range(2):
        i = torch.arange(p.lens[b])
        pool[p.bt[b].long()[i // 64], :, i % 64] = rows[:p.lens[b]]
    p.pool, p.scale = pool.cuda(), 1.0
    p.q = (k[torch.arange(2 * Hq) * 3, 0].view(2, Hq, D).double() * 2.0 ** power).to(BF).cuda()
    p.run(dsa)
    assert dsa.get_status(p.ws) == 0
    o, l, m, total = attend_cache64(p.q, p.pool, p.bt, p.lens, 64, p.nb, D, D, 1.0)
    assert_rows_close(p.out, None, o, l, m, FP16, f"2^{power}", floor=2.0 ** -32 * total)
    # a score of 68 * 2^power is 2^(6.7 + power) in log2 units, and rounded at most four times
    assert bool(((p.lse.double().cpu() - l).abs() <= 2.0 ** (power - 15)).all())


def test_large_scores_that_rise_by_less_than_the_lag():
    """Maxima of 2^12 to 2^21 that rise by up to 8 (log2) from tile to tile: no weight passes fp16's range."""
    need_gpu()
    dsa = lib()
    n = 4096
    for top in (4e3, 1e5, 5e5, 7e5, 1.4e6):
        p = Attn(45, [n], Hq=2, Hk=1, Dk=32, fill=False)
        k = torch.zeros((n, 1, 32), dtype=BF)
        k[:, :, :16] = 6.0                                               # codes of 6 behind a scale of 1
        k[:, 0, 16] = 6.0
        k[:, 0, 17] = (torch.arange(n) // 64 % 5).to(BF)                 # 0 to 4
        rows = pack_rows(quantise64(k), quantise64(torch.randn((n, 1, 32), generator=p.g).to(BF)), p.row)
        i = torch.arange(n)
        pool = p.pool.cpu()
        pool[p.bt[0].long()[i // 64], :, i % 64] = rows
        p.pool, p.scale = pool.cuda(), 1.0
        p.q.zero_()
        p.q[0, :, 0] = float(torch.tensor(top / 6).to(BF))
        p.q[0, :, 17] = 1.25
        p.run(dsa)
        o, l, m, total = attend_cache64(p.q, p.pool, p.bt, p.lens, 64, p.nb, 32, 32, 1.0)
        # a score is exact; its product with log2(e), where rounded, is off by half a step, 2^-24 of it, and a
        # weight by that power of two
        weight = 2.0 ** (2 * top * 1.4427 * 2.0 ** -24) - 1
        assert_rows_close(p.out, None, o, l, m, FP16 + weight, f"{top}", floor=2.0 ** -32 * total)
