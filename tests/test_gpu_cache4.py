"""GPU tests of the 4-bit cache: bytes against the definition, attention against 64 bits."""
import math

import pytest
import torch

from gpu_common import lib, need_gpu
from heads_reference import assert_heads_close, transform64
from prompt_reference import (assert_rows_close, attend_cache64, attend_prompt64, pack_rows, quantise64,
                              values64)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FP16 = 2.0 ** -11                       # weights as fp16


class Cache:
    """A paged 4-bit cache whose bytes outside every sequence are NaN scales (0xff)."""

    def __init__(self, seed, lens, Hk, Dk, Dv=None, bs=64, scaled=False, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.Hk, self.Dk, self.Dv, self.bs = g, list(lens), Hk, Dk, Dv or Dk, bs
        need = [(n + bs - 1) // bs for n in lens]
        self.nb = sum(need) + 2
        perm = torch.randperm(self.nb, generator=g).to(torch.int32)
        self.bt = torch.full((len(lens), max(1, *need)), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        self.ks, self.vs = ((torch.rand(Hk, generator=g) + 0.5, torch.rand(Hk, generator=g) + 0.5)
                            if scaled else (None, None))
        self.row = (9 * (self.Dk + self.Dv) // 16 + 15) // 16 * 16
        pool = torch.full((self.nb, Hk, bs, self.row), 0xff, dtype=torch.uint8)
        if fill:
            for b, n in enumerate(lens):
                p = torch.arange(n)
                k, v = torch.randn((n, Hk, self.Dk), generator=g).to(BF), torch.randn((n, Hk, self.Dv), generator=g).to(BF)
                rows = pack_rows(quantise64(k, self.ks), quantise64(v, self.vs), self.row)
                pool[self.bt[b].long()[p // bs], :, p % bs] = rows
        self.pool = pool.cuda()
        if scaled:
            self.ks, self.vs = self.ks.cuda(), self.vs.cuda()

    def layout(self, dsa, max_len=None):
        self.dev_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return dsa.PagedLayout(self.bt.cuda(), self.dev_lens, self.bs, self.nb,
                               max(self.lens) if max_len is None else max_len)


class Attn(Cache):
    def __init__(self, seed, lens, Hq, q_amp=1.0, **kw):
        super().__init__(seed, lens, **kw)
        self.q = (torch.randn((len(lens), Hq, self.Dk), generator=self.g) * q_amp).to(BF).cuda()
        self.Hq, self.scale = Hq, self.Dk ** -0.5
        self.out = torch.full((len(lens), Hq, self.Dv), 5.0, dtype=BF, device="cuda")
        self.lse = torch.full((len(lens), Hq), 5.0, device="cuda")

    def run(self, dsa, ws=None, lse=True):
        self.lay = self.layout(dsa)
        self.ws = ws if ws is not None else dsa.workspace(
            dsa.cache4_attn_decode_workspace_size(len(self.lens), self.Hq, self.Hk, self.Dk, self.Dv))
        self.call(dsa, lse=lse)
        torch.cuda.synchronize()
        return self

    def call(self, dsa, lse=True, **kw):
        dsa.cache4_attn_decode(self.lay, self.q, self.pool, self.scale, self.out, self.lse if lse else None,
                               self.ws, k_scale=self.ks, v_scale=self.vs, **kw)

    def check(self, what="", lens=None):
        # Weights are kept 2^7 above their size, the largest at 2^7 or more, and fp16's smallest half
        # step is 2^-25: a weight is off by 2^-11 of itself or by 2^-32 of the largest, which is at most
        # 1 after the division by their sum; so the result by at most 2^-32 sum |v| more.
        o, l, m, total = attend_cache64(self.q, self.pool, self.bt, lens or self.lens, self.bs, self.nb,
                                        self.Dk, self.Dv, self.scale, self.ks, self.vs)
        assert_rows_close(self.out, self.lse, o, l, m, FP16, what, floor=2.0 ** -32 * total)


# ------------------------------------------------------------------------------- write, read
def hard_values(g, N, H, D):
    """Groups whose elements lie on and next to the borders between codes, of every exponent; zeros
    of both signs, subnormals, infinities and NaN."""
    m = torch.randint(128, 256, (N, H, D // 16, 16), generator=g).double()
    x = m * 2.0 ** torch.randint(-11, -6, m.shape, generator=g).double()
    e = torch.randint(-60, 60, (N, H, D // 16, 1), generator=g).double()
    e = torch.where(torch.rand(e.shape, generator=g) < 0.7, e / 6, e)
    x = (x * 2.0 ** e.round() * (1 - 2 * torch.randint(0, 2, m.shape, generator=g))).flatten(-2)
    odd = torch.tensor([0.0, -0.0, 1e-40, -1e-40, math.inf, -math.inf, math.nan, 3e38], dtype=torch.float64)
    pick = odd[torch.randint(0, 8, x.shape, generator=g)]
    return torch.where(torch.rand(x.shape, generator=g) < 0.01, pick, x).to(BF)


@pytest.mark.parametrize("Hk,Dk,Dv", [(1, 16, 16), (3, 128, 128), (8, 64, 64), (2, 256, 48), (5, 80, 112),
                                      (1, 240, 256), (40, 16, 32)])
@pytest.mark.parametrize("scales", [None, (1.0, 0.7, 1 / 3, 3.0, 1.25), (6.0, 1e-3, 1e25, 1e-30, 0.9999999)])
def test_written_bytes_are_those_of_the_definition(Hk, Dk, Dv, scales):
    need_gpu()
    dsa = lib()
    N = 300
    c = Cache(Hk + Dk, [N], Hk, Dk, Dv, bs=48, fill=False)
    k, v = hard_values(c.g, N, Hk, Dk), hard_values(c.g, N, Hk, Dv)
    ks = vs = None
    if scales:
        ks = torch.tensor(scales, dtype=torch.float32).repeat(8)[:Hk].cuda()
        vs = ks.flip(0).contiguous()
    pos = torch.randperm(N, generator=c.g).to(torch.int32).cuda()
    seq = torch.zeros(N, dtype=torch.int32, device="cuda")
    ws = dsa.workspace(dsa.cache4_write_workspace_size())
    ko, vo = torch.empty((N, Hk, Dk), dtype=BF).cuda(), torch.empty((N, Hk, Dv), dtype=BF).cuda()
    want = pack_rows(quantise64(k, ks), quantise64(v, vs), c.row)
    kept = values64(want, Dk, Dv, ks, vs)
    for back in (False, True):
        pool = c.pool.clone()
        dsa.cache4_write(c.layout(dsa), seq, pos, k.cuda(), v.cuda(), pool, ws, k_scale=ks, v_scale=vs,
                         k_out=ko if back else None, v_out=vo if back else None)
        assert dsa.get_status(ws) == 0
        p = pos.cpu().long()
        got = pool.cpu()[c.bt[0].long()[p // 48], :, p % 48]
        assert torch.equal(got, want)
        untouched = torch.ones(pool.shape[:3], dtype=torch.bool)
        untouched[c.bt[0].long()[p // 48], :, p % 48] = False
        assert bool((pool.cpu()[untouched] == 0xff).all())
    ki, vi = torch.empty_like(ko), torch.empty_like(vo)
    dsa.cache4_read(c.layout(dsa), seq, pos, pool, ki, vi, ws, k_scale=ks, v_scale=vs)
    # (codes times scales are exact; times a head scale one fp32 rounding and one to bf16)
    for got, again, x in ((ko, ki, kept[0]), (vo, vi, kept[1])):
        assert torch.equal(got.view(torch.int16), again.view(torch.int16))
        g = got.double().cpu()
        assert torch.equal(torch.isnan(g), torch.isnan(x))
        fin = ~torch.isnan(x) & (x.abs() < 3e38)
        assert bool(((g - x).abs()[fin] <= (2.0 ** -8 + 2.0 ** -23) * x.abs()[fin] + 1e-40).all())
        if scales is None:
            assert torch.equal(g[fin], x[fin])


@pytest.mark.parametrize("layout", ["fused", "heads", "wide"])
def test_strided_rows(layout):
    need_gpu()
    dsa = lib()
    N, Hk, D = 77, 4, 96
    c = Cache(3, [N], Hk, D, bs=16, fill=False)
    x = torch.randn((N, 2 * Hk, D), generator=c.g).to(BF)
    if layout == "fused":
        xs = x.cuda()
        k, v = xs[:, :Hk], xs[:, Hk:]
    elif layout == "heads":
        xs = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        k, v = xs[:, :Hk], xs[:, Hk:]
    else:
        buf = torch.zeros((N, 2 * Hk, D + 8), dtype=BF, device="cuda")
        buf[:, :, 8:] = x.cuda()
        k, v = buf[:, :Hk, 8:], buf[:, Hk:, 8:]
    ws = dsa.workspace(dsa.cache4_write_workspace_size())
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    dsa.cache4_write(c.layout(dsa), torch.zeros_like(pos), pos, k, v, c.pool, ws)
    want = pack_rows(quantise64(x[:, :Hk]), quantise64(x[:, Hk:]), c.row)
    p = pos.cpu().long()
    assert torch.equal(c.pool.cpu()[c.bt[0].long()[p // 16], :, p % 16], want)


def test_append_form_and_tokens_without_a_place():
    need_gpu()
    dsa = lib()
    lens = [5, 64, 65, 1, 0, 130]
    c = Cache(4, lens, 2, 64, bs=64, fill=False)
    k, v = (torch.randn((6, 2, 64), generator=c.g).to(BF).cuda() for _ in range(2))
    ws = dsa.workspace(dsa.cache4_write_workspace_size())
    dsa.cache4_write(c.layout(dsa), None, None, k, v, c.pool, ws)
    assert dsa.get_status(ws) == dsa.STATUS_BAD_BLOCK        # the empty sequence has no position
    want = pack_rows(quantise64(k), quantise64(v), c.row)
    full = torch.full_like(c.pool, 0xff).cpu()
    for b, n in enumerate(lens):
        if n:
            full[int(c.bt[b, (n - 1) // 64]), :, (n - 1) % 64] = want[b]
    assert torch.equal(c.pool.cpu(), full)
    # sequences, positions and pages out of range: nothing stored, the values come back all the same
    c.bt[1, 0] = c.nb
    seq = torch.tensor([0, -1, 6, 0, 1, 5], dtype=torch.int32, device="cuda")
    pos = torch.tensor([-1, 0, 0, 1000000, 3, 3], dtype=torch.int32, device="cuda")
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    dsa.cache4_write(c.layout(dsa), seq, pos, k, v, c.pool, ws, k_out=ko, v_out=vo)
    assert dsa.get_status(ws) == dsa.STATUS_BAD_BLOCK
    full[int(c.bt[5, 0]), :, 3] = want[5]
    assert torch.equal(c.pool.cpu(), full)
    kept = values64(want, 64, 64)
    assert torch.equal(ko.double().cpu(), kept[0]) and torch.equal(vo.double().cpu(), kept[1])
    dsa.cache4_read(c.layout(dsa), seq, pos, c.pool, ko, vo, ws)
    assert dsa.get_status(ws) == dsa.STATUS_BAD_BLOCK
    assert bool((ko[:5] == 0).all()) and bool((vo[:5] == 0).all())
    assert torch.equal(ko[5].double().cpu(), kept[0][5])
    none = k[:0]
    dsa.cache4_write(c.layout(dsa), seq[:0], pos[:0], none, none, c.pool, ws)  # no tokens
    dsa.cache4_read(c.layout(dsa), seq[:0], pos[:0], c.pool, none, none, ws)
    assert dsa.get_status(ws) == 0 and torch.equal(c.pool.cpu(), full)


def test_a_position_named_twice_holds_bytes_of_either():
    """... and no other position is touched."""
    need_gpu()
    dsa = lib()
    c = Cache(5, [300], 3, 64, bs=64, fill=False)
    N = 200
    k, v = (torch.randn((N, 3, 64), generator=c.g).to(BF).cuda() for _ in range(2))
    pos = (torch.arange(N, device="cuda", dtype=torch.int32) % 100)          # each of 100 twice
    ws = dsa.workspace(dsa.cache4_write_workspace_size())
    dsa.cache4_write(c.layout(dsa), torch.zeros_like(pos), pos, k, v, c.pool, ws)
    assert dsa.get_status(ws) == 0
    want = pack_rows(quantise64(k), quantise64(v), c.row).cpu()              # [N][Hk][row]
    pool = c.pool.cpu()
    got = torch.stack([pool[int(c.bt[0, p // 64]), :, p % 64] for p in range(300)])
    assert bool(((got[:100] == want[:100]) | (got[:100] == want[100:])).all())
    assert bool((got[100:] == 0xff).all())


# ------------------------------------------------------------------------------- attention
CASES = {
    "one-position": dict(lens=[1], Hq=1, Hk=1, Dk=64),
    "empty": dict(lens=[0, 0], Hq=4, Hk=2, Dk=64),
    "tile-edges": dict(lens=[31, 32, 33, 0, 255, 256, 257, 63, 64, 65, 511, 512, 513], Hq=8, Hk=2, Dk=64),
    "tile-edges-128": dict(lens=[31, 32, 33, 0, 255, 256, 257, 63, 64, 65], Hq=8, Hk=2, Dk=128),
    "long-ragged": dict(lens=[5000, 3, 1, 8191, 2049], Hq=16, Hk=2, Dk=128, scaled=True),
    "sixteen-heads": dict(lens=[4096], Hq=16, Hk=1, Dk=128),
    "head-blocks": dict(lens=[700, 90], Hq=40, Hk=2, Dk=64, scaled=True),
    "head-blocks-wide": dict(lens=[700, 90], Hq=40, Hk=2, Dk=256),
    "head-blocks-24": dict(lens=[300, 1], Hq=24, Hk=1, Dk=128, Dv=96),
    "odd-dims": dict(lens=[900, 513, 777, 1], Hq=18, Hk=3, Dk=80, Dv=112, bs=48, scaled=True),
    "smallest-dims": dict(lens=[130, 99], Hq=3, Hk=3, Dk=16, bs=24),
    "k-wide": dict(lens=[600, 17], Hq=5, Hk=5, Dk=256, Dv=16, bs=128),
    "v-wide": dict(lens=[600, 17], Hq=5, Hk=5, Dk=32, Dv=240, bs=32),
    "three-chunks": dict(lens=[333, 400], Hq=4, Hk=4, Dk=192, Dv=176, bs=16),
    "page-1": dict(lens=[260, 70], Hq=16, Hk=2, Dk=64, bs=1),
    "page-7": dict(lens=[260, 70, 300], Hq=8, Hk=1, Dk=128, bs=7),
    "page-1024": dict(lens=[3000, 1500], Hq=8, Hk=1, Dk=128, bs=1024),
    "page-96": dict(lens=[3000, 95, 96, 97], Hq=8, Hk=1, Dk=64, bs=96),
    "many": dict(lens=[(37 * i) % 300 for i in range(150)], Hq=8, Hk=4, Dk=64, bs=32),
    "many-long": dict(lens=[1000 + 61 * i for i in range(40)], Hq=4, Hk=4, Dk=128),
}


@pytest.mark.parametrize("name", CASES)
def test_cache4_attention_matches_64_bits(name):
    need_gpu()
    dsa = lib()
    p = Attn(sum(map(ord, name)), **CASES[name]).run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check(name)
    first, lse = p.out.clone(), p.lse.clone()
    for _ in range(30):                        # equal bit for bit, whatever the warps' order
        p.out.fill_(3.0)
        p.call(dsa)
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    p.call(dsa, lse=False)
    assert torch.equal(p.out, first)


@pytest.mark.parametrize("Dk,Dv", [(16 * i, 16 * ((5 * i) % 16 + 1)) for i in range(1, 17)])
def test_every_width(Dk, Dv):
    need_gpu()
    dsa = lib()
    p = Attn(Dk, [300, 65], Hq=6, Hk=2, Dk=Dk, Dv=Dv, scaled=True).run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check(f"{Dk} / {Dv}")


@pytest.mark.parametrize("amp", [1e-30, 1e-3, 30.0, 1e30])
def test_query_magnitudes(amp):
    """Queries far outside fp16's range; scores of hundreds, where one position decides."""
    need_gpu()
    dsa = lib()
    p = Attn(7, [900, 64], Hq=4, Hk=2, Dk=128, q_amp=amp)
    if amp > 1e10:
        p.scale /= amp
    p.run(dsa).check(f"queries of {amp}")
    p = Attn(8, [70], Hq=4, Hk=2, Dk=64)
    p.q[0, 1] = 0.0
    p.run(dsa).check("a query of zeros")


def test_a_maximum_that_keeps_rising():
    need_gpu()
    dsa = lib()
    p = Attn(9, [3000], Hq=2, Hk=1, Dk=64, fill=False)
    k = (torch.arange(3000)[:, None, None] * 0.02 * torch.ones(64)).to(BF)
    v = torch.randn((3000, 1, 64), generator=p.g).to(BF)
    rows = pack_rows(quantise64(k), quantise64(v), p.row)
    i = torch.arange(3000)
    pool = p.pool.cpu()
    pool[p.bt[0].long()[i // 64], :, i % 64] = rows
    p.pool = pool.cuda()
    p.q[:] = 1.0
    p.run(dsa).check("rising")


def test_bad_block_ids_are_left_out_and_flagged():
    need_gpu()
    dsa = lib()
    for bs in (64, 48):
        p = Attn(11, [700, 520], Hq=8, Hk=2, Dk=64, bs=bs)
        p.bt[0, 7], p.bt[1, 3] = p.nb + 3, -1
        p.run(dsa).check("bad pages")
        assert dsa.get_status(p.ws) == dsa.STATUS_BAD_BLOCK
        p.bt[:] = 1 << 30
        p.run(dsa)
        assert bool((p.out == 0).all()) and bool((p.lse == -math.inf).all())


def test_lengths_beyond_the_bound_are_cut_and_flagged():
    need_gpu()
    dsa = lib()
    p = Attn(12, [128, 100], Hq=4, Hk=2, Dk=64).run(dsa)
    p.dev_lens.copy_(torch.tensor([100000, 100], dtype=torch.int32))
    p.call(dsa)
    p.check("cut", lens=[128, 100])
    assert dsa.get_status(p.ws) == dsa.STATUS_BAD_LENGTH
    p.dev_lens.copy_(torch.tensor([-5, 100], dtype=torch.int32))
    p.call(dsa)
    p.check("negative", lens=[0, 100])


def test_a_nan_stays_in_its_sequence_and_head():
    need_gpu()
    dsa = lib()
    p = Attn(13, [700, 900, 650], Hq=8, Hk=2, Dk=128).run(dsa)
    want = p.out.clone()
    p.q[0, 5, 100] = math.nan
    page = int(p.bt[2, 640 // 64])
    p.pool[page, 1, 640 % 64, 128] = 0x7f              # a K scale of key head 1
    p.pool[int(p.bt[1, 0]), 0, 3, 136] = 0x7f          # a V scale of key head 0
    p.run(dsa, ws=p.ws)
    keep = torch.ones((3, 8), dtype=torch.bool)
    keep[0, 5] = False
    keep[2, 4:] = False
    keep[1, :4] = False
    assert torch.equal(p.out.cpu()[keep], want.cpu()[keep])
    assert bool(torch.isnan(p.out[0, 5].float()).all()) and bool(torch.isnan(p.out[2, 4:].float()).all())
    assert bool(torch.isnan(p.out[1, :4, :16].float()).all()) and bool(torch.isfinite(p.out[1, :4, 16:].float()).all())


def test_two_streams_and_a_shared_workspace_on_one():
    need_gpu()
    dsa = lib()
    ps = [Attn(20 + i, [1500 + i, 1300, 29], Hq=16, Hk=2, Dk=128).run(dsa) for i in range(2)]
    want = [p.out.clone() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    for p in ps:
        p.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for p, st in zip(ps, streams):
            p.call(dsa, stream=st)
    torch.cuda.synchronize()
    for p, w in zip(ps, want):
        assert torch.equal(p.out, w)
    others = [Attn(i, **CASES[n]) for i, n in enumerate(("head-blocks", "one-position", "many", "k-wide"))]
    ws = dsa.workspace(max(dsa.cache4_attn_decode_workspace_size(len(p.lens), p.Hq, p.Hk, p.Dk, p.Dv)
                           for p in others))
    for p in others + others:
        p.run(dsa, ws=ws).check("shared workspace")


def test_captured_call_follows_the_lengths():
    need_gpu()
    dsa = lib()
    p = Attn(30, [1200, 1100, 64], Hq=16, Hk=4, Dk=64).run(dsa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call(dsa)
    for lens in ([1200, 1100, 64], [1001, 1, 64], [5, 1099, 0], [0, 0, 0]):
        p.dev_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check(f"lens {lens}", lens=lens)


def test_a_pool_beyond_32_bits():
    need_gpu()
    dsa = lib()
    Hk, D, bs = 8, 128, 64
    nb = (1 << 32) // (Hk * bs * 144) + 200                # 4 GB of rows
    small = Attn(31, [1500, 700], Hq=16, Hk=Hk, Dk=D)
    pool = torch.zeros((nb, Hk, bs, 144), dtype=torch.uint8, device="cuda")
    pool[nb - small.nb:] = small.pool
    small.run(dsa)
    want = small.out.clone()
    small.bt += nb - small.nb
    small.pool, small.nb = pool, nb
    small.run(dsa)
    assert dsa.get_status(small.ws) == 0 and torch.equal(small.out, want)
    ws = dsa.workspace(dsa.cache4_write_workspace_size())
    k, v = (torch.randn((2, Hk, D), generator=small.g).to(BF).cuda() for _ in range(2))
    dsa.cache4_write(small.lay, None, None, k, v, pool, ws)
    rows = pack_rows(quantise64(k), quantise64(v), 144)
    for b, n in enumerate(small.lens):
        assert torch.equal(pool[int(small.bt[b, (n - 1) // bs]), :, (n - 1) % bs].cpu(), rows[b])


def test_a_prompt_then_decode_steps_over_the_4_bit_cache():
    """Raw projections -> head_norm_rope -> cache4_write with the values kept -> prompt_attn over them;
    a second chunk behind the cached prefix by cache4_read; then decode steps by cache4_write (append)
    and cache4_attn_decode.  Every output against 64 bits on the kept values, and the last prompt
    token's by both attentions."""
    need_gpu()
    dsa = lib()
    Hq, Hk, D, bs, n1, n2 = 12, 2, 128, 64, 150, 90
    g = torch.Generator().manual_seed(50)
    total = n1 + n2 + 3
    qkv = torch.randn((total, Hq + 2 * Hk, D), generator=g).to(BF).cuda()
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    pos = torch.arange(total, dtype=torch.int32, device="cuda")
    q, k = torch.empty((total, Hq, D), dtype=BF, device="cuda"), torch.empty((total, Hk, D), dtype=BF, device="cuda")
    spec = dict(norm="rms", weight=w, rope_dim=D, inv_freq=f)
    dsa.head_norm_rope([dsa.HeadPart(qkv[:, :Hq], q, **spec), dsa.HeadPart(qkv[:, Hq:Hq + Hk], k, **spec)], pos)
    want, e = transform64(qkv[:, :Hq], pos, **spec)
    assert_heads_close(q, want, e, "queries")
    v = qkv[:, Hq + Hk:]
    nb = (total + bs - 1) // bs
    lens = torch.tensor([n1], dtype=torch.int32, device="cuda")
    lay = dsa.PagedLayout(torch.randperm(nb, generator=g).to(torch.int32).view(1, -1).cuda(), lens, bs, nb, total)
    pool = dsa.cache4_pool(nb, Hk, bs, D, D)
    ws = dsa.workspace(dsa.cache4_write_workspace_size())
    wp = dsa.workspace(dsa.prompt_attn_workspace_size(1, n1, Hq, Hk, D, D))
    kk, vv = torch.empty((total, Hk, D), dtype=BF, device="cuda"), torch.empty((total, Hk, D), dtype=BF, device="cuda")
    out, lse = torch.empty((total, Hq, D), dtype=BF, device="cuda"), torch.empty((total, Hq), device="cuda")
    seq = torch.zeros_like(pos)
    # the prompt
    dsa.cache4_write(lay, seq[:n1], pos[:n1], k[:n1], v[:n1], pool, ws, k_out=kk[:n1], v_out=vv[:n1])
    dsa.prompt_attn(q[:n1], kk[:n1], vv[:n1], D ** -0.5, out[:n1], lse[:n1], wp)
    # a chunk behind it: the cached prefix read back
    n = n1 + n2
    kr, vr = torch.empty((n, Hk, D), dtype=BF, device="cuda"), torch.empty((n, Hk, D), dtype=BF, device="cuda")
    dsa.cache4_write(lay, seq[n1:n], pos[n1:n], k[n1:n], v[n1:n], pool, ws, k_out=kk[n1:n], v_out=vv[n1:n])
    dsa.cache4_read(lay, seq[:n], pos[:n], pool, kr, vr, ws)
    assert torch.equal(kr, kk[:n]) and torch.equal(vr, vv[:n])
    wc = dsa.workspace(dsa.prompt_attn_workspace_size(1, n2, Hq, Hk, D, D))
    dsa.prompt_attn(q[n1:n], kr, vr, D ** -0.5, out[n1:n], lse[n1:n], wc)
    # decode: the chunk's last token again, then three new ones
    wa = dsa.workspace(dsa.cache4_attn_decode_workspace_size(1, Hq, Hk, D, D))
    o1, l1 = torch.empty((1, Hq, D), dtype=BF, device="cuda"), torch.empty((1, Hq), device="cuda")
    for t in range(n - 1, total):
        lens.fill_(t + 1)
        if t >= n:
            dsa.cache4_write(lay, None, None, k[t:t + 1], v[t:t + 1], pool, ws, k_out=kk[t:t + 1], v_out=vv[t:t + 1])
        dsa.cache4_attn_decode(lay, q[t:t + 1], pool, D ** -0.5, o1, l1, wa)
        o, l, m = attend_prompt64(q[t:t + 1], kk[:t + 1], vv[:t + 1], [0, 1], [0, t + 1], D ** -0.5)
        assert_rows_close(o1, l1, o, l, m, FP16, f"decode step {t}")
        if t == n - 1:
            assert_rows_close(out[t:n], lse[t:n], o, l, m, 2.0 ** -16, "the same token of the chunk")
    o, l, m = attend_prompt64(q[:n], kk[:n], vv[:n], [0, n1], [0, n1], D ** -0.5)
    assert_rows_close(out[:n1], lse[:n1], o[:n1], l[:n1], m[:n1], 2.0 ** -16, "prompt")
    for x in (ws, wp, wc, wa):
        assert dsa.get_status(x) == 0
