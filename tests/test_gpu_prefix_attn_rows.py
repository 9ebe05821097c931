"""GPU tests of dsa_prefix_attn_decode where single positions count: masks of
every tile, positions that decide a row, the accuracy of short sequences."""
import numpy as np
import pytest
import torch

from gpu_common import assert_out_close, lib, need_gpu
from heads_reference import assert_attn_close, attend64
from test_gpu_prefix_attn import LATENT, Problem

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _again(dsa, p):
    dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, p.prefix, p.scale, p.out, p.lse, p.ws)


@pytest.mark.parametrize("bs", [16, 32, 64])
def test_every_tile_has_a_mask_of_its_own(bs):
    """Bad block ids scattered over every tile, also with more tiles per pair
    than masks are kept: each tile's scores meet its own mask, in every run."""
    need_gpu()
    dsa = lib()
    g = np.random.default_rng(bs)
    for prefix, B, Hq in ((0, 8, 24), (5000, 40, 128)):    # 2 tiles a pair, 12
        p = Problem(bs, [prefix + (100 if prefix else 3000) + 37 * i for i in range(B)], bs=bs,
                    prefix=prefix, Hq=Hq, Dqk=64, Dv=64, latent=False)
        p.bt[g.random(p.bt.shape) < 0.3] = -1
        p.run(dsa).check(f"pages of {bs} behind {prefix}")
        assert dsa.get_status(p.ws) == dsa.STATUS_BAD_BLOCK
        first = p.out.clone()
        for _ in range(50):
            _again(dsa, p)
            assert torch.equal(p.out, first)


# ---------------------------------------------------- accuracy of short sequences --
# Sequences of at most 512 positions are close to a few single rows of V, and
# their weights are kept as bf16 hi + lo: off by (2^-8)^2, which with the fp32
# scores and sums (heads_reference: 2^-11 sum p |v| covers both) leaves the
# output's own rounding, 2^-8 of the value.  Longer ones have one bf16.
SHORT = 512
LENS = [2, 3] * 8 + [1, 4, 5, 7, 0, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 383, 384, 385,
                     511, 512, 513, 700, 2100]


def check_short(p, what):
    w, l, m = attend64(p.q, p.kp, p.vp, p.bt, p.lens, p.bs, p.nb, p.prefix, p.scale, p.Dv)
    assert_attn_close(p.out, p.lse, w, l, m, what)
    few = [b for b, n in enumerate(p.lens) if n <= SHORT]
    g = p.out.double().cpu()
    bad = ~((g - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -11 * m)[few]
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} elements of short sequences off"
    # the bar of every other attention call
    assert_out_close(p.out[few], p.lse[few], w[few].numpy(), l[few].numpy(), what)


def test_short_sequences_keep_the_framework_s_accuracy():
    need_gpu()
    dsa = lib()
    p = Problem(60, LENS, bs=64, prefix=0, **LATENT).run(dsa)
    check_short(p, "no prefix")
    assert dsa.get_status(p.ws) == 0


@pytest.mark.parametrize("prefix", [1, 2, 63, 100, 128, 129, 300, 500, 511, 512, 513])
def test_short_prefixes_keep_the_framework_s_accuracy(prefix):
    """Rows joined from a line over the prefix and one of their own; sequences
    shorter than the prefix; longer ones in the same call."""
    need_gpu()
    dsa = lib()
    lens = [n for n in LENS if n < prefix][:6]
    lens += [prefix + k for k in (0, 1, 2, 3, 5, 64, 127, 128, 129, 400, 513, 900)]
    p = Problem(61 + prefix, lens, bs=64, prefix=prefix, **LATENT).run(dsa)
    check_short(p, f"prefix {prefix}")


SHAPES = [dict(bs=48, prefix=50, Hq=24, Dqk=200, Dv=104, latent=False),
          dict(bs=24, prefix=0, Hq=3, Dqk=8, Dv=8, latent=False),
          dict(bs=1, prefix=33, Hq=16, Dqk=64, Dv=64, latent=False),
          dict(bs=7, prefix=130, Hq=128, Dqk=576, Dv=512, latent=True),
          dict(bs=8, prefix=3, Hq=72, Dqk=96, Dv=320, latent=False),
          dict(bs=16, prefix=0, Hq=64, Dqk=128, Dv=256, latent=False),
          dict(bs=32, prefix=290, Hq=1, Dqk=576, Dv=512, latent=True),
          dict(bs=1024, prefix=0, Hq=65, Dqk=64, Dv=512, latent=False)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['bs']}-{s['Hq']}-{s['Dqk']}-{s['Dv']}")
def test_short_sequences_of_other_shapes(shape):
    need_gpu()
    dsa = lib()
    p = Problem(shape["bs"], LENS, **shape).run(dsa)
    check_short(p, str(shape))
    first = p.out.clone()
    for _ in range(20):
        _again(dsa, p)
        assert torch.equal(p.out, first)


# --------------------------------------------------------- positions that decide --
class Planted(Problem):
    """A problem in which chosen positions decide one head each: K there is that
    head's query scaled to a score of 24, e^24 against at most 8191 others of
    N(0, 1) (their sum ~ e^9.5), so that the head's output is the position's
    row of V."""

    def __init__(self, seed, lens, **kw):
        super().__init__(seed, lens, **kw)
        self.plants = []

    def plant(self, b, h, pos, table=None):
        t = b if table is None else table
        page, r = int(self.bt[t, pos // self.bs]), pos % self.bs
        q = self.q[b, h].float()
        self.kp[page, r, :self.Dqk] = (q * (24.0 / (self.scale * float(q @ q)))).to(BF)
        self.plants.append((b, h, page, r))

    def check_plants(self, what):
        """The weight of the row is 1 to 1e-4 (fp32), rounded to bf16 at most
        once, and so is the output: 2^-7 of the value, and 1e-3 for the others
        (1e-4 times values of up to 6).  A position counted twice would move
        the lse, which check() holds, by log 2."""
        self.check(what)
        for b, h, page, r in self.plants:
            v = self.vp[page, r, :self.Dv].double()
            err = (self.out[b, h].double() - v).abs()
            assert bool((err <= 2.0 ** -7 * v.abs() + 1e-3).all()), (what, b, h, page, r)


def edges(p0, p1, step):
    """First and last positions of the tiles and of the chunks of 64 of a line
    over [p0, p1), the line's ends first."""
    at = [p1 - 1, p0]
    for a in range(p0 - p0 % step, p1, step):
        at += [a, a + step - 1]
    for a in range(p0 - p0 % 64, p1, 64):
        at += [a, a + 63]
    return list(dict.fromkeys(p for p in at if p0 <= p < p1))


PLANTED = [dict(Hq=64, Dqk=576, Dv=512, latent=True), dict(Hq=128, Dqk=128, Dv=64, latent=False)]


@pytest.mark.parametrize("shape", PLANTED, ids=["latent", "gqa"])
@pytest.mark.parametrize("bs", [16, 64])
def test_every_edge_of_a_long_line_counts_once(bs, shape):
    need_gpu()
    dsa = lib()
    lens = [5000, 8191, 8191, 8191, 4096, 300, 512, 513, 1]
    p = Planted(bs, lens, bs=bs, prefix=0, **shape)
    done = {}
    for b, n in enumerate(lens):
        at = edges(0, n, 128 if n <= SHORT else 256)
        first = done.get(n, 0)                           # equal lengths share the edges out
        for h, pos in enumerate(at[first:first + p.Hq]):
            p.plant(b, h, pos)
        done[n] = first + p.Hq
    p.run(dsa).check_plants(f"pages of {bs}")
    assert dsa.get_status(p.ws) == 0


@pytest.mark.parametrize("shape", PLANTED, ids=["latent", "gqa"])
@pytest.mark.parametrize("bs,prefix", [(64, 4100), (16, 4096), (48, 5001), (64, 300)])
def test_every_edge_of_a_prefix_and_behind_it_counts_once(bs, prefix, shape):
    need_gpu()
    dsa = lib()
    lens = [prefix + k for k in (0, 1, 300, 2100)] + [prefix + 511, prefix + 512, prefix - 1, prefix + 64]
    p = Planted(prefix + bs, lens, bs=bs, prefix=prefix, **shape)
    shared = edges(0, prefix, 128 if prefix <= SHORT else 256)
    box = next(r for r in (64, 32, 16, 8) if bs % r == 0)
    start = prefix - prefix % box                        # where the sequences' own tiles begin
    nth = 0
    for b, n in enumerate(lens):
        h = 0
        if n >= prefix:                                  # half of its heads to its own positions
            step = 128 if n <= SHORT else 256
            own = [n - 1, prefix] + [a + d for a in range(start, n, step) for d in (0, step - 1)]
            for pos in list(dict.fromkeys(x for x in own if prefix <= x < n))[:p.Hq // 2]:
                p.plant(b, h, pos)
                h += 1
            for pos in shared[nth:nth + p.Hq - h]:       # the others to the prefix's edges
                p.plant(b, h, pos, table=0)              # sequence 0 has all of it
                h += 1
                nth += 1
        else:
            for h, pos in enumerate(edges(0, n, 256)[:p.Hq]):
                p.plant(b, h, pos)
    p.run(dsa).check_plants(f"prefix {prefix}")
    assert dsa.get_status(p.ws) == 0


@pytest.mark.parametrize("Hq", [65, 72, 127])
def test_lines_with_few_rows_in_the_second_cta_stay_in_step(Hq):
    """Heads beyond 64 lie in the pair's second CTA: one row, a handful, all but
    one.  Many runs of one problem, all equal bit for bit."""
    need_gpu()
    dsa = lib()
    g = np.random.default_rng(Hq)
    p = Problem(Hq, [int(n) for n in g.integers(1, 2049, 40)], bs=64, prefix=0, Hq=Hq, Dqk=576, Dv=512,
                latent=True).run(dsa)
    p.check("first run")
    first = p.out.clone()
    for _ in range(100):
        _again(dsa, p)
        assert torch.equal(p.out, first)


def test_both_attention_calls_meet_the_same_bar_on_short_sequences():
    """Every position selected: the sparse call and this one, each within the
    common bar of the exact values."""
    need_gpu()
    dsa = lib()
    lens = [2, 3, 1, 17, 200, 511, 512, 700] + [2, 3] * 8
    p = Problem(80, lens, bs=64, prefix=0, **LATENT).run(dsa)
    check_short(p, "prefix attention")
    B, K = len(lens), 768
    idx = torch.full((B, K), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        idx[b, :n] = torch.arange(n, dtype=torch.int32)
    out, lse = torch.empty_like(p.out), torch.empty_like(p.lse)
    ws = dsa.workspace(dsa.sparse_attn_decode_workspace_size(B, 64, 576, 512, K))
    dsa.sparse_attn_decode(p.lay, p.q, p.kp, p.vp, idx.cuda(), p.scale, out, lse, ws)
    w, l, _ = attend64(p.q, p.kp, p.vp, p.bt, p.lens, p.bs, p.nb, 0, p.scale, p.Dv)
    assert_out_close(out, lse, w.numpy(), l.numpy(), "sparse attention, all selected")
    assert_out_close(p.out, p.lse, w.numpy(), l.numpy(), "prefix attention")
    assert dsa.get_status(ws) == 0 and dsa.get_status(p.ws) == 0
