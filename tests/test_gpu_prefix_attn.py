"""GPU tests of dsa_prefix_attn_decode against exact attention in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_common import lib, need_gpu
from heads_reference import assert_attn_close, attend64, transform64, assert_heads_close

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Problem:
    """A paged cache whose rows outside every sequence are NaN; whole prefix
    pages shared, the page the prefix ends in copied per sequence."""

    def __init__(self, seed, lens, Hq, Dqk, Dv, latent, bs, prefix, pad=0, scale=None, q_amp=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.bs, self.prefix = list(lens), bs, prefix
        self.Hq, self.Dqk, self.Dv = Hq, Dqk, Dv
        B = len(lens)
        shared = prefix // bs
        maxb = max([1, shared] + [(n + bs - 1) // bs for n in lens])
        need = [max(0, (n + bs - 1) // bs - (shared if n >= prefix else 0)) for n in lens]
        nb = shared + sum(need) + 2
        perm = torch.randperm(nb, generator=g).numpy().astype(np.int32)
        bt = np.full((B, maxb), -7, np.int32)              # unused entries hold rubbish
        at = shared
        for b, n in enumerate(lens):
            s0 = 0
            if n >= prefix:
                bt[b, :shared] = perm[:shared]
                s0 = shared
            bt[b, s0:s0 + need[b]] = perm[at:at + need[b]]
            at += need[b]
        self.bt, self.nb = bt, nb
        def pool(width):
            full = torch.full((nb, bs, width + pad), float("nan"), dtype=BF)
            for b, n in enumerate(lens):
                for s in range((n + bs - 1) // bs):
                    rows = min(bs, n - s * bs)
                    page = full[int(bt[b, s])]
                    if bool(torch.isnan(page[:rows, :width]).any()):
                        page[:rows, :width] = torch.randn((rows, width), generator=g).to(BF)
            src = next((b for b in range(B) if lens[b] >= prefix), None)
            if prefix % bs and src is not None:
                for b in range(B):
                    if lens[b] >= prefix and b != src:
                        full[int(bt[b, shared]), :prefix % bs] = full[int(bt[src, shared]), :prefix % bs]
            return full.cuda()
        self.kp = pool(Dqk)
        self.vp = self.kp if latent else pool(Dv)
        self.q = (q_amp * torch.randn((B, Hq, Dqk), generator=g)).to(BF).cuda()
        self.scale = scale or Dqk ** -0.5

    def run(self, dsa, ws=None, lse=True):
        B = len(self.lens)
        self.dev_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.lay = dsa.PagedLayout(torch.from_numpy(self.bt).cuda(), self.dev_lens, self.bs, self.nb,
                                   max(max(self.lens), self.prefix))
        self.out = torch.full((B, self.Hq, self.Dv), 5.0, dtype=BF, device="cuda")
        self.lse = torch.full((B, self.Hq), 5.0, device="cuda") if lse else None
        n = dsa.prefix_attn_decode_workspace_size(B, self.Hq, self.Dqk, self.Dv, self.prefix)
        self.ws = dsa.workspace(n) if ws is None else ws
        dsa.prefix_attn_decode(self.lay, self.q, self.kp, self.vp, self.prefix, self.scale, self.out,
                               self.lse, self.ws)
        torch.cuda.synchronize()
        return self

    def check(self, what="", lens=None):
        w, l, m = attend64(self.q, self.kp, self.vp, self.bt, lens or self.lens, self.bs, self.nb,
                           self.prefix, self.scale, self.Dv)
        assert_attn_close(self.out, self.lse, w, l, m, what)


LATENT = dict(Hq=64, Dqk=576, Dv=512, latent=True)
CASES = {
    # one short sequence; one token; none
    "one-token": dict(lens=[1], bs=64, prefix=0, **LATENT),
    "empty": dict(lens=[0, 0], bs=64, prefix=0, **LATENT),
    "tile-edges": dict(lens=[127, 128, 129, 255, 256, 257, 511, 513, 0, 64], bs=64, prefix=0, **LATENT),
    "long-ragged": dict(lens=[5000, 3, 1, 8191, 2049], bs=64, prefix=0, **LATENT),
    "prefix": dict(lens=[1500, 1025, 1024, 2048, 1031], bs=64, prefix=1024, **LATENT),
    "prefix-only": dict(lens=[4096] * 3, bs=64, prefix=4096, **LATENT),
    "prefix-in-page": dict(lens=[1000, 1001, 1700], bs=64, prefix=1000, **LATENT),
    # some sequences shorter than the prefix, the first among them
    "short-first": dict(lens=[10, 700, 0, 650, 639, 1], bs=64, prefix=640, **LATENT),
    "none-has-it": dict(lens=[10, 70, 0], bs=64, prefix=640, **LATENT),
    "one-head": dict(lens=[300, 301], bs=16, prefix=290, Hq=1, Dqk=576, Dv=512, latent=True),
    "heads-128": dict(lens=[700, 90], bs=64, prefix=64, Hq=128, Dqk=576, Dv=512, latent=True),
    "gqa": dict(lens=[2300, 2049, 2200, 2100], bs=64, prefix=2048, Hq=16, Dqk=128, Dv=128, latent=False),
    "odd-dims": dict(lens=[900, 513, 777, 1], bs=48, prefix=513, Hq=24, Dqk=200, Dv=104, latent=False),
    "small-dims": dict(lens=[130, 99], bs=24, prefix=50, Hq=3, Dqk=8, Dv=8, latent=False),
    "wide-v": dict(lens=[600, 17], bs=128, prefix=0, Hq=5, Dqk=64, Dv=512, latent=False),
    "v-320": dict(lens=[600, 17], bs=32, prefix=16, Hq=40, Dqk=320, Dv=320, latent=True),
    "page-1": dict(lens=[260, 70], bs=1, prefix=33, Hq=16, Dqk=64, Dv=64, latent=False),
    "page-7": dict(lens=[260, 70, 300], bs=7, prefix=66, Hq=16, Dqk=576, Dv=512, latent=True),
    "page-1024": dict(lens=[3000, 1500], bs=1024, prefix=1100, **LATENT),
    "padded-rows": dict(lens=[400, 300], bs=64, prefix=256, pad=64, Hq=20, Dqk=128, Dv=96, latent=False),
    "many": dict(lens=[(37 * i) % 300 for i in range(150)], bs=32, prefix=0, Hq=8, Dqk=64, Dv=64,
                 latent=False),
    "many-prefix": dict(lens=[500 + (37 * i) % 90 for i in range(70)], bs=32, prefix=500, Hq=64,
                        Dqk=96, Dv=64, latent=False),
}


@pytest.mark.parametrize("name", CASES)
def test_prefix_attn_matches_64_bits(name):
    need_gpu()
    dsa = lib()
    p = Problem(sum(map(ord, name)), **CASES[name]).run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check(name)


@pytest.mark.parametrize("bs", [16, 48, 64, 128, 1024])
@pytest.mark.parametrize("prefix", [1, 31, 33, 63, 100, 319, 1023])
def test_prefixes_that_end_anywhere(bs, prefix):
    """The sequences' own tiles begin inside a group of positions: what their
    own pages hold ahead of them (NaN) is neither K nor V of theirs."""
    need_gpu()
    dsa = lib()
    lens = [prefix - 1, prefix + 300, prefix, prefix + 1, prefix + 63, prefix + 64, prefix + 257]
    for kw in (LATENT, dict(Hq=5, Dqk=72, Dv=200, latent=False)):
        p = Problem(bs + prefix, lens, bs=bs, prefix=prefix, **kw)
        if prefix % bs:
            for b in range(2, len(lens)):          # sequence 1 is the prefix's source
                page = int(p.bt[b, prefix // bs])
                if lens[b] > prefix:
                    p.kp[page, :prefix % bs] = float("nan")
                    p.vp[page, :prefix % bs] = float("nan")
        p.run(dsa)
        assert dsa.get_status(p.ws) == 0
        p.check(f"prefix {prefix} pages of {bs}")


def test_many_short_lines_per_pair_stay_in_step():
    """Sequences of a few tiles with 64 heads: one CTA of a pair has no rows of
    any line, and must not run ahead of the other.  Many runs of one problem,
    all equal bit for bit."""
    need_gpu()
    dsa = lib()
    g = np.random.default_rng(5)
    p = Problem(50, [int(n) for n in g.integers(1, 2049, 48)], bs=64, prefix=0, **LATENT).run(dsa)
    p.check("first run")
    first = p.out.clone()
    for _ in range(200):
        dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, 0, p.scale, p.out, p.lse, p.ws)
        assert torch.equal(p.out, first)


def test_slow_copies_of_v_do_not_reorder_a_pair():
    """Pages that leave boxes of 4 rows and 1 row (V arrives slowly) with
    several tiles of a line on one pair, so that the softmax runs far ahead of
    the second product."""
    need_gpu()
    dsa = lib()
    for prefix, bs, dv in ((500, 4, 64), (500, 12, 128), (1021, 1, 512), (516, 20, 320), (500, 32, 64),
                           (1021, 16, 512)):
        p = Problem(prefix, [prefix + (37 * i) % 90 for i in range(70)], bs=bs, prefix=prefix, Hq=64,
                    Dqk=96, Dv=dv, latent=False).run(dsa)
        p.check(f"prefix {prefix} dv {dv}")
        first = p.out.clone()
        for _ in range(20):
            dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, prefix, p.scale, p.out, p.lse, p.ws)
            assert torch.equal(p.out, first)


def test_large_scores_and_peaked_rows():
    """Scores of +-hundreds: the running maximum moves by far more than fp32's
    exponent range between tiles."""
    need_gpu()
    dsa = lib()
    p = Problem(3, [900, 1400], bs=64, prefix=512, q_amp=30.0, **LATENT).run(dsa)
    g = p.out.float()
    assert bool(torch.isfinite(g).all())
    # scores up to ~150: the fp32 products' error 2^-21 * sum |q k| reaches
    # 2^-21 * 30 * 24 * 0.64 = 2e-4 in z, inside the 2^-11 of the bound
    p.check("large scores")
    # every key of the second half beats the first half by hundreds
    p = Problem(4, [1200], bs=64, prefix=0, **LATENT)
    rows = torch.from_numpy(p.bt[0, np.arange(600, 1200) // 64].astype(np.int64) * 64
                            + np.arange(600, 1200) % 64)
    flat = p.kp.view(-1, 576)
    flat[rows.cuda()] = (flat[rows.cuda()].float() * 0.25 + p.q[0, 0].float() * 4).to(BF)
    p.run(dsa).check("second half")


def test_bad_block_ids_are_left_out_and_flagged():
    need_gpu()
    dsa = lib()
    for prefix in (0, 256):
        p = Problem(11, [700, 520], bs=64, prefix=prefix, **LATENT)
        p.bt[0, 9] = p.nb + 3
        p.bt[1, 6] = -1
        p.run(dsa).check(f"prefix {prefix}")
        assert dsa.get_status(p.ws) == dsa.STATUS_BAD_BLOCK
    p = Problem(12, [700, 520], bs=64, prefix=256, **LATENT)
    p.bt[:, 2] = 1 << 30
    p.run(dsa).check("inside the prefix")
    assert dsa.get_status(p.ws) == dsa.STATUS_BAD_BLOCK
    # every page bad: nothing is attended
    p = Problem(13, [100], bs=64, prefix=0, **LATENT)
    p.bt[:] = -1
    p.run(dsa)
    assert bool((p.out == 0).all()) and bool((p.lse == float("-inf")).all())


def test_lengths_beyond_the_table_are_cut_and_flagged():
    need_gpu()
    dsa = lib()
    p = Problem(14, [128, 100], bs=64, prefix=0, **LATENT)
    p.run(dsa)
    p.dev_lens.copy_(torch.tensor([100000, 100], dtype=torch.int32))
    dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, 0, p.scale, p.out, p.lse, p.ws)
    p.check("cut", lens=[128, 100])
    assert dsa.get_status(p.ws) == dsa.STATUS_BAD_LENGTH
    p.dev_lens.copy_(torch.tensor([-5, 100], dtype=torch.int32))
    dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, 0, p.scale, p.out, p.lse, p.ws)
    p.check("negative", lens=[0, 100])


def test_other_rows_do_not_see_a_nan():
    """A NaN in one sequence's query, and one in another's own cached rows,
    stay in their sequences' outputs."""
    need_gpu()
    dsa = lib()
    p = Problem(17, [700, 900, 650, 800], bs=64, prefix=640, **LATENT).run(dsa)
    want, lse = p.out.clone(), p.lse.clone()
    p.q[1, 5, 100] = float("nan")
    page = int(p.bt[2, 645 // 64])
    p.kp[page, 645 % 64, 3] = float("inf")
    p.run(dsa, ws=p.ws)
    assert torch.equal(p.out[0], want[0]) and torch.equal(p.out[3], want[3])
    assert torch.equal(p.lse[0], lse[0]) and torch.equal(p.lse[3], lse[3])
    keep = [h for h in range(64) if h != 5]
    assert torch.equal(p.out[1, keep], want[1, keep])
    assert bool(torch.isnan(p.out[1, 5].float()).all())
    assert not bool(torch.isfinite(p.out[2].float()).all())


def test_results_repeat_bit_for_bit_and_workspaces_are_reusable():
    need_gpu()
    dsa = lib()
    p = Problem(15, [3000, 2100, 2050, 2600], bs=64, prefix=2048, **LATENT).run(dsa)
    first, lse = p.out.clone(), p.lse.clone()
    small = Problem(16, [77, 5, 0, 9], bs=64, prefix=0, **LATENT).run(dsa, ws=p.ws)
    small.check("another problem on the same workspace")
    p.run(dsa, ws=p.ws)
    assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    p.run(dsa, ws=p.ws, lse=False)
    assert torch.equal(p.out, first)


def test_two_streams_with_their_own_workspaces():
    need_gpu()
    dsa = lib()
    ps = [Problem(20 + i, [1500 + i, 1300, 1029], bs=64, prefix=1024, **LATENT).run(dsa) for i in range(2)]
    want = [p.out.clone() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    for p in ps:
        p.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for p, st in zip(ps, streams):
            dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, p.prefix, p.scale, p.out, p.lse, p.ws,
                                   stream=st)
    torch.cuda.synchronize()
    for p, w in zip(ps, want):
        assert torch.equal(p.out, w)


def test_captured_call_follows_the_lengths():
    need_gpu()
    dsa = lib()
    p = Problem(30, [1200, 1100, 1064], bs=64, prefix=1000, **LATENT).run(dsa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.prefix_attn_decode(p.lay, p.q, p.kp, p.vp, p.prefix, p.scale, p.out, p.lse, p.ws)
    for lens in ([1200, 1100, 1064], [1001, 1000, 1064], [5, 1099, 0], [0, 0, 0]):
        p.dev_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check(f"lens {lens}", lens=lens)


def test_one_decode_step_from_projections_to_output():
    """Raw projections -> cache_append (cache rows, indexer keys, queries) ->
    attention, and through the sparse path (every position selected) -> the
    same result; all against 64 bits on the stored cache."""
    need_gpu()
    dsa = lib()
    prefix, K = 640, 2048
    p = Problem(40, [700, 641, 1999], bs=64, prefix=prefix, **LATENT)
    B, Hq = 3, 64
    g = torch.Generator().manual_seed(41)
    kv = torch.randn((B, 1, 576), generator=g).to(BF).cuda()
    ki = torch.randn((B, 1, 128), generator=g).to(BF).cuda()
    qp = torch.randn((B, Hq, 192), generator=g).to(BF).cuda()
    qi = torch.randn((B, 64, 128), generator=g).to(BF).cuda()
    w = torch.rand((B, 64), generator=g).cuda()
    kidx = torch.randint(0, 127, (p.nb, 64, 128), generator=g, dtype=torch.uint8).cuda()
    f = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    ones = (1 + 0.1 * torch.randn(512, generator=g)).cuda()
    p.lay = lay = dsa.PagedLayout(torch.from_numpy(p.bt).cuda(),
                                  torch.tensor(p.lens, dtype=torch.int32).cuda(), 64, p.nb, 1999)
    qio = torch.empty((B, 64, 128), dtype=torch.uint8, device="cuda")
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    dsa.cache_append(lay, None, None,
                     [dsa.HeadPart(kv, p.kp, norm="rms", norm_dim=512, weight=ones, rope_offset=512,
                                   rope_dim=64, interleaved=True, inv_freq=f),
                      dsa.HeadPart(ki, kidx, norm="layer", rope_dim=64, inv_freq=f)], ws,
                     heads=[dsa.HeadPart(qp[:, :, 128:], p.q[:, :, 512:], rope_dim=64, interleaved=True,
                                         inv_freq=f),
                            dsa.HeadPart(qi, qio, norm="rms", rope_dim=64, inv_freq=f)])
    out = torch.empty((B, Hq, 512), dtype=BF, device="cuda")
    lse = torch.empty((B, Hq), device="cuda")
    wp = dsa.workspace(dsa.prefix_attn_decode_workspace_size(B, Hq, 576, 512, prefix))
    dsa.prefix_attn_decode(lay, p.q, p.kp, p.kp, prefix, p.scale, out, lse, wp)
    pipe = dsa.Pipeline(lay, kind="decode", Nq=B, Hq=Hq, Dqk=576, Dv=512, H_i=64, D_i=128, K=K)
    pipe.run(p.q, qio, w, kidx, p.kp, p.kp, p.scale)
    torch.cuda.synchronize()
    assert dsa.get_status(ws) == 0 and dsa.get_status(wp) == 0 and pipe.status() == 0
    pos = torch.tensor(p.lens) - 1
    want, e = transform64(qp[:, :, 128:], pos, rope_dim=64, interleaved=True, inv_freq=f)
    assert_heads_close(p.q[:, :, 512:], want, e, "queries")
    o, l, m = attend64(p.q, p.kp, p.kp, p.bt, p.lens, 64, p.nb, prefix, p.scale, 512)
    assert_attn_close(out, lse, o, l, m, "prefix attention")
    assert_attn_close(pipe.out, pipe.lse, o, l, m, "sparse attention, all selected")
