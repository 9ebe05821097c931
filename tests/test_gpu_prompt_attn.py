"""GPU tests of dsa_prompt_attn against exact attention in 64 bits."""
import itertools

import pytest
import torch

from gpu_common import lib, need_gpu
from prompt_reference import assert_rows_close, attend_prompt64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ONE, TWO = 2.0 ** -8, 2.0 ** -16        # weights as bf16, as bf16 hi + lo


def cu(lens):
    return [0, *itertools.accumulate(lens)]


class Problem:
    """Packed sequences of (query tokens, keys)."""

    def __init__(self, seed, seqs, Hq, Hk, Dk, Dv=None, layout="packed", scale=None, q_amp=1.0):
        g = torch.Generator().manual_seed(seed)
        Dv = Dk if Dv is None else Dv
        self.nq, self.nk = [a for a, _ in seqs], [b for _, b in seqs]
        Nq, Nk = sum(self.nq), sum(self.nk)
        r = lambda *s: torch.randn(s, generator=g).to(BF).cuda()  # noqa: E731
        if layout == "fused":                              # slices of one projection
            assert Nq == Nk and Dk == Dv
            x = r(Nq, Hq + 2 * Hk, Dk)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        elif layout == "heads":                            # [heads, tokens, dim] seen as tokens first
            q, k, v = (r(h, n, d).transpose(0, 1) for h, n, d in ((Hq, Nq, Dk), (Hk, Nk, Dk), (Hk, Nk, Dv)))
        elif layout == "wide":                             # head slots wider than the heads
            q, k, v = (r(n, h, d + 24)[:, :, 8:8 + d] for h, n, d in ((Hq, Nq, Dk), (Hk, Nk, Dk), (Hk, Nk, Dv)))
        else:
            q, k, v = r(Nq, Hq, Dk), r(Nk, Hk, Dk), r(Nk, Hk, Dv)
        if q_amp != 1.0:
            q = (q.float() * q_amp).to(BF)
        self.q, self.k, self.v, self.scale = q, k, v, scale or Dk ** -0.5
        self.Hq, self.Hk, self.Dk, self.Dv = Hq, Hk, Dk, Dv
        if layout == "wide":
            self.out = torch.full((Nq, Hq, Dv + 24), 5.0, dtype=BF, device="cuda")[:, :, 16:16 + Dv]
        elif layout == "heads":
            self.out = torch.full((Hq, Nq, Dv), 5.0, dtype=BF, device="cuda").transpose(0, 1)
        else:
            self.out = torch.full((Nq, Hq, Dv), 5.0, dtype=BF, device="cuda")
        self.lse = torch.full((Nq, Hq), 5.0, device="cuda")
        self.cu_q = torch.tensor(cu(self.nq), dtype=torch.int32, device="cuda")
        self.cu_k = torch.tensor(cu(self.nk), dtype=torch.int32, device="cuda")

    def workspace(self, dsa):
        return dsa.workspace(dsa.prompt_attn_workspace_size(len(self.nq), self.q.shape[0], self.Hq, self.Hk,
                                                            self.Dk, self.Dv))

    def run(self, dsa, ws=None, lse=True, **kw):
        self.ws = self.workspace(dsa) if ws is None else ws
        dsa.prompt_attn(self.q, self.k, self.v, self.scale, self.out, self.lse if lse else None, self.ws,
                        cu_q=self.cu_q, cu_k=self.cu_k, **kw)
        torch.cuda.synchronize()
        return self

    def check(self, what="", weight=ONE, lse=True):
        o, l, m = attend_prompt64(self.q, self.k, self.v, self.cu_q.tolist(), self.cu_k.tolist(), self.scale)
        assert_rows_close(self.out, self.lse if lse else None, o, l, m, weight, what)


def same(*n):
    return [(x, x) for x in n]


CASES = {
    "one-token": dict(seqs=same(1), Hq=1, Hk=1, Dk=64),
    "tile-edges": dict(seqs=same(127, 128, 129, 1, 0, 255, 256, 257, 64), Hq=2, Hk=2, Dk=64),
    "grouped-edges": dict(seqs=same(7, 8, 9, 31, 32, 33, 65, 0, 1), Hq=32, Hk=2, Dk=128),
    "fused": dict(seqs=same(300, 77), Hq=12, Hk=2, Dk=80, layout="fused"),
    "heads-first": dict(seqs=same(200, 130), Hq=6, Hk=3, Dk=96, layout="heads"),
    "wide-slots": dict(seqs=same(190, 3), Hq=10, Hk=5, Dk=40, layout="wide"),
    "many-heads-one-key": dict(seqs=same(65, 2), Hq=128, Hk=1, Dk=32),
    "group-of-three": dict(seqs=same(140, 520), Hq=9, Hk=3, Dk=72),
    "latent": dict(seqs=same(260, 100), Hq=8, Hk=8, Dk=192, Dv=128),
    "small-dims": dict(seqs=same(70, 600), Hq=3, Hk=1, Dk=8, Dv=8),
    "narrow-v": dict(seqs=same(300), Hq=4, Hk=2, Dk=256, Dv=16),
    "wide-v": dict(seqs=same(300, 5), Hq=4, Hk=2, Dk=64, Dv=256),
    "widest": dict(seqs=same(700, 130), Hq=4, Hk=1, Dk=256),
    "odd-wide": dict(seqs=same(131, 400), Hq=2, Hk=2, Dk=200, Dv=136),
    "chunks": dict(seqs=[(100, 300), (1, 513), (128, 128), (64, 1000), (0, 40)], Hq=8, Hk=2, Dk=128),
    "fewer-keys": dict(seqs=[(100, 40), (300, 1), (5, 0), (257, 129)], Hq=4, Hk=4, Dk=64),
    "long": dict(seqs=same(1500, 700), Hq=4, Hk=2, Dk=128),
    "many": dict(seqs=[((37 * i) % 90, (37 * i) % 90 + (i % 3) * 50) for i in range(70)], Hq=4, Hk=2, Dk=64),
    # few rows over many keys: cut in pieces (one for each head block and column half)
    "cut-row": dict(seqs=[(1, 5000)], Hq=4, Hk=1, Dk=64),
    "cut-chunk": dict(seqs=[(40, 3500), (3, 2600), (200, 1700), (1, 100)], Hq=4, Hk=2, Dk=64),
    "cut-wide-v": dict(seqs=[(9, 2600), (16, 40)], Hq=6, Hk=2, Dk=136, Dv=200),
    "cut-prompt": dict(seqs=[(2300, 2300)], Hq=2, Hk=1, Dk=64),
    "cut-rows-of-many": dict(seqs=[(1, 4000)] * 40 + [(0, 0), (3, 2)], Hq=4, Hk=2, Dk=64),
    "cut-some-of-200": dict(seqs=[((7 * i) % 30, (7 * i) % 30 + (2900 if i % 60 == 0 else i % 90)) for i in range(200)],
                            Hq=4, Hk=2, Dk=64),
    "more-rows-than-pieces": dict(seqs=[(1, 2500)] * 70, Hq=8, Hk=8, Dk=32),
    # more items than CTAs, the last of them in pieces
    "cut-last-wave": dict(seqs=[(600, 2000)], Hq=64, Hk=64, Dk=64),
    "cut-last-wave-of-two": dict(seqs=[(5, 40), (900, 3100), (0, 3)], Hq=40, Hk=8, Dk=64),
    "cut-last-wave-wide-v": dict(seqs=[(300, 1900)], Hq=40, Hk=40, Dk=40, Dv=136),
}


@pytest.mark.parametrize("name", CASES)
def test_prompt_attn_matches_64_bits(name):
    need_gpu()
    dsa = lib()
    p = Problem(sum(map(ord, name)), **CASES[name]).run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check(name)
    first, lse = p.out.clone(), p.lse.clone()
    p.out.fill_(3.0)
    p.run(dsa, ws=p.ws)                        # the workspace's counters are back at zero
    assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    p.run(dsa, ws=p.ws, lse=False)
    assert torch.equal(p.out, first)


@pytest.mark.parametrize("Dk,Dv", [(8 * i, 8 * ((11 * i) % 32 + 1)) for i in range(1, 33, 3)])
def test_every_width(Dk, Dv):
    need_gpu()
    dsa = lib()
    p = Problem(Dk, [(140, 150), (3, 300)], Hq=4, Hk=2, Dk=Dk, Dv=Dv).run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check(f"{Dk} / {Dv}")


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (24, 4), (7, 7), (64, 1), (40, 8), (256, 2)])
@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_head_groups(Hq, Hk, n):
    need_gpu()
    dsa = lib()
    p = Problem(Hq + n, [(n, n + 9), (n, n)], Hq=Hq, Hk=Hk, Dk=64).run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check(f"{Hq} over {Hk}, {n} tokens")


def test_rows_that_see_few_keys_have_exact_weights():
    """Up to 512 keys a weight is bf16 hi + lo: the bound without the single rounding's 2^-8."""
    need_gpu()
    dsa = lib()
    for Hq, Hk in ((4, 4), (16, 1)):
        p = Problem(5, same(2, 3, 100, 384, 1, 256), Hq=Hq, Hk=Hk, Dk=128).run(dsa)
        p.check("short", weight=TWO)


def test_large_scores_and_a_maximum_that_keeps_rising():
    """Scores of +-hundreds, and keys that each beat all before them by more than 2^8."""
    need_gpu()
    dsa = lib()
    Problem(3, same(600, 90), Hq=2, Hk=1, Dk=128, q_amp=30.0).run(dsa).check("large scores")
    p = Problem(4, same(900), Hq=2, Hk=1, Dk=64)
    up = torch.arange(900, device="cuda").float()[:, None] * 0.05
    p.k[:, 0] = (p.q[:, 0].float().mean(0) * 0 + up).to(BF).expand(900, 64)
    p.q[:] = 1.0
    p.run(dsa).check("rising")
    assert dsa.get_status(p.ws) == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_a_token_does_not_see_does_not_reach_it(value):
    """A value in one sequence's V or K, at a token in the middle of a tile: earlier tokens and the
    other sequences do not change by a bit, later ones have it."""
    need_gpu()
    dsa = lib()
    for Hq, Hk, Dk, Dv in ((4, 2, 64, 64), (16, 1, 128, 128), (2, 2, 64, 200)):
        for at in (0, 5, 130, 299):
            p = Problem(9, same(70, 300, 60), Hq=Hq, Hk=Hk, Dk=Dk, Dv=Dv).run(dsa)
            before, lse = p.out.clone(), p.lse.clone()
            p.v[70 + at, Hk - 1, 3] = value
            p.v[70 + at, Hk - 1, Dv - 1] = value
            p.run(dsa, ws=p.ws)
            p.check(f"V at {at}")
            assert torch.equal(p.out[:70 + at], before[:70 + at]) and torch.equal(p.out[370:], before[370:])
            assert torch.equal(p.lse, lse)
            p.k[70 + at, 0, 1] = float("nan")
            p.run(dsa, ws=p.ws)
            assert torch.equal(p.out[:70 + at], before[:70 + at]) and torch.equal(p.out[370:], before[370:])
            assert bool(torch.isnan(p.out[70 + at:370, 0].float()).all())


def test_other_rows_do_not_see_a_query_s_nan():
    need_gpu()
    dsa = lib()
    p = Problem(10, same(40, 200), Hq=8, Hk=2, Dk=64).run(dsa)
    before = p.out.clone()
    p.q[100, 3, 7] = float("nan")
    p.run(dsa, ws=p.ws)
    keep = torch.ones(p.out.shape[:2], dtype=torch.bool, device="cuda")
    keep[100, 3] = False
    assert torch.equal(p.out[keep], before[keep])
    assert bool(torch.isnan(p.out[100, 3].float()).all())


def test_cut_items_with_odd_values():
    """Pieces of a cut item: rows that see nothing of the last piece, and infinities in it."""
    need_gpu()
    dsa = lib()
    p = Problem(11, [(60, 2000)], Hq=2, Hk=1, Dk=64).run(dsa)
    before = p.out.clone()
    p.v[1990, 0, 5] = float("inf")
    p.run(dsa, ws=p.ws)
    p.check("inf in the last piece")
    assert torch.equal(p.out[:50], before[:50])


def test_tokens_of_no_sequence_are_left_as_they_are():
    need_gpu()
    dsa = lib()
    p = Problem(12, same(50, 60, 40), Hq=4, Hk=4, Dk=64)
    p.cu_q = torch.tensor([10, 50, 50, 130], dtype=torch.int32, device="cuda")
    p.cu_k = torch.tensor([0, 45, 60, 140], dtype=torch.int32, device="cuda")
    p.run(dsa)
    assert bool((p.out[:10] == 5).all()) and bool((p.out[130:] == 5).all())
    assert bool((p.lse[:10] == 5).all()) and bool((p.lse[130:] == 5).all())
    want, l, m = attend_prompt64(p.q, p.k, p.v, [10, 50, 50, 130], [0, 45, 60, 140], p.scale)
    assert_rows_close(p.out[10:130], p.lse[10:130], want[10:130], l[10:130], m[10:130], ONE, "inside")


def test_bad_offsets_are_left_out_and_flagged():
    need_gpu()
    dsa = lib()
    p = Problem(13, same(50, 60, 40), Hq=4, Hk=4, Dk=64).run(dsa)
    first = p.out.clone()
    for bad in ([0, 50, 20, 150], [0, 50, 110, 151], [-1, 50, 110, 150], [0, 50, 1 << 30, 150]):
        p.out.fill_(5.0)
        p.cu_q = torch.tensor(bad, dtype=torch.int32, device="cuda")
        p.run(dsa, ws=p.ws)
        assert dsa.get_status(p.ws) == dsa.STATUS_BAD_LENGTH
        if bad[:2] == [0, 50]:                 # (a later sequence that begins inside the first writes over it)
            n = min(50, *(x for x in bad[1:]))
            assert torch.equal(p.out[:n], first[:n])
    p.cu_q = torch.tensor(cu([50, 60, 40]), dtype=torch.int32, device="cuda")
    p.cu_k = torch.tensor([0, 50, 110, 300], dtype=torch.int32, device="cuda")
    p.out.fill_(5.0)
    p.run(dsa, ws=p.ws)
    assert dsa.get_status(p.ws) == dsa.STATUS_BAD_LENGTH
    assert torch.equal(p.out[:110], first[:110]) and bool((p.out[110:] == 5).all())


def test_one_sequence_needs_no_offsets():
    need_gpu()
    dsa = lib()
    p = Problem(14, same(130), Hq=4, Hk=2, Dk=64).run(dsa)
    first = p.out.clone()
    p.out.zero_()
    dsa.prompt_attn(p.q, p.k, p.v, p.scale, p.out, None, p.ws)
    assert torch.equal(p.out, first)
    p.out.zero_()
    dsa.prompt_attn(p.q, p.k, p.v, p.scale, p.out, None, p.ws, cu_q=p.cu_q)
    assert torch.equal(p.out, first)
    none = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    dsa.prompt_attn(none, p.k, p.v, p.scale, none, None, p.ws)                 # no tokens
    kv = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    p.run(dsa, ws=p.ws)
    dsa.prompt_attn(p.q, kv, kv, p.scale, p.out, p.lse, p.ws)                  # no keys
    assert bool((p.out == 0).all()) and bool((p.lse == -float("inf")).all())


def test_two_streams_with_their_own_workspaces():
    need_gpu()
    dsa = lib()
    ps = [Problem(20 + i, [(300, 900), (100, 100 + i)], Hq=8, Hk=2, Dk=128).run(dsa) for i in range(2)]
    want = [p.out.clone() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    for p in ps:
        p.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for p, st in zip(ps, streams):
            dsa.prompt_attn(p.q, p.k, p.v, p.scale, p.out, p.lse, p.ws, cu_q=p.cu_q, cu_k=p.cu_k, stream=st)
    torch.cuda.synchronize()
    for p, w in zip(ps, want):
        assert torch.equal(p.out, w)


def test_captured_call_follows_the_offsets():
    need_gpu()
    dsa = lib()
    p = Problem(30, same(400, 300, 100), Hq=4, Hk=1, Dk=64).run(dsa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.prompt_attn(p.q, p.k, p.v, p.scale, p.out, p.lse, p.ws, cu_q=p.cu_q, cu_k=p.cu_k)
    for nq, nk in (([400, 300, 100], [400, 300, 100]), ([1, 2, 3], [700, 2, 98]), ([0, 800, 0], [0, 800, 0]),
                   ([5, 5, 5], [0, 0, 800])):
        p.cu_q.copy_(torch.tensor(cu(nq), dtype=torch.int32))
        p.cu_k.copy_(torch.tensor(cu(nk), dtype=torch.int32))
        p.out.fill_(9.0)
        p.lse.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(nq)
        o, l, m = attend_prompt64(p.q, p.k, p.v, cu(nq), cu(nk), p.scale)
        assert_rows_close(p.out[:n], p.lse[:n], o[:n], l[:n], m[:n], ONE, f"{nq} over {nk}")
        assert bool((p.out[n:] == 9).all())


def test_two_graphs_of_one_workspace():
    need_gpu()
    dsa = lib()
    p = Problem(32, [(5, 4000), (100, 900)], Hq=4, Hk=2, Dk=64).run(dsa)
    want, other, graphs = p.out.clone(), torch.empty_like(p.out), []
    for out in (p.out, other):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            dsa.prompt_attn(p.q, p.k, p.v, p.scale, out, p.lse, p.ws, cu_q=p.cu_q, cu_k=p.cu_k)
        out.zero_()
    for _ in range(20):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want) and torch.equal(other, want)


def test_one_workspace_serves_problems_of_any_shape():
    need_gpu()
    dsa = lib()
    ps = [Problem(i, **CASES[n]) for i, n in enumerate(("cut-chunk", "one-token", "widest", "cut-wide-v", "many"))]
    ws = dsa.workspace(max(p.workspace(dsa).numel() for p in ps))
    for _ in range(2):
        for p in ps:
            p.run(dsa, ws=ws).check("shared workspace")
    assert dsa.get_status(ws) == 0


def test_rows_far_apart():
    """Token strides whose offsets pass 32 bits."""
    need_gpu()
    dsa = lib()
    step = (1 << 30) + 64
    buf = torch.zeros(2 * step + 4096, dtype=BF, device="cuda")
    p = Problem(31, same(3), Hq=4, Hk=4, Dk=64)
    for name, at in (("q", 0), ("k", 512), ("v", 1024)):
        far = buf[at:].as_strided((3, 4, 64), (step, 64, 1))
        far.copy_(getattr(p, name))
        setattr(p, name, far)
    p.out = buf[2048:].as_strided((3, 4, 64), (step, 64, 1))
    p.run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check("far", weight=TWO)
