"""GPU tests of dsa_prompt_attn at the edges of its ranges."""
import math

import pytest
import torch

from gpu_common import lib, need_gpu
from test_gpu_prompt_attn import Problem, same

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture
def room():
    """100 GB of free device memory, given back after the test."""
    need_gpu()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("100 GB of free device memory are needed")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("short", [0, 126, 127, 128])
def test_keys_next_to_the_largest_count(short, room):
    """Two tokens over 2^31 - 1 keys and somewhat fewer: the last key decides the last token's two heads,
    the token before it weighs all the others alike.  (Sums of ones and halves below 2^24 are exact.)"""
    dsa = lib()
    N = (1 << 31) - 1 - short
    k, v = torch.zeros((N, 1, 8), dtype=BF, device="cuda"), torch.full((N, 1, 8), 0.5, dtype=BF, device="cuda")
    q = torch.ones((2, 2, 8), dtype=BF, device="cuda")
    k[-1], v[-1] = 8.0, torch.arange(8, device="cuda").to(BF)
    out, lse = torch.full((2, 2, 8), 5.0, dtype=BF, device="cuda"), torch.full((2, 2), 5.0, device="cuda")
    ws = dsa.workspace(dsa.prompt_attn_workspace_size(1, 2, 2, 1, 8, 8))
    dsa.prompt_attn(q, k, v, 1.0, out, lse, ws)
    assert dsa.get_status(ws) == 0
    # (the others weigh (N - 1) exp(-64) < 2^-60 of the last token's)
    assert bool((out[0] == 0.5).all()) and torch.equal(out[1, :, 1:], v[-1, :, 1:].expand(2, 7))
    assert bool((out[1, :, 0].abs() <= 2.0 ** -60).all())
    # (an fp32 logarithm and its factor: 4 steps of a value below 32)
    assert bool(((lse[0] - math.log(N - 1)).abs() <= 2.0 ** -17).all())
    assert bool(((lse[1] - 64.0).abs() <= 2.0 ** -15).all())
    v[-1, 0, 3] = math.inf                                # what the products leave out is added in its place
    dsa.prompt_attn(q, k, v, 1.0, out, lse, ws)
    assert bool((out[0] == 0.5).all()) and torch.equal(out[1, :, 1:], v[-1, :, 1:].expand(2, 7))


@pytest.mark.parametrize("short", [0, 255])
def test_tokens_next_to_the_largest_count(short, room):
    """2^31 - 1 query tokens and somewhat fewer over three keys: only the last three see any."""
    dsa = lib()
    N = (1 << 31) - 1 - short
    q, out = torch.zeros((N, 1, 8), dtype=BF, device="cuda"), torch.full((N, 1, 8), 5.0, dtype=BF, device="cuda")
    k = torch.ones((3, 1, 8), dtype=BF, device="cuda")
    v = torch.tensor([1.0, 3.0, 5.0], device="cuda").to(BF)[:, None, None].expand(3, 1, 8).contiguous()
    lse = torch.full((N, 1), 5.0, device="cuda")
    ws = dsa.workspace(dsa.prompt_attn_workspace_size(1, N, 1, 1, 8, 8))
    dsa.prompt_attn(q, k, v, 1.0, out, lse, ws)
    assert dsa.get_status(ws) == 0
    assert out[-3:, 0, 0].tolist() == [1.0, 2.0, 3.0]
    assert float((lse[-3:, 0].cpu() - torch.tensor([1.0, 2.0, 3.0]).log()).abs().max()) <= 2.0 ** -21
    for i in range(0, N - 3, 1 << 28):
        j = min(N - 3, i + (1 << 28))
        assert int(out[i:j].count_nonzero()) == 0 and bool((lse[i:j] == -math.inf).all())


def _deciding(seqs, Hq, Hk, rounds):
    """A problem of keys of +-1 (a code of 64 dims for each), every row asking for one key by that key's
    code: the ones next to the borders of tiles, the sequence's first and last, in turn."""
    p = Problem(71, seqs, Hq=Hq, Hk=Hk, Dk=64, scale=1.0)
    p.k = torch.where(p.k.float() > 0, 1.0, -1.0).to(BF)
    G, queries = Hq // Hk, []
    for r in range(rounds):
        target, at, ak = [], 0, 0
        for s, (nq, nk) in enumerate(seqs):
            near = [x for x in range(nk) if x % 64 in (0, 1, 62, 63)] + [nk - 1, nk - 2]
            near = torch.tensor([x for x in near if x >= 0] or [0], device="cuda")
            i = torch.arange(nq * Hq, device="cuda").view(nq, Hq)
            t = near[(i + 7 * s + r * nq * Hq) % len(near)]
            last = torch.arange(nq, device="cuda")[:, None] + nk - nq
            target.append(ak + torch.where(t <= last, t, last.clamp(min=0)))
            at, ak = at + nq, ak + nk
        target = torch.cat(target)
        heads = torch.arange(Hq, device="cuda") // G
        queries.append(p.k[target, heads.expand_as(target)])
    return p, queries


def _check_exact(p, what, lse_tol=2.0 ** -15):
    """Against 64 bits on the GPU.  lse: products of +-1 are whole, so a score is off by the rounding of
    log2(e), of its product with a score up to 64 (2^6.6 in log2 units) and of the sum with the logarithm,
    2^-24 each of 2^6.6; beside it the sum of weights, 2^-20."""
    G, aq, ak = p.Hq // p.Hk, 0, 0
    for nq, nk in zip(p.nq, p.nk):
        last = torch.arange(nq, device="cuda") + nk - nq
        hidden = torch.arange(nk, device="cuda")[None, :] > last[:, None]
        for h in range(p.Hq):
            q, k, v = p.q[aq:aq + nq, h].double(), p.k[ak:ak + nk, h // G].double(), p.v[ak:ak + nk, h // G].double()
            z = (q @ k.t() * p.scale).masked_fill_(hidden, -math.inf)
            l = torch.logsumexp(z, -1)
            w = torch.where((l > -math.inf)[:, None], torch.softmax(z, -1), 0.0)
            o, m = w @ v, w @ v.abs()
            tol = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11) * m
            d = (p.out[aq:aq + nq, h].double() - o).abs()
            assert bool((d <= tol).all()), f"{what}: head {h}, row {(d > tol).any(-1).nonzero()[0].item()} of {nq} x {nk}"
            some = l > -math.inf
            assert bool(((p.lse[aq:aq + nq, h].double() - l)[some].abs() <= lse_tol).all()), f"{what}: lse, head {h}"
        aq, ak = aq + nq, ak + nk


DECIDING = {
    "one-row": dict(seqs=[(1, 5000)], Hq=128, Hk=1, rounds=3),
    "one-row-of-each-head": dict(seqs=[(1, 2500)] * 70, Hq=8, Hk=8, rounds=3),
    "chunks-in-pieces": dict(seqs=[(40, 3500), (3, 2600), (200, 1700), (1, 100)], Hq=4, Hk=2, rounds=3),
    "a-prompt-in-pieces": dict(seqs=[(2300, 2300)], Hq=2, Hk=1, rounds=2),
    "last-wave-in-pieces": dict(seqs=[(5, 40), (900, 3100), (0, 3)], Hq=40, Hk=8, rounds=1),
    "ragged": dict(seqs=[((37 * i) % 300, (37 * i) % 300 + (i % 3) * 150) for i in range(60)], Hq=6, Hk=2, rounds=2),
    "uncut": dict(seqs=[(700, 700), (1300, 1300)], Hq=3, Hk=3, rounds=2),
}


@pytest.mark.parametrize("name", DECIDING)
def test_every_key_at_a_border_counts_once(name):
    need_gpu()
    dsa = lib()
    p, queries = _deciding(**DECIDING[name])
    p.ws = p.workspace(dsa)
    for q in queries:
        p.q = q
        p.out.fill_(5.0)
        p.run(dsa, ws=p.ws)
        _check_exact(p, name)
    assert dsa.get_status(p.ws) == 0


def test_a_long_prompt_of_many_items_per_sm():
    """From twelve items per SM on nothing is cut: 4,000 tokens of 120 heads, and ragged ones."""
    need_gpu()
    dsa = lib()
    p, (q,) = _deciding([(4000, 4000)], 120, 120, 1)
    p.q = q
    p.run(dsa)
    _check_exact(p, "long")
    p = Problem(72, same(1700, 3, 900, 128, 2100), Hq=128, Hk=32, Dk=128).run(dsa)
    # (N(0, 1): a score is a sum of 128 products of size 1, off by 2^-24 of each partial sum below 64 at
    # worst, 128 * 2^-18 / 11)
    _check_exact(p, "ragged", lse_tol=2.0 ** -14)
    assert dsa.get_status(p.ws) == 0


def test_many_items_with_and_without_odd_values():
    """Sixteen items and more for every CTA, one in eight of them with infinities or NaN in V."""
    need_gpu()
    dsa = lib()
    seqs = [(1 + (37 * i) % 100, 1 + (37 * i) % 100 + (600 if i % 3 == 0 else i % 50)) for i in range(640)]
    p = Problem(73, seqs, Hq=4, Hk=4, Dk=32)
    g = torch.Generator().manual_seed(74)
    begin = p.cu_k.tolist()
    v = p.v.cpu()
    for i in range(0, 640, 8):
        nk = seqs[i][1]
        for value in (math.inf, -math.inf, math.nan):
            at = torch.randint(0, nk, (1,), generator=g).item()
            h, d = torch.randint(0, 4, (1,), generator=g).item(), torch.randint(0, 32, (1,), generator=g).item()
            v[begin[i] + at, h, d] = value
    p.v = v.cuda()
    p.run(dsa)
    assert dsa.get_status(p.ws) == 0
    p.check("odd values")
    first, lse = p.out.clone(), p.lse.clone()
    for _ in range(20):
        p.out.fill_(3.0)
        p.run(dsa, ws=p.ws)
        assert torch.equal(p.out.view(torch.int16), first.view(torch.int16)) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("power", [0, 5, 10, 14, 16, 18, 20, 22, 25, 30, 60, 115])
@pytest.mark.parametrize("seqs,Hq,Hk", [([(3, 3000), (70, 70)], 16, 2), ([(2, 5000)], 128, 1), ([(300, 700)], 3, 3)])
def test_scores_of_any_size(seqs, Hq, Hk, power):
    """Scores of up to 64 * 2^power, whole and exact in fp32, up to where fp32 ends: the key that a row asks
    for is there twice (tiles or pieces apart), so that its two places share the row in halves."""
    need_gpu()
    dsa = lib()
    p, (q,) = _deciding(seqs, Hq, Hk, 1)
    ak = 0
    for nq, nk in seqs:                                   # the second half of the keys repeats the first
        p.k[ak + nk // 2:ak + nk // 2 * 2] = p.k[ak:ak + nk // 2]
        ak += nk
    target = torch.tensor([min(7, nk // 2 - 1) for nq, nk in seqs for _ in range(nq)], device="cuda")
    base = torch.tensor([b for (nq, _), b in zip(seqs, p.cu_k.tolist()) for _ in range(nq)], device="cuda")
    p.q = p.k[base + target].repeat_interleave(Hq // Hk, 1) * 2.0 ** power
    p.run(dsa)
    assert dsa.get_status(p.ws) == 0
    # lse: as _check_exact's, of scores 2^power times as large
    _check_exact(p, f"2^{power}", lse_tol=2.0 ** (power - 15))


def test_items_that_take_longer_than_a_wait_of_their_parts(room):
    """One token of 193 heads over 200 million keys: more items than SMs and too few partial results to cut
    them, so the warps that an item has no work for wait seconds for the next."""
    dsa = lib()
    N, Hq = 200_000_000, 193
    k, v = torch.zeros((N, 1, 8), dtype=BF, device="cuda"), torch.full((N, 1, 8), 0.5, dtype=BF, device="cuda")
    q = torch.ones((1, Hq, 8), dtype=BF, device="cuda")
    q[0, 1::2] = -1.0
    k[-1], v[-1] = 8.0, 3.0
    out, lse = torch.full((1, Hq, 8), 5.0, dtype=BF, device="cuda"), torch.full((1, Hq), 5.0, device="cuda")
    ws = dsa.workspace(dsa.prompt_attn_workspace_size(1, 1, Hq, 1, 8, 8))
    dsa.prompt_attn(q, k, v, 1.0, out, lse, ws)
    assert dsa.get_status(ws) == 0
    # even heads see the last key alone (the others weigh exp(-64) N < 2^-60), odd ones all but it: the sums
    # of ones end at 2^24 in fp32, as the sums of halves do, so what is left is the order of size
    assert bool((out[0, ::2] == 3.0).all()) and bool(((lse[0, ::2] - 64.0).abs() <= 2.0 ** -15).all())
    assert bool(((out[0, 1::2] > 0.2) & (out[0, 1::2] < 1.1)).all())


def test_long_sums_are_not_cut_off():
    """193 heads of one token over a million keys and positive values, in as many uncut items.  A weight's
    rounding averages out over so many; the matrix unit's sums lose 2^-27 for each of 65,536 keys, an item's
    sum of them and the sum of weights next to nothing; the output is rounded once."""
    need_gpu()
    dsa = lib()
    N, Hq = 1_000_000, 193
    g = torch.Generator().manual_seed(75)
    k, q = torch.randn((N, 1, 8), generator=g).to(BF).cuda(), (torch.randn((1, Hq, 8), generator=g) * 0.5).to(BF).cuda()
    v = (torch.rand((N, 1, 8), generator=g) + 0.5).to(BF).cuda()
    out, lse = torch.full((1, Hq, 8), 5.0, dtype=BF, device="cuda"), torch.full((1, Hq), 5.0, device="cuda")
    ws = dsa.workspace(dsa.prompt_attn_workspace_size(1, 1, Hq, 1, 8, 8))
    dsa.prompt_attn(q, k, v, 1.0, out, lse, ws)
    assert dsa.get_status(ws) == 0
    z = q[0].double() @ k[:, 0].double().t()
    want, l = torch.softmax(z, -1) @ v[:, 0].double(), torch.logsumexp(z, -1)
    d = (out[0].double() - want) / want
    assert float(d.abs().max()) <= 2.0 ** -8 + 2.0 ** -10, float(d.abs().max())
    assert abs(float(d.mean())) <= 2.0 ** -10, float(d.mean())
    # (7,813 tiles' sums added one by one, half a step of a sum that is half of the last on average)
    assert float((lse[0].double() - l).abs().max()) <= 7813 * 2.0 ** -25


@pytest.mark.parametrize("Hq,nq,nk", [(193, 1, 300_000), (16, 2, 400_000), (40, 130, 270_000)])
def test_maxima_that_rise_across_long_sums(Hq, nq, nk):
    """Every row asks for one key of many: O that has left for the workspace is scaled with what follows."""
    need_gpu()
    dsa = lib()
    p = Problem(76, [(nq, nk)], Hq=Hq, Hk=1, Dk=64, Dv=40, scale=1.0)
    p.k = torch.where(p.k.float() > 0, 1.0, -1.0).to(BF)
    g = torch.Generator().manual_seed(77)
    target = torch.randint(0, nk - nq, (nq, Hq), generator=g)
    target[0, :3] = torch.tensor([0, 65535, 65536])
    for scale in (1.0, 0.3, 2.0 ** 40):                    # one key; a few; scores that are rounded
        p.q, p.scale = p.k[target.cuda(), 0], scale
        p.out.fill_(5.0)
        p.run(dsa)
        assert dsa.get_status(p.ws) == 0
        _check_exact(p, f"scale {scale}", lse_tol=2.0 ** -15 * max(1.0, scale))
