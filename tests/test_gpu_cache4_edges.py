"""GPU tests of the 4-bit cache's decode attention at the edges of its ranges."""
import pytest
import torch

from gpu_common import lib, need_gpu
from test_gpu_cache4 import Attn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


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
