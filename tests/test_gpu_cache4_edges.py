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
