"""GPU tests of dsa_prefix_attn_decode where single positions count: masks of
every tile, positions that decide a row, the accuracy of short sequences."""
import numpy as np
import pytest
import torch

from gpu_common import lib, need_gpu
from test_gpu_prefix_attn import LATENT, Problem

pytestmark = pytest.mark.gpu


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
