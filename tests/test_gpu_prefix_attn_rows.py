"""GPU tests of dsa_prefix_attn_decode where single positions count: masks of
every tile, positions that decide a row, the accuracy of short sequences."""
import numpy as np
import pytest
import torch

from gpu_common import assert_out_close, lib, need_gpu
from heads_reference import assert_attn_close, attend64
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
