"""GPU tests of dsa_prompt_attn at the edges of its ranges."""
import math

import pytest
import torch

from gpu_common import lib, need_gpu

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
