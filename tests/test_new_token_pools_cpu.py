"""Shapes and types of the tensors that the new-token calls take, on the host:
what the binding hands to the C ABI, and what it refuses before."""
import pytest
import torch

from gpu_common import lib

dsa = lib()
BF = torch.bfloat16


def _x(heads, dim, n=3):
    return torch.zeros((n, heads, dim), dtype=BF)


@pytest.mark.parametrize("heads,dim,shape,row,head", [
    (4, 64, (8, 16, 4, 64), 256, 64),
    (4, 64, (8, 16, 4, 80), 320, 80),          # head slots wider than the head
    (4, 64, (8, 16, 6, 64), 384, 64),          # more slots than heads
    (1, 64, (8, 16, 1, 64), 64, 64),
    (4, 64, (8, 16, 256), 256, 64),            # a 3-D pool's heads are packed
    (4, 64, (8, 16, 320), 320, 64),
])
def test_a_part_s_rows_and_heads_lie_where_the_pool_s_shape_says(heads, dim, shape, row, head):
    pool = torch.zeros(shape, dtype=BF)
    parts = dsa.HeadParts([dsa.HeadPart(_x(heads, dim), pool)])
    c = parts.c(True)[0]
    assert (c.out_token_stride, c.out_head_stride) == (row, head)
    assert parts.pool_rows == 8 * 16


@pytest.mark.parametrize("shape", [(8, 16, 2, 128), (8, 16, 4, 56), (8, 16, 3, 64), (8, 16, 1, 256)])
def test_a_pool_whose_heads_do_not_hold_the_part_s_is_refused(shape):
    with pytest.raises(ValueError, match="pool"):
        dsa.HeadParts([dsa.HeadPart(_x(4, 64), torch.zeros(shape, dtype=BF))]).c(True)
