"""GPU tests of the pools that cache_append fills and the attention reads."""
import numpy as np
import pytest
import torch

from gpu_common import lib, need_gpu
from heads_reference import assert_heads_close, transform64

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("slots,width,dtype", [(4, 64, BF), (4, 80, BF), (6, 72, F8)])
def test_heads_go_to_the_slots_of_a_pool_with_heads(slots, width, dtype):
    """Four heads of 64 into pools of other slot widths and counts; bytes that
    no head covers stay."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(slots * width)
    nb, bs, N = 5, 16, 9
    bt = torch.arange(nb, dtype=torch.int32).reshape(1, nb).flip(1).contiguous()
    lay = dsa.PagedLayout(bt.cuda(), torch.tensor([70], dtype=torch.int32).cuda(), bs, nb, nb * bs)
    x = torch.randn((N, 4, 64), generator=g).to(BF).cuda()
    pool = torch.full((nb, bs, slots, width), 3.0).to(dtype).cuda()
    pos = torch.arange(40, 40 + N, dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    dsa.cache_append(lay, torch.zeros(N, dtype=torch.int32).cuda(), pos.cuda(),
                     [dsa.HeadPart(x, pool, rope_dim=64, inv_freq=f)], ws)
    assert dsa.get_status(ws) == 0
    p = pos.numpy()
    rows = bt[0].numpy()[p // bs].astype(np.int64) * bs + p % bs
    flat = pool.float().cpu().reshape(nb * bs, slots, width)
    got = flat[rows][:, :4, :64]
    assert_heads_close(got.to(dtype), *transform64(x, pos, rope_dim=64, inv_freq=f))
    rest = torch.ones(flat.shape, dtype=torch.bool)
    rest[torch.from_numpy(rows), :4, :64] = False
    assert bool((flat[rest] == 3.0).all())
