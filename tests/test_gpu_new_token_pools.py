"""GPU tests of the pools that cache_append fills and the attention reads."""
import numpy as np
import pytest
import torch

from gpu_common import lib, need_gpu
from heads_reference import assert_attn_close, assert_heads_close, attend64, transform64

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


def test_each_key_head_of_a_pool_of_several_is_attended_by_a_call_of_its_own():
    """cache_append fills K and V rows of four heads; the C call on a head's
    first element, with the rows' stride, attends its group of query heads."""
    need_gpu()
    dsa = lib()
    g = torch.Generator().manual_seed(77)
    B, Hk, G, D, bs, nb = 3, 4, 6, 64, 16, 40
    lens = [200, 33, 129]
    bt = torch.full((B, 13), -1, dtype=torch.int32)
    order = torch.randperm(nb, generator=g).int()
    at = 0
    for b, n in enumerate(lens):
        pages = (n + bs - 1) // bs
        bt[b, :pages] = order[at:at + pages]
        at += pages
    N = sum(lens)
    seq = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], dtype=torch.int32)
    pos = torch.tensor([p for n in lens for p in range(n)], dtype=torch.int32)
    kv = torch.randn((N, 2 * Hk, D), generator=g).to(BF).cuda()
    kp = torch.full((nb, bs, Hk * D), float("nan"), dtype=BF, device="cuda")
    vp = kp.clone()
    lay = dsa.PagedLayout(bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), bs, nb, 13 * bs)
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    ws = dsa.workspace(dsa.cache_append_workspace_size())
    dsa.cache_append(lay, seq.cuda(), pos.cuda(),
                     [dsa.HeadPart(kv[:, :Hk], kp, norm="rms", rope_dim=D, inv_freq=f),
                      dsa.HeadPart(kv[:, Hk:], vp)], ws)
    q = torch.randn((B, Hk, G, D), generator=g).to(BF).cuda()
    wa = dsa.workspace(dsa.prefix_attn_decode_workspace_size(B, G, D, D, 0))
    scale = float(np.float32(D ** -0.5))
    for h in range(Hk):
        qh = q[:, h].contiguous()
        out = torch.empty((B, G, D), dtype=BF, device="cuda")
        lse = torch.empty((B, G), device="cuda")
        at = 2 * h * D                                   # bytes
        rc = dsa.lib().dsa_prefix_attn_decode(
            lay.c(), qh.data_ptr(), kp.data_ptr() + at, Hk * D, vp.data_ptr() + at, Hk * D, G, D, D, 0,
            scale, out.data_ptr(), lse.data_ptr(), wa.data_ptr(), wa.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        k, v = (t[..., h * D:(h + 1) * D].contiguous() for t in (kp, vp))
        want, lse_want, mag = attend64(qh, k, v, bt.numpy(), lens, bs, nb, 0, scale, D)
        assert_attn_close(out, lse, want, lse_want, mag, f"key head {h}")
    assert dsa.get_status(ws) == 0 and dsa.get_status(wa) == 0
