"""The front page's example of grouped heads, run as it stands."""
import pytest
import torch

from gpu_common import lib, need_gpu
from prompt_reference import assert_rows_close, attend_prompt64
from test_examples_cpu import examples

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_packed_prompts_then_a_step_over_the_4_bit_cache():
    need_gpu()
    dsa = lib()
    (code,) = [e for e in examples() if "cache4_pool" in e]
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g).to(BF).cuda()  # noqa: E731
    B, Hq, Hk, Dk, Dv, block_size, lens = 2, 8, 2, 64, 48, 16, [37, 20]
    N, most = sum(lens), max(lens) + 1
    slots = (most + block_size - 1) // block_size
    num_blocks = B * slots
    table = torch.arange(num_blocks, dtype=torch.int32).view(B, slots).cuda()
    layout = dsa.PagedLayout(table, torch.tensor(lens, dtype=torch.int32).cuda() + 1, block_size, num_blocks, most)
    seq = torch.arange(B, dtype=torch.int32).repeat_interleave(torch.tensor(lens)).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    names = dict(dsa=dsa, B=B, N=N, Hq=Hq, Hk=Hk, Dk=Dk, Dv=Dv, block_size=block_size, num_blocks=num_blocks,
                 layout=layout, seq=seq, pos=pos, sm_scale=Dk ** -0.5, q=r(N, Hq, Dk), k=r(N, Hk, Dk), v=r(N, Hk, Dv),
                 k4=r(N, Hk, Dk), v4=r(N, Hk, Dv), out=r(N, Hq, Dv), lse=torch.zeros((N, Hq), device="cuda"),
                 cu=torch.tensor([0, lens[0], N], dtype=torch.int32).cuda(), k_new=r(B, Hk, Dk), v_new=r(B, Hk, Dv),
                 q_new=r(B, Hq, Dk), out_new=r(B, Hq, Dv), lse_new=torch.zeros((B, Hq), device="cuda"))
    exec(code, names)
    o, l, m = attend_prompt64(names["q"], names["k4"], names["v4"], [0, lens[0], N], [0, lens[0], N], Dk ** -0.5)
    assert_rows_close(names["out"], names["lse"], o, l, m, 2.0 ** -16, "prompts")
    # the step: the kept rows of each sequence and the new one's
    k1, v1 = r(B, Hk, Dk), r(B, Hk, Dv)
    last = torch.tensor(lens, dtype=torch.int32).cuda()
    dsa.cache4_read(layout, torch.arange(B, dtype=torch.int32).cuda(), last, names["pool"], k1, v1, names["ws4"])
    at = 0
    for b, n in enumerate(lens):
        kb, vb = torch.cat([names["k4"][at:at + n], k1[b:b + 1]]), torch.cat([names["v4"][at:at + n], v1[b:b + 1]])
        o, l, m = attend_prompt64(names["q_new"][b:b + 1], kb, vb, [0, 1], [0, n + 1], Dk ** -0.5)
        assert_rows_close(names["out_new"][b:b + 1], names["lse_new"][b:b + 1], o, l, m, 2.0 ** -11, f"step of {b}")
        at += n
