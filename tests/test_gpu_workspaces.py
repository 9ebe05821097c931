"""GPU tests of one workspace that different calls take in turn."""
import pytest
import torch

import workloads as W
from gpu_common import lib, need_gpu
from test_gpu_bounds import TINY, _bounds, _cold_pages
from test_gpu_prompt_attn import Problem
from workloads import device as wdev

pytestmark = pytest.mark.gpu


def test_bounded_scores_and_prompts_in_turn():
    """The bounded scores' counts stay in the workspace until their next call; a prompt's counters are
    others, and neither call finds or changes the other's."""
    need_gpu()
    dsa = lib()
    c = W.make_case("bounded-then-prompt", seed=831, seq_lens=(4096, 1500), K=256, **TINY)
    c.kidx_pool = _cold_pages(c, 3, 832)
    d = wdev.upload(c, "cuda")
    lay = wdev.layout_of(c, d)
    kb = _bounds(dsa, c, d, lay)
    scores = torch.empty((c.B, 4096), dtype=torch.float32, device="cuda")
    p = Problem(60, [(300, 300), (2, 2600)], Hq=8, Hk=2, Dk=128)
    ws = dsa.workspace(max(p.workspace(dsa).numel(),
                           dsa.index_score_bounded_workspace_size(c.B, c.H_i, c.D_i, 4096, c.K)))
    counts = None
    for _ in range(3):
        scores.fill_(5.0)
        dsa.index_score_bounded(lay, d.q_idx, d.w, d.kidx_pool, kb, c.K, scores, ws)
        first = scores.clone() if counts is None else first
        counts = dsa.index_bounded_stats(ws) if counts is None else counts
        assert counts[0] > 0 and torch.equal(scores, first)
        p.out.fill_(5.0)
        p.run(dsa, ws=ws).check("a prompt on the scores' workspace")
        assert dsa.index_bounded_stats(ws) == counts
    assert dsa.get_status(ws) == 0


def test_a_workspace_for_the_largest_prompt_serves_the_shortest():
    need_gpu()
    dsa = lib()
    ws = dsa.workspace(dsa.prompt_attn_workspace_size(8, 16384, 64, 64, 16, 16))
    for seqs in ([(1, 4000)], [(100, 100)], [(40, 3500), (3, 2600), (200, 1700), (1, 100)]):
        p = Problem(62, seqs, Hq=64, Hk=64, Dk=16).run(dsa, ws=ws)
        p.check(f"{seqs}")
    assert dsa.get_status(ws) == 0
