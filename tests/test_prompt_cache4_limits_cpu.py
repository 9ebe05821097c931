"""Sizes and limits of dsa_prompt_attn and the 4-bit cache's calls that the host answers for."""
import pytest

from gpu_common import lib

dsa = lib()


def test_the_prompt_s_workspace_serves_shorter_calls_too():
    """Asked for once with the largest batch: no smaller call needs more."""
    for heads in ((64, 8, 128, 128), (64, 64, 192, 128), (1, 1, 8, 8), (24, 4, 256, 256)):
        last = 0
        for B, Nq in ((1, 0), (1, 1), (4, 100), (4, 4096), (32, 16384), (1000, 1 << 20)):
            need = dsa.prompt_attn_workspace_size(B, Nq, *heads)
            assert need >= last, (heads, B, Nq)
            last = need
