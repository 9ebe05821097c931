"""Sizes and limits of dsa_prompt_attn and the 4-bit cache's calls that the host answers for."""
import ctypes

import pytest

from gpu_common import lib

dsa = lib()
FAKE = 0x100000                        # never dereferenced: the calls below fail validation


def _lay(**kw):
    f = dict(block_size=64, num_blocks=16, max_blocks_per_seq=4, batch=2, max_seq_len=200,
             block_table=0x10000, seq_lens=0x20000)
    f.update(kw)
    return ctypes.byref(dsa.PagedLayoutC(**f))


def test_the_prompt_s_workspace_serves_shorter_calls_too():
    """Asked for once with the largest batch: no smaller call needs more."""
    for heads in ((64, 8, 128, 128), (64, 64, 192, 128), (1, 1, 8, 8), (24, 4, 256, 256)):
        last = 0
        for B, Nq in ((1, 0), (1, 1), (4, 100), (4, 4096), (32, 16384), (1000, 1 << 20)):
            need = dsa.prompt_attn_workspace_size(B, Nq, *heads)
            assert need >= last, (heads, B, Nq)
            last = need


@pytest.mark.parametrize("Hk,D", [(1 << 27, 128), (1 << 26, 256), ((1 << 25) + 1, 128), (3 << 26, 64), ((1 << 31) - 1, 16),
                                  ((1 << 31) - 1, 256)])
def test_rows_of_more_heads_than_a_block_counts_are_refused(Hk, D):
    """(2^32 half groups of a token were 0 in 32 bits, and the host divided by them.)"""
    L = dsa.lib()
    assert L.dsa_cache4_read(_lay(), FAKE, FAKE, 1, Hk, D, D, None, None, FAKE, FAKE, FAKE, FAKE, 256, None) == -2
    assert L.dsa_cache4_write(_lay(), FAKE, FAKE, 1, FAKE, D, D, FAKE, D, D, Hk, D, D, None, None, FAKE, None, None,
                              FAKE, 256, None) == -2


@pytest.mark.parametrize("Hq,Hk,B,Nq", [(1 << 30, 1 << 30, 1, 1), ((1 << 31) - 1, (1 << 31) - 1, 1, 1),
                                        (1 << 30, 1 << 29, (1 << 31) - 1, 1), ((1 << 31) - 1, 1, (1 << 31) - 1, 1000),
                                        ((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1)])
def test_prompts_of_more_items_than_32_bits_count_are_refused(Hq, Hk, B, Nq):
    """(Heads of 256 take two items each: 2^30 of them were a negative count.)"""
    ws = dsa.prompt_attn_workspace_size(B, Nq, Hq, Hk, 256, 256)
    ts = 256 << 28
    assert dsa.lib().dsa_prompt_attn(FAKE, ts, 256, FAKE, ts, 256, FAKE, ts, 256, FAKE, FAKE, B, Nq, 1, Hq, Hk, 256, 256,
                                     0.1, FAKE, ts, 256, None, FAKE, ws, None) == -2
