"""The whole-warp bounded wait of the CTA-pair attention, exercised without a
hang: it gives up after its limit, or as soon as the abort flag is raised, and
reports; a completed barrier passes; the context stays usable."""
import ctypes

import pytest
import torch

from gpu_common import lib, need_gpu
from test_gpu_prefix_attn import LATENT, Problem

pytestmark = pytest.mark.gpu


def _ms(dsa, mode, limit_ns, ws):
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    rc = dsa.lib().dsa_selftest_warp_wait(mode, ctypes.c_uint64(limit_ns), ctypes.c_void_p(ws.data_ptr()),
                                          ws.numel(),
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, dsa.lib().dsa_last_error_string()
    ev[1].record()
    torch.cuda.synchronize()
    return ev[0].elapsed_time(ev[1])


def test_a_warp_s_wait_gives_up_and_reports():
    need_gpu()
    dsa = lib()
    ws = dsa.workspace(256)
    _ms(dsa, 0, 1_000_000_000, ws)
    assert dsa.get_status(ws) == 0
    ms = _ms(dsa, 1, 20_000_000, ws)
    assert 19.0 <= ms < 500.0                             # its limit, no more
    assert dsa.get_status(ws) == dsa.STATUS_TIMEOUT
    ms = _ms(dsa, 2, 1_000_000_000, ws)
    assert 4.0 <= ms < 500.0                              # the flag ends it, not the second's limit
    assert dsa.get_status(ws) == dsa.STATUS_TIMEOUT
    p = Problem(70, [300, 129, 1000], bs=64, prefix=0, **LATENT).run(dsa)
    p.check("after the waits that gave up")
    assert dsa.get_status(p.ws) == 0


def test_the_warp_wait_selftest_rejects_bad_arguments():
    need_gpu()
    dsa = lib()
    ws = dsa.workspace(256)
    n0 = dsa.launch_count()
    for mode, limit in ((1, 0), (1, 10), (1, 2_000_000_000), (-1, 20_000_000), (3, 20_000_000)):
        assert dsa.lib().dsa_selftest_warp_wait(mode, ctypes.c_uint64(limit),
                                                ctypes.c_void_p(ws.data_ptr()), ws.numel(), None) == -1
    assert dsa.launch_count() == n0
