"""The operators around a scan at their edges: the failure path of the chunked selective scan,
and kernel instances and inputs that test_layer_ops.py does not reach."""

import pytest
import torch

import delta_rule_recurrent_chunked_b200 as drs
from delta_rule_recurrent_chunked_b200 import build as drbuild
from test_layer_ops import ssm_inputs


# ------------------------------------------------------------------ a wait that runs out

def test_wait_limit_refusals():
    drbuild.build_library()
    call = drs.lib().dr_debug_wait_limit
    for bad in (-2, 2000000001, 1 << 40):
        assert call(bad) == drs.DR_ERR_INVALID_ARG
    for good in (0, 1000, 2000000000, -1):
        assert call(good) == drs.DR_OK
    assert call(-1) == drs.DR_OK


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,P,N", [(1, 2, 100, 64, 64),     # one chunk: no tile is loaded twice
                                       (2, 3, 250, 128, 128),   # two
                                       (3, 40, 900, 64, 128),   # many heads, one segment
                                       (1, 4, 6000, 64, 128)])  # in segments
def test_ssm_scan_gives_up_on_a_wait_and_returns(B, H, T, P, N):
    """With a limit of 0 the first poll that fails ends its role, with longer ones some wait on the
    way. The kernel returns well before the 2 s that it grants the loads and products it started,
    latches the status, and leaves nothing behind: the next scans give their usual bits."""
    assert drs.poll_error() == drs.DR_OK
    i = ssm_inputs(T, B, H, 1, T, P, N, torch.bfloat16, "token")
    run = lambda: drs.ssm_scan(**{**i, "out": torch.zeros_like(i["out"])})
    want = [t.clone() for t in run()]
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for limit in (0, 0, 100, 500, 1000, 2000, 5000, 20000, 100000):
        torch.cuda.synchronize()
        assert drs.lib().dr_debug_wait_limit(limit) == drs.DR_OK
        try:
            begin.record()
            run()
            end.record()
        finally:
            assert drs.lib().dr_debug_wait_limit(-1) == drs.DR_OK
        torch.cuda.synchronize()
        assert begin.elapsed_time(end) < 1000.0
        assert drs.poll_error() in ((drs.DR_ERR_TIMEOUT,) if limit == 0
                                    else (drs.DR_OK, drs.DR_ERR_TIMEOUT))
        for _ in range(3):
            for a, b in zip(run(), want):
                assert torch.equal(a, b)
        assert drs.poll_error() == drs.DR_OK
