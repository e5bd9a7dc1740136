"""The operators around a scan at their edges: the failure path of the chunked selective scan,
and kernel instances and inputs that test_layer_ops.py does not reach."""

import math

import pytest
import torch

import delta_rule_recurrent_chunked_b200 as drs
from delta_rule_recurrent_chunked_b200 import build as drbuild
from test_layer_ops import U, device_status_stays_clear, ssm_inputs, within  # noqa: F401 (a fixture)


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


# ------------------------------------------------------------------ decays

@pytest.mark.gpu
@pytest.mark.parametrize("wiped", [40, 96, 104, 112])
def test_ssm_scan_gentle_tokens_behind_many_that_wipe_the_state(wiped):
    """The first `wiped` tokens of a chunk decay by 2^-161 each, those behind them hardly; only the
    first of these has an x, so each output is one weight of one token: off by the rounding of the
    weight and of the output to bf16 (2^-8 each, 2^-16 together), its fp32 factors (N + 64 u) and its
    decay, a difference of sums of a block of 32 tokens. There at most 16 tokens wipe, 2560 in all,
    so an addition is off by 2^-13, a sum by three of them, the difference by 6 * 2^-13 in the
    exponent of 2; where the block holds 8 (1280) by 6 * 2^-14, where none by 32 * 2^-21."""
    B, H, T, P, N = 8, 64, 128, 64, 32
    g = torch.Generator().manual_seed(wiped)
    delta = 1e-3 + 0.05 * torch.rand(B, H, T, generator=g)
    delta[:, :, :wiped] = 161 * math.log(2)
    pos = lambda *s: (0.5 + torch.rand(*s, generator=g)).to(torch.bfloat16)
    x, Bm, Cm = torch.zeros(B, H, T, P, dtype=torch.bfloat16), pos(B, H, T, N), pos(B, H, T, N)
    x[:, :, wiped] = pos(B, H, P)
    A = -torch.ones(H)
    out, S = drs.ssm_scan(x.cuda(), delta.cuda(), A.cuda(), Bm.cuda(), Cm.cuda(), dt_softplus=False)
    d64 = delta[:, :, wiped:].double()
    decay = torch.exp(-(d64.cumsum(-1) - d64[..., :1]))
    score = (Cm[:, :, wiped:].double() * Bm[:, :, wiped, None].double()).sum(-1)
    want = (score * decay * d64[..., :1])[..., None] * x[:, :, wiped, None].double()
    power = {40: 6 * 2.0 ** -14, 96: 32 * 2.0 ** -21, 104: 6 * 2.0 ** -14, 112: 6 * 2.0 ** -13}[wiped]
    tol = 2.0 ** -7 + 2.0 ** -16 + power * math.log(2) + (N + 64) * U
    within(out[:, :, wiped:], want, tol * want.abs())
    assert (out[:, :, :wiped] == 0).all()
    want = (decay[..., -1:] * d64[..., :1] * x[:, :, wiped].double())[..., None] * \
        Bm[:, :, wiped, None].double()
    within(S, want, 300 * U * want.abs())  # 128 steps, summed from the chunk's end
