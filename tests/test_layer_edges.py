"""The operators around a scan at their edges: the failure path of the chunked selective scan,
and kernel instances and inputs that test_layer_ops.py does not reach."""

import math

import pytest
import torch

import delta_rule_recurrent_chunked_b200 as drs
import layer_ref as ref
from delta_rule_recurrent_chunked_b200 import build as drbuild
from test_layer_ops import (EPS, TYPES, U, conv_tol, device_status_stays_clear,  # noqa: F401
                            gen_of, norm_tol, rnd, ssm_check, ssm_inputs, within)


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


# ------------------------------------------------------------------ instances for large sizes

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,T,d,heads", [
    (torch.bfloat16, 3, 33337, 128, 1),  # four items a group: from 9472 CTAs of 8 on
    (torch.bfloat16, 5, 60641, 32, 1),   # .. of 32
    (torch.float32, 1, 37913, 128, 1),   # .. of 4
    (torch.bfloat16, 8, 9503, 128, 4),   # two items: from 4736 CTAs of 4 on
    (torch.float32, 3, 18953, 64, 3),    # .. with lanes behind a row
])
@pytest.mark.parametrize("act,first,shared", [("silu", False, True), ("sigmoid", True, False)])
def test_gated_norm_of_many_rows(dtype, H, T, d, heads, act, first, shared):
    """Thread groups that take several rows each, the last of them idle."""
    g = gen_of(T)
    y, gate = rnd(g, 1, H, T, d, dtype=dtype), rnd(g, 1, T, H * d, std=2.0, dtype=dtype)
    w = rnd(g, d if shared else H * d)
    want = ref.gated(y, gate, w, heads, act, first, EPS)
    out = drs.gated_norm(y, gate, w, norm_heads=heads, act=act, gate_first=first, eps=EPS)
    within(out, want, norm_tol(dtype, want, heads * d))
    same = drs.gated_norm(y, gate, w, norm_heads=heads, act=act, gate_first=first, eps=EPS, out=gate)
    assert torch.equal(same, out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [12713, 25417, 50633])
@pytest.mark.parametrize("K", [2, 4])
def test_short_conv_with_longer_tiles(dtype, T, K):
    """Tiles of 16, 32 and 64 tokens: the longest of which 9472 are left, in four columns of one
    head and three sequences."""
    g = gen_of(T + K)
    B, C, splits = 3, 128, [(1, 32, True), (1, 32, False), (1, 32, True), (1, 32, False)]
    x, w, bias = rnd(g, B, T, C, dtype=dtype), rnd(g, C, K, std=0.5), rnd(g, C, std=0.1)
    state0 = rnd(g, B, K - 1, C, dtype=dtype)
    lengths = [T, 0, T - 4711]
    mark = [torch.full((B, 1, T, 32), 7.0, dtype=dtype, device="cuda") for _ in splits]
    outs, final = drs.short_conv(x, w, bias, splits=splits, state0=state0, eps=EPS, outs=mark,
                                 lengths=torch.tensor(lengths, dtype=torch.int32).cuda())
    for b, n in enumerate(lengths):
        rows = torch.cat([ref.f64(state0[b]), ref.f64(x[b, :n])])
        assert torch.equal(ref.f64(final[b]), rows[n:])
        terms = rows.unfold(0, K, 1) * ref.f64(w) if n else torch.empty(0, C, K)
        c, m = terms.sum(-1) + ref.f64(bias), terms.abs().sum(-1) + ref.f64(bias).abs()
        for i, (_, d, normed) in enumerate(splits):
            v, mv = (t[:n, 32 * i:32 * i + 32] for t in (c, m))
            v = v * torch.sigmoid(v)
            if normed:
                r = 1 / torch.sqrt((v * v).sum(1, keepdim=True) + EPS)
                v, mv = v * r, mv * r
            within(outs[i][b, 0, :n], v, conv_tol(dtype, v, mv, normed, d), f"sequence {b} split {i}")
            assert (outs[i][b, 0, n:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("P", [32, 64, 128])
def test_ssm_scan_into_rows_on_odd_16_byte_places(P):
    i = ssm_inputs(P, 2, 3, 1, 300, P, 64, torch.bfloat16, "token", ragged=True)
    want = drs.ssm_scan(**{**i, "out": i["out"].clone()})
    wide = torch.full((2, 300, 3 * P + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    i["out"] = wide[..., 8:8 + 3 * P].unflatten(-1, (3, P)).transpose(1, 2)
    assert i["out"].data_ptr() % 32 == 16
    got = drs.ssm_scan(**i)
    ssm_check(i, got, torch.bfloat16, 300, 64)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (wide[..., :8] == 5.0).all() and (wide[..., 8 + 3 * P:] == 5.0).all()
