"""GPU parity of the operators around a scan (short convolution, selective state space scan, its
one-token step, gated norm, block norm) against their definitions in fp64.

Tolerances. u is the unit roundoff of fp32 (2^-24), h that of the output's type (bf16 2^-8, fp32
2^-24), mag the sum of the magnitudes that enter an output. One rounding of the output costs
h |y|; everything else is bounded relative to mag, as the comment at each check says."""
import ctypes
import math

import numpy as np
import pytest
import torch

import delta_rule_recurrent_chunked_b200 as drs
import layer_ref as ref
from delta_rule_recurrent_chunked_b200 import build as drbuild

U = 2.0 ** -24
H_OF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float32]
EPS = 1e-6


@pytest.fixture(autouse=True)
def device_status_stays_clear(request):
    """No kernel latched a status (a wait that ran out) during a GPU test."""
    yield
    if "gpu" in request.keywords:
        assert drs.poll_error() == drs.DR_OK


def rnd(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen) * std).to(dtype).cuda()


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol, what=""):
    """Every element that has a value within tol (a tensor or number)."""
    got = ref.f64(got)
    live = ~torch.isnan(want)
    err = (got - want).abs()
    bad = live & ~(err <= tol)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        t = tol[i] if torch.is_tensor(tol) else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(live.sum())} off, first at {i}: "
                             f"{float(got[i])} for {float(want[i])}, tolerance {float(t)}")


# ------------------------------------------------------------------ refusals (no GPU)

A16 = 0x10000  # a fake, 16-byte aligned address: validation rejects before any dereference


@pytest.fixture(scope="module")
def lib():
    drbuild.build_library()
    return drs.lib()


def view(p=A16, sb=0, sh=0, st=0):
    return drs.DrView(p, sb, sh, st)


def at(*views):
    """The addresses of views (kept alive by the caller's arguments)."""
    return [ctypes.addressof(v) for v in views]


def call_conv(lib, x=None, w=A16, bias=None, state0=None, lengths=None, splits=None, final=None,
              eps=1e-6, B=2, T=8, C=64, K=4, mode=drs.DR_IN_BF16, step=False, state=A16):
    P = ctypes.c_void_p
    x = view(sb=8 * C, st=C) if x is None else x
    if splits is None:
        splits = [drs.ConvSplit(view(sb=8 * C, sh=8 * 32, st=32), C // 32, 32, 0)]
    arr = (drs.ConvSplit * max(1, len(splits)))(*splits)
    if step:
        return lib.short_conv_step(*at(x), P(w), P(bias), P(state), arr, len(splits), eps, B, C, K, mode,
                                   None)
    return lib.short_conv_fwd(*at(x), P(w), P(bias), P(state0), P(lengths), arr, len(splits), P(final),
                              eps, B, T, C, K, mode, None)


INV, UNS, OK = drs.DR_ERR_INVALID_ARG, drs.DR_ERR_UNSUPPORTED, drs.DR_OK


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), INV), (dict(w=A16 + 4), INV), (dict(bias=A16 + 8), INV),
    (dict(x=view(None, 512, 0, 64)), INV), (dict(x=view(A16 + 2, 512, 0, 64)), INV),
    (dict(x=view(A16, 512, 0, 63)), INV),            # rows not on 16-byte boundaries
    (dict(x=view(A16, 512, 0, 32)), INV),            # rows that overlap
    (dict(x=view(A16, -512, 0, 64)), INV),
    (dict(state0=A16 + 2), INV), (dict(final=A16 + 2), INV), (dict(lengths=A16 + 2), INV),
    (dict(state0=A16, final=A16), INV),
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(C=0), INV), (dict(K=0), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(mode=0x2000), INV),
    (dict(splits=[]), INV),
    (dict(splits=[drs.ConvSplit(view(sb=512, sh=256, st=32), 1, 32, 0)]), INV),    # not all channels
    (dict(splits=[drs.ConvSplit(view(None, 512, 256, 32), 2, 32, 0)]), INV),
    (dict(splits=[drs.ConvSplit(view(A16, 512, 256, 0), 2, 32, 0)]), INV),         # rows overlap
    (dict(splits=[drs.ConvSplit(view(A16, 512, 16, 32), 2, 32, 0)]), INV),
    (dict(splits=[drs.ConvSplit(view(A16, 256, 256, 32), 2, 32, 0)]), INV),  # batches into heads
    (dict(splits=[drs.ConvSplit(view(sb=512, sh=256, st=32), 4, 16, 0)]), UNS),
    (dict(K=5), UNS), (dict(K=1), UNS),
    (dict(T=16776961, B=1, splits=[drs.ConvSplit(view(sh=1 << 30, st=32), 2, 32, 0)]), UNS),
    (dict(T=(1 << 31) - 1, B=1, splits=[drs.ConvSplit(view(sh=1 << 36, st=32), 2, 32, 0)]), UNS),
    (dict(splits=[drs.ConvSplit(view(sb=512, sh=256, st=32), 1, 32, 0)] * 5, C=160,
          x=view(sb=2000, st=160)), UNS),
    (dict(B=0), OK), (dict(B=0, x=view(None)), OK), (dict(T=0), OK), (dict(T=0, w=None), OK),
])
def test_short_conv_refusals(lib, kw, code):
    assert call_conv(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(state=None), INV), (dict(state=A16 + 4), INV), (dict(w=None), INV), (dict(K=6), UNS),
    (dict(mode=0x2000), INV), (dict(B=0), OK), (dict(B=0, state=None), OK),
])
def test_short_conv_step_refusals(lib, kw, code):
    assert call_conv(lib, step=True, **kw) == code


def call_ssm(lib, x=None, dt=None, A=A16, b=None, c=None, D=None, bias=None, S0=None, lengths=None,
             out=None, Sf=None, B=2, H=4, G=2, T=8, P=64, N=64, mode=drs.DR_IN_BF16, step=False,
             S=A16):
    V = ctypes.c_void_p
    x = view(sb=H * T * P, sh=T * P, st=P) if x is None else x
    out = view(sb=H * T * P, sh=T * P, st=P) if out is None else out
    b = view(sb=G * T * N, sh=T * N, st=N) if b is None else b
    c = view(sb=G * T * N, sh=T * N, st=N) if c is None else c
    dt = view(sb=H * T, sh=T, st=1) if dt is None else dt
    if step:
        return lib.ssm_step(*at(x, dt), V(A), *at(b, c), V(D), V(bias), V(S), *at(out), B, H, G, P, N,
                            mode, None)
    return lib.ssm_scan_fwd(*at(x, dt), V(A), *at(b, c), V(D), V(bias), V(S0), V(lengths), *at(out),
                            V(Sf), B, H, G, T, P, N, mode, None)


SSM_REFUSALS = [
    (dict(A=None), INV), (dict(A=A16 + 4), INV), (dict(D=A16 + 4), INV), (dict(bias=A16 + 8), INV),
    (dict(x=view(None, 8, 8, 8)), INV), (dict(x=view(A16 + 8, 2048, 512, 64)), INV),
    (dict(b=view(A16, 1024, 512, 60)), INV) , (dict(c=view(A16, -8, 512, 64)), INV),
    (dict(out=view(A16, 2048, 0, 64)), INV),        # heads written over one another
    (dict(out=view(A16, 64, 64, 2048)), INV),       # batches over heads, in a scan and in a step
    (dict(dt=view(None)), INV), (dict(dt=view(A16 + 2, 32, 8, 1)), INV),
    (dict(dt=view(A16 + 1, 32, 8, 1), mode=drs.DR_IN_BF16 | drs.SSM_DT_BF16), INV),
    (dict(G=3), INV), (dict(G=0), INV), (dict(H=-1), INV), (dict(P=0), INV),
    (dict(mode=drs.DR_IN_BF16 | 0x4000), INV), (dict(mode=drs.DR_GDN), INV),
    (dict(P=48), UNS), (dict(N=256), UNS),
    (dict(B=0), OK), (dict(H=0), OK), (dict(B=0, x=view(None), A=None), OK),
]


@pytest.mark.parametrize("kw,code", SSM_REFUSALS + [
    (dict(S0=A16 + 8), INV), (dict(Sf=A16 + 8), INV), (dict(S0=A16, Sf=A16), INV),
    (dict(lengths=A16 + 1), INV), (dict(T=-1), INV), (dict(T=0, x=view(None)), OK),
    (dict(T=(1 << 30) + 1), UNS), (dict(T=(1 << 31) - 1, B=1, H=1, G=1), UNS),
    (dict(T=(1 << 31) - 1, B=1, H=1, G=1, mode=0), UNS),
])
def test_ssm_scan_refusals(lib, kw, code):
    assert call_ssm(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [r for r in SSM_REFUSALS if "b" not in r[0]] + [
    (dict(S=None), INV), (dict(S=A16 + 8), INV),
    (dict(mode=drs.DR_IN_BF16 | drs.DR_FORCE_SEQUENTIAL), INV), (dict(B=0, S=None), OK),
])
def test_ssm_step_refusals(lib, kw, code):
    assert call_ssm(lib, step=True, **kw) == code


def call_gated(lib, y=None, gate=None, w=A16, out=None, eps=1e-6, B=2, H=4, T=8, d=64, heads=1,
               mode=drs.DR_IN_BF16):
    y = view(sb=H * T * d, sh=T * d, st=d) if y is None else y
    gate = view(sb=T * H * d, st=H * d) if gate is None else gate
    out = view(sb=T * H * d, st=H * d) if out is None else out
    return lib.gated_norm_fwd(*at(y, gate), ctypes.c_void_p(w), *at(out), eps, B, H, T, d, heads,
                              mode, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), INV), (dict(w=A16 + 4), INV), (dict(y=view(None)), INV),
    (dict(out=view(None)), INV), (dict(out=view(A16, 2048, 0, 64)), INV),
    (dict(out=view(A16, 1024, 0, 256)), INV),       # the second sequence's rows among the first's
    (dict(gate=view(A16 + 2, 2048, 0, 256)), INV), (dict(heads=3), INV), (dict(heads=0), INV),
    (dict(eps=-1.0), INV), (dict(mode=0x8000), INV), (dict(d=48), UNS),
    (dict(H=512, heads=512), UNS), (dict(H=128, heads=128, d=128, mode=0), UNS),
    (dict(B=0), OK), (dict(T=0, y=view(None)), OK), (dict(H=0, w=None), OK),
])
def test_gated_norm_refusals(lib, kw, code):
    assert call_gated(lib, **kw) == code


def call_block(lib, x=A16, pitch=64, res=None, w=A16, post=None, sv=None, out=A16, ro=None,
               eps=1e-6, rows=4, D=64, mode=drs.DR_IN_BF16):
    P = ctypes.c_void_p
    return lib.block_norm_fwd(P(x), pitch, P(res), P(w), P(post), P(sv), 1.0, P(out), P(ro), eps,
                              rows, D, mode, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(x=A16 + 2), INV),
    (dict(res=A16 + 2), INV), (dict(post=A16 + 4), INV), (dict(sv=A16 + 4), INV),
    (dict(ro=A16 + 8), INV), (dict(pitch=63), INV), (dict(pitch=-64), INV), (dict(rows=-1), INV),
    (dict(D=0), INV), (dict(mode=0x2000), INV), (dict(eps=-1e-6), INV), (dict(D=60), UNS),
    (dict(D=16392), UNS), (dict(D=8196, mode=0), UNS), (dict(rows=0), OK),
    (dict(rows=0, x=None, w=None, out=None), OK),
])
def test_block_norm_refusals(lib, kw, code):
    assert call_block(lib, **kw) == code


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    x = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        drs.short_conv(x, torch.zeros(64, 4), splits=[(2, 32)])
    with pytest.raises(ValueError, match="bf16 or fp32"):
        drs.block_norm(x.to(torch.float16), torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        drs.gated_norm(torch.zeros(1, 2, 4, 32), None, torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        drs.ssm_scan(torch.zeros(1, 2, 4, 32), torch.zeros(1, 2, 4), torch.zeros(2),
                     torch.zeros(1, 1, 4, 32), torch.zeros(1, 1, 4, 32))


# ------------------------------------------------------------------ short convolution

def conv_tol(dtype, want, mag, normalised, d):
    """The sum has K + 1 terms: (K + 1) u mag; silu multiplies an error of c by at most 1.1 and
    adds a few u of its own (exp of an argument up to 100 off by 100 u); the norm divides by a
    sum of d squares: (d + 4) u more, and, before it is divided, mag is divided with it."""
    return H_OF[dtype] * want.abs() + (150 + (2 * d if normalised else 0)) * U * (mag + want.abs())


CONV_SPLITS = [
    [(2, 64, False)],
    [(3, 128, True), (3, 128, True), (3, 64, False)],
    [(5, 32, False), (1, 64, True), (1, 64, False), (2, 128, True)],
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("splits", CONV_SPLITS)
@pytest.mark.parametrize("T,ragged", [(1, False), (2, True), (7, False), (8, True), (9, False),
                                      (33, True), (70, False)])
def test_short_conv(dtype, K, splits, T, ragged):
    g = gen_of(T * 10 + K)
    B, C = 3, sum(s[0] * s[1] for s in splits)
    x = rnd(g, B, T, C, dtype=dtype)
    w, bias = rnd(g, C, K, std=0.5), rnd(g, C, std=0.1)
    state0 = rnd(g, B, K - 1, C, dtype=dtype) if ragged else None
    lengths = torch.tensor([T, 0, max(0, T - 2)], dtype=torch.int32).cuda() if ragged else None
    mark = [torch.full((B, s[0], T, s[1]), 7.0, dtype=dtype, device="cuda") for s in splits]
    outs, final = drs.short_conv(x, w, bias, splits=splits, state0=state0, lengths=lengths, eps=EPS,
                                 outs=mark)
    want, wfinal, mags = ref.conv(x, w, bias, splits, state0, lengths, EPS)
    for o, y, m, s in zip(outs, want, mags, splits):
        within(o, y, conv_tol(dtype, y, m, s[2], s[1]), "out")
        assert (ref.f64(o)[torch.isnan(y)] == 7.0).all()  # rows behind a sequence
    assert torch.equal(ref.f64(final), wfinal)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_short_conv_layouts_and_garbage_behind_a_sequence(dtype):
    """x as columns of a wider projection, outputs token-major; NaN and infinities behind a
    sequence reach nothing; without activation and bias."""
    g = gen_of(5)
    B, T, splits = 2, 21, [(2, 64, True), (1, 32, False)]
    C = 160
    wide = rnd(g, B, T, C + 64, dtype=dtype)
    lengths = torch.tensor([13, 21], dtype=torch.int32).cuda()
    wide[0, 13:] = float("nan")
    wide[0, 14] = float("inf")
    x = wide[..., 32:32 + C]
    w = rnd(g, C, 4)
    rows = torch.full((B, T, C), 3.0, dtype=dtype, device="cuda")
    outs = [rows[..., :128].unflatten(-1, (2, 64)).transpose(1, 2),
            rows[..., 128:].unflatten(-1, (1, 32)).transpose(1, 2)]
    got, final = drs.short_conv(x, w, splits=splits, lengths=lengths, silu=False, outs=outs, eps=EPS)
    want, wfinal, mags = ref.conv(x, w, None, splits, None, lengths, EPS, silu=False)
    for o, y, m, s in zip(got, want, mags, splits):
        within(o, y, conv_tol(dtype, y, m, s[2], s[1]))
    assert (rows[0, 13:] == 3.0).all()
    assert torch.equal(ref.f64(final), wfinal)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 4])
def test_short_conv_steps_are_the_prompt_bit_for_bit(dtype, K):
    g = gen_of(K)
    B, T, splits = 5, 12, [(3, 128, True), (1, 64, False)]
    C = 448
    x, w, bias = rnd(g, B, T, C, dtype=dtype), rnd(g, C, K), rnd(g, C)
    outs, final = drs.short_conv(x, w, bias, splits=splits)
    first, state = drs.short_conv(x[:, :4], w, bias, splits=splits)  # a prompt, then its tokens
    for t in range(4, T):
        got = drs.short_conv_step(x[:, t], w, bias, splits=splits, state=state)
        for a, b in zip(got, outs):
            assert torch.equal(a, b[:, :, t])
    for a, b in zip(first, outs):
        assert torch.equal(a, b[:, :, :4])
    assert torch.equal(state, final)
    empty, same = drs.short_conv(x[:, :0], w, bias, splits=splits, state0=state)
    assert torch.equal(same, state) and empty[0].shape == (B, 3, 0, 128)


# ------------------------------------------------------------------ selective scan

def ssm_inputs(seed, B, H, G, T, P, N, dtype, rows="head", state=True, ragged=False, dt_type=None,
               rate=None):
    g = gen_of(seed)
    dt_type = dt_type or torch.float32
    if rows == "token":
        row = rnd(g, B, T, H * P + 2 * G * N + 64, dtype=dtype)
        x = row[..., :H * P].unflatten(-1, (H, P)).transpose(1, 2)
        Bm = row[..., H * P:H * P + G * N].unflatten(-1, (G, N)).transpose(1, 2)
        Cm = row[..., H * P + G * N:H * P + 2 * G * N].unflatten(-1, (G, N)).transpose(1, 2)
        dt = rnd(g, B, T, H, std=0.5, dtype=dt_type).transpose(1, 2)
        out = torch.full((B, T, H, P), 5.0, dtype=dtype, device="cuda").transpose(1, 2)
    else:
        x, Bm, Cm = (rnd(g, B, h, T, w, dtype=dtype) for h, w in ((H, P), (G, N), (G, N)))
        dt = rnd(g, B, H, T, std=0.5, dtype=dt_type)
        out = torch.full((B, H, T, P), 5.0, dtype=dtype, device="cuda")
    rates = torch.exp(math.log(1e-3) + (math.log(0.1) - math.log(1e-3)) * torch.rand(H, generator=g))
    if rate is not None:
        rates = torch.full((H,), rate)
    lengths = None
    if ragged:
        lengths = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        lengths[0], lengths[-1] = T, 0
        lengths = lengths.cuda()
    return dict(x=x, dt=dt, A=-(1 + 15 * torch.rand(H, generator=g)).cuda(), B=Bm, C=Cm,
                D=rnd(g, H), dt_bias=torch.log(torch.expm1(rates)).cuda(),
                S0=rnd(g, B, H, P, N, std=0.3) if state else None, lengths=lengths, out=out)


def ssm_check(i, got, dtype, T, N, what=""):
    """y: the chunked kernel rounds the weights of a chunk's tokens and the state to bf16 (2^-8
    of each product, so of mag) for bf16 inputs; in fp32 T steps of 16 u (exp of the decay, its
    argument, two products) and a sum of N. S: fp32 sums (delta x goes in three bf16 parts, 24
    bits)."""
    y, S, my, mS = ref.ssm(i["x"], i["dt"], i["A"], i["B"], i["C"], i["D"], i["dt_bias"], True,
                           i["S0"], i["lengths"])
    f32 = (16 * T + N + 64) * U
    bf = dtype == torch.bfloat16
    within(got[0], y, H_OF[dtype] * y.abs() + ((2.0 ** -8 if bf else 0) + f32) * my, what + " y")
    assert (ref.f64(got[0])[torch.isnan(y)] == 5.0).all(), "rows behind a sequence"
    if got[1] is not None:
        within(got[1], S, f32 * mS, what + " S")
        # over all elements the roundings average out, far below the worst case of each: some tens
        # of u where the sums are not much larger than their results
        assert float((ref.f64(got[1]) - S).norm()) <= 2e-6 * float(S.norm()) + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P,N", [(32, 32), (64, 128), (128, 64), (128, 128), (32, 128), (64, 32)])
@pytest.mark.parametrize("T,G,rows,ragged", [(1, 1, "head", False), (2, 3, "token", False),
                                             (31, 1, "token", True), (64, 3, "head", True),
                                             (130, 1, "head", False), (300, 3, "token", True)])
def test_ssm_scan(dtype, P, N, T, G, rows, ragged):
    i = ssm_inputs(T + P, 2, 3, G, T, P, N, dtype, rows, state=T % 2 == 0, ragged=ragged,
                   dt_type=dtype if rows == "token" else None)
    ssm_check(i, drs.ssm_scan(**i), dtype, T, N)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [127, 128, 129, 255, 257, 700])
def test_ssm_scan_around_chunk_ends(dtype, T):
    i = ssm_inputs(T, 1, 2, 1, T, 64, 64, dtype)
    ssm_check(i, drs.ssm_scan(**i), dtype, T, 64)
    i["out"] = torch.full_like(i["out"], 5.0)
    ssm_check(i, drs.ssm_scan(**i, force_sequential=True), dtype, T, 64, "per token")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rate", [1e-5, 1e-3, 0.1, 3.0, 40.0])
def test_ssm_scan_decays(dtype, rate):
    """From almost no decay over the sequence to states that are gone after one token (decays
    that underflow)."""
    i = ssm_inputs(3, 2, 4, 2, 400, 32, 64, dtype, rate=rate, ragged=True)
    ssm_check(i, drs.ssm_scan(**i), dtype, 400, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rate", [30.0, 4e4])
def test_ssm_scan_tokens_that_wipe_the_state(dtype, rate):
    """Now and then a token whose decay underflows by far, among tokens that hardly decay."""
    T = 300
    i = ssm_inputs(5, 2, 2, 1, T, 64, 64, dtype)
    i["dt_bias"], i["A"] = None, torch.full_like(i["A"], -rate)
    i["dt"] = torch.full_like(i["dt"], math.log(1e-3 / rate))  # delta of 1e-3 / rate
    for t in (5, 70, 71, 128, 200, 255):
        i["dt"][:, :, t] = 30.0
    ssm_check(i, drs.ssm_scan(**i), dtype, T, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_ssm_scan_garbage_behind_a_sequence(dtype):
    i = ssm_inputs(11, 3, 2, 1, 200, 64, 64, dtype)
    i["lengths"] = torch.tensor([77, 200, 128], dtype=torch.int32).cuda()
    clean = drs.ssm_scan(**{**i, "out": i["out"].clone()})
    for t in ("x", "dt", "B", "C"):
        for b, n in ((0, 77), (2, 128)):
            i[t][b, :, n:] = float("nan")
            i[t][b, :, n + 1:n + 3] = float("inf")
    got = drs.ssm_scan(**i)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    i["lengths"] = torch.tensor([-5, 2000, 0], dtype=torch.int32).cuda()  # clamped to 0..T
    out, S = drs.ssm_scan(**{**i, "out": torch.full_like(i["out"], 5.0)})
    assert (out[0] == 5.0).all() and (out[2] == 5.0).all()
    assert torch.equal(S[0], i["S0"][0]) and torch.equal(S[2], i["S0"][2])
    assert torch.equal(S[1], clean[1][1]) and torch.equal(out[1], clean[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,T,P,N,ragged", [(1, 1, 5000, 32, 32, False), (2, 1, 4100, 64, 128, True),
                                              (1, 3, 3333, 128, 64, False)])
def test_ssm_scan_long_with_few_heads(dtype, B, H, T, P, N, ragged):
    """The scan cut into segments."""
    i = ssm_inputs(T, B, H, 1, T, P, N, dtype, "token", ragged=ragged, rate=2e-3)
    if ragged:
        i["lengths"][-1] = 3000
    ssm_check(i, drs.ssm_scan(**i), dtype, T, N)
    again = drs.ssm_scan(**{**i, "out": torch.full_like(i["out"], 5.0)})
    assert torch.equal(again[0], drs.ssm_scan(**i)[0])  # the same bits every time


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_ssm_scan_without_options_and_broadcast_views(dtype):
    """No D, no bias, no softplus, no state wanted; B and C repeated over the heads, x over the
    batch, by views that repeat memory."""
    i = ssm_inputs(8, 2, 4, 1, 150, 32, 64, dtype, state=False)
    i["dt"] = i["dt"].abs() * 0.1
    i["B"], i["C"] = i["B"].expand(2, 4, 150, 64), i["C"].expand(2, 4, 150, 64)
    i["x"] = i["x"][:1].expand(2, 4, 150, 32)
    i["D"] = i["dt_bias"] = None
    i["dt"] = i["dt"][:, :, :1].expand(2, 4, 150)
    out, S = drs.ssm_scan(**i, dt_softplus=False, want_state=False)
    assert S is None
    y, _, my, _ = ref.ssm(i["x"], i["dt"], i["A"], i["B"], i["C"], None, None, False, None, None)
    bf = dtype == torch.bfloat16
    within(out, y, H_OF[dtype] * y.abs() + ((2.0 ** -8 if bf else 0) + 3000 * U) * my)


@pytest.mark.gpu
def test_ssm_scan_empty():
    i = ssm_inputs(1, 2, 2, 1, 4, 32, 32, torch.bfloat16)
    e = {**i, **{k: i[k][:, :, :0] for k in ("x", "dt", "B", "C", "out")}}
    out, S = drs.ssm_scan(**e)
    assert out.shape == (2, 2, 0, 32) and torch.equal(S, i["S0"])
    _, S = drs.ssm_scan(**{**e, "S0": None})
    assert (S == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,G,P,N", [(1, 1, 1, 32, 32), (3, 6, 2, 64, 128), (2, 5, 1, 128, 64),
                                       (7, 4, 4, 32, 128), (2, 2, 1, 128, 32)])
def test_ssm_step(dtype, B, H, G, P, N):
    i = ssm_inputs(B + N, B, H, G, 1, P, N, dtype, "token", dt_type=dtype)
    S = i["S0"].clone()
    out = drs.ssm_step(i["x"][:, :, 0], i["dt"][:, :, 0], i["A"], i["B"][:, :, 0], i["C"][:, :, 0],
                       i["D"], i["dt_bias"], S=S)
    y, Sr, my, mS = ref.ssm(i["x"], i["dt"], i["A"], i["B"], i["C"], i["D"], i["dt_bias"], True,
                            i["S0"], None)
    within(out, y[:, :, 0], H_OF[dtype] * y[:, :, 0].abs() + (N + 80) * U * my[:, :, 0])
    within(S, Sr, 80 * U * mS)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_ssm_steps_go_on_from_a_prompt(dtype):
    i = ssm_inputs(21, 2, 4, 2, 140, 64, 64, dtype)
    out, S = drs.ssm_scan(**{**{k: v[:, :, :133] if k in ("x", "dt", "B", "C") else v
                                for k, v in i.items()}, "out": None})
    outs = [out]
    for t in range(133, 140):
        outs.append(drs.ssm_step(i["x"][:, :, t], i["dt"][:, :, t], i["A"], i["B"][:, :, t],
                                 i["C"][:, :, t], i["D"], i["dt_bias"], S=S)[:, :, None])
    ssm_check(i, (torch.cat(outs, 2), S), dtype, 140, 64)


# ------------------------------------------------------------------ norms

def norm_tol(dtype, want, W):
    """Squares and their mean: (W + 8) u of the mean, half of it in the root; five products; an
    activation off by up to 100 u (its exponential's argument). All relative to the output."""
    return (H_OF[dtype] + (W + 150) * U) * want.abs() + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,T,d,heads", [(1, 1, 1, 32, 1), (2, 3, 5, 64, 1), (2, 6, 3, 32, 3),
                                           (3, 4, 7, 128, 2), (2, 8, 9, 128, 8), (1, 24, 3, 128, 24),
                                           (1, 64, 2, 128, 64), (2, 5, 33, 128, 1), (1, 40, 1, 64, 40)])
@pytest.mark.parametrize("act,first,shared", [("silu", False, True), ("silu", True, False),
                                              ("sigmoid", False, False)])
def test_gated_norm(dtype, B, H, T, d, heads, act, first, shared):
    g = gen_of(H * d + T)
    y, gate = rnd(g, B, H, T, d, dtype=dtype), rnd(g, B, T, H * d, std=2.0, dtype=dtype)
    w = rnd(g, d if shared else H * d)
    out = drs.gated_norm(y, gate, w, norm_heads=heads, act=act, gate_first=first, eps=EPS)
    want = ref.gated(y, gate, w, heads, act, first, EPS)
    within(out, want, norm_tol(dtype, want, heads * d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_norm_layouts(dtype):
    """y token-major, gate as columns of a projection, in place of the gate; no gate; a row of
    zeros; values at the ends of the type's range of exponents."""
    g = gen_of(2)
    B, H, T, d = 2, 4, 6, 64
    y = rnd(g, B, T, H, d, dtype=dtype)
    y[0, 0] = 0
    y[1, 1] *= 1e15
    y[1, 2] *= 1e-18
    w = rnd(g, H * d)
    wide = rnd(g, B, T, H * d + 64, dtype=dtype)
    gate = wide[..., 32:32 + H * d]
    gate[0, 1, :8] = -200.0
    gate[0, 1, 8:16] = 200.0
    want = ref.gated(y.transpose(1, 2), gate, w, H, "silu", False, EPS)
    out = drs.gated_norm(y.transpose(1, 2), gate, w, norm_heads=H, eps=EPS, out=gate)
    within(out, want, norm_tol(dtype, want, H * d))
    want = ref.gated(y.transpose(1, 2), None, w, 2, "silu", False, EPS)
    out = drs.gated_norm(y.transpose(1, 2), None, w, norm_heads=2, eps=EPS)
    within(out, want, norm_tol(dtype, want, 2 * d))
    assert (out[0, 0] == 0).all()
    assert drs.gated_norm(y.transpose(1, 2)[:, :, :0], None, w).shape == (B, 0, H * d)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wide", [(torch.bfloat16, False), (torch.bfloat16, True),
                                        (torch.float32, False)])
@pytest.mark.parametrize("rows,D", [(1, 8), (5, 32), (7, 72), (9, 128), (3, 520), (4, 1024),
                                    (3, 2056), (130, 256), (2, 8192), (1, 4104)])
@pytest.mark.parametrize("post,vector,first", [(False, False, False), (True, True, False),
                                               (True, False, True)])
def test_block_norm(dtype, wide, rows, D, post, vector, first):
    g = gen_of(rows * D)
    rt = torch.float32 if wide else dtype
    x, w = rnd(g, rows, D, dtype=dtype), rnd(g, D)
    res = None if first else rnd(g, rows, D, std=3.0, dtype=rt)
    pw = rnd(g, D) if post else None
    scale = rnd(g, D) if vector else 0.37
    out, r = drs.block_norm(x, w, residual=res, scale=scale, post_weight=pw, residual_dtype=rt,
                            eps=EPS)
    want, wr, mag = ref.block(x, w, res, scale, pw, EPS)
    assert r.dtype == rt and out.dtype == dtype
    # r: the post norm's (D + 20) u of z; out: an error of r moves it by that, times the weight,
    # over the row's root mean square, and the mean by (D + 8) u
    within(r, wr, H_OF[rt] * wr.abs() + (D + 20) * U * mag)
    rms = torch.sqrt((wr * wr).mean(-1, keepdim=True) + EPS)
    tol = H_OF[dtype] * want.abs() + (D + 40) * U * (2 * want.abs() + mag / rms * ref.f64(w).abs())
    within(out, want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_block_norm_in_place_and_layouts(dtype):
    g = gen_of(9)
    x, w = rnd(g, 2, 3, 640, dtype=dtype), rnd(g, 256)
    cols = x[..., 64:320]
    res = rnd(g, 2, 3, 256, dtype=dtype)
    want_out, want_r = drs.block_norm(cols.contiguous(), w, residual=res, scale=0.5)
    got_out, got_r = drs.block_norm(cols, w, residual=res, scale=0.5, residual_out=res)
    assert got_r.data_ptr() == res.data_ptr()
    assert torch.equal(got_out, want_out) and torch.equal(got_r, want_r)
    y = cols.contiguous()
    out, _ = drs.block_norm(y, w, out=y)
    assert torch.equal(out, drs.block_norm(cols, w)[0])
    assert drs.block_norm(x[:0], w.new_ones(640))[0].shape == (0, 3, 640)


# ------------------------------------------------------------------ together

def layer(p, u, r, state=None, lengths=None):
    """A state space layer on rows u [B,T,E] with residual stream r: norm, projection, short
    convolution, scan, gated norm, projection. Returns (block output, r, state)."""
    B, T, E = u.shape
    H, P, G, N = p["H"], p["P"], p["G"], p["N"]
    n, r = drs.block_norm(u, p["norm"], residual=r, scale=0.5)
    z, xbc, dt = (n @ p["w_in"]).split([H * P, H * P + 2 * G * N, 64], dim=-1)
    splits = [(H, P, False), (G, N, False), (G, N, False)]
    conv_state, S = state if state is not None else (None, None)
    if T == 1 and state is not None:
        x, Bm, Cm = drs.short_conv_step(xbc[:, 0], p["conv"], p["conv_b"], splits=splits,
                                        state=conv_state)
        y = drs.ssm_step(x, dt[:, 0, :H], p["A"], Bm, Cm, p["D"], p["dt_bias"], S=S)[:, :, None]
    else:
        (x, Bm, Cm), conv_state = drs.short_conv(xbc, p["conv"], p["conv_b"], splits=splits,
                                                 state0=conv_state, lengths=lengths)
        y, S = drs.ssm_scan(x, dt[..., :H].transpose(1, 2), p["A"], Bm, Cm, p["D"], p["dt_bias"],
                            S0=S, lengths=lengths)
    o = drs.gated_norm(y, z, p["gnorm"], norm_heads=H)
    return o @ p["w_out"], r, (conv_state, S)


def layer_params(g, dtype, H=4, P=64, G=2, N=64, E=128):
    C = H * P + 2 * G * N
    return dict(H=H, P=P, G=G, N=N, norm=rnd(g, E), w_in=rnd(g, E, H * P + C + 64, std=E ** -0.5,
                                                              dtype=dtype),
                conv=rnd(g, C, 4, std=0.5), conv_b=rnd(g, C, std=0.1),
                A=-(1 + 15 * torch.rand(H, generator=g)).cuda(), D=rnd(g, H),
                dt_bias=torch.full((H,), -4.0).cuda(), gnorm=rnd(g, H * P),
                w_out=rnd(g, H * P, E, std=(H * P) ** -0.5, dtype=dtype))


@pytest.mark.gpu
def test_layer_prompt_then_tokens_is_the_longer_prompt():
    """fp32: a prompt of 150 and 10 tokens one at a time against a prompt of 160. Each is off the
    exact result by the operators' roundings alone; 1e-4 of the largest value is 1700 u, a tenth
    of the worst case of a 160 token scan (16 T u of the magnitudes) through the layer."""
    g = gen_of(4)
    p = layer_params(g, torch.float32)
    B, T, n = 2, 160, 150
    u, r = rnd(g, B, T, 128), rnd(g, B, T, 128)
    want, wr, wstate = layer(p, u, r)
    y, r1, state = layer(p, u[:, :n].contiguous(), r[:, :n].contiguous())
    rows = [y]
    for t in range(n, T):
        y, _, state = layer(p, u[:, t:t + 1].contiguous(), r[:, t:t + 1].contiguous(), state)
        rows.append(y)
    got = torch.cat(rows, 1)
    assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())
    assert float((state[1] - wstate[1]).abs().max()) <= 1e-4 * float(wstate[1].abs().max())
    assert float((state[0] - wstate[0]).abs().max()) <= 1e-4 * float(wstate[0].abs().max())


@pytest.mark.gpu
def test_layer_padded_batch_is_each_sequence_alone():
    g = gen_of(6)
    p = layer_params(g, torch.bfloat16)
    lengths = [130, 0, 61]
    u = rnd(g, 3, 140, 128, dtype=torch.bfloat16)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    x = rnd(g, 3, 140, 512, dtype=torch.bfloat16)
    splits = [(4, 64, False), (2, 64, False), (2, 64, False)]
    dt = rnd(g, 3, 4, 140)

    def run(x, dt, n):
        (q, b, c), cs = drs.short_conv(x, p["conv"], p["conv_b"], splits=splits, lengths=n)
        y, S = drs.ssm_scan(q, dt, p["A"], b, c, p["D"], p["dt_bias"], lengths=n)
        return y, cs, S

    y, cs, S = run(x, dt, n)
    for b, k in enumerate(lengths):
        y1, cs1, S1 = run(x[b:b + 1, :k].contiguous(), dt[b:b + 1, :, :k].contiguous(), None)
        assert torch.equal(y[b:b + 1, :, :k], y1)
        assert torch.equal(cs[b:b + 1], cs1) and torch.equal(S[b:b + 1], S1)


@pytest.mark.gpu
def test_short_conv_feeds_the_delta_rule_scan(oracle):
    """q, k (L2-normalised) and v from the convolution, head-major, into Gated DeltaNet, then the
    gated norm per head: the scan against the oracle on the same q, k, v (its bf16 tolerance),
    unit keys to bf16's rounding."""
    g = gen_of(12)
    B, H, T, d = 2, 2, 150, 128
    x = rnd(g, B, T, 3 * H * d, dtype=torch.bfloat16)
    splits = [(H, d, True), (H, d, True), (H, d, False)]
    (q, k, v), _ = drs.short_conv(x, rnd(g, 3 * H * d, 4, std=0.5), splits=splits)
    beta, gate = torch.rand(B, H, T, generator=g).cuda(), (0.9 + 0.1 * torch.rand(B, H, T, generator=g)).cuda()
    out, S = drs.scan(q, k, v, beta, gate, mode="gdn")
    torch.cuda.synchronize()
    assert drs.poll_error() == drs.DR_OK
    nrm = ref.f64(k).norm(dim=-1)
    assert float((nrm - 1).abs().max()) <= 2.0 ** -8 + 1e-4  # eps beside the sum of squares
    want, wS = oracle.dr_scan(*(t.double().cpu().numpy() for t in (q, k, v, beta, gate)), None, drs.DR_GDN)
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2e-2 * np.abs(want).max()
    y = drs.gated_norm(out, x[..., :H * d], rnd(g, d))
    assert y.shape == (B, T, H * d) and torch.isfinite(y).all()


# ------------------------------------------------------------------ streams, graphs, sizes

@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,P,N,ragged,runs", [(8, 16, 1024, 128, 128, False, 30),
                                                   (1, 16, 16384, 64, 128, False, 30),
                                                   (2, 4, 4096, 64, 64, False, 60),
                                                   (4, 16, 700, 64, 64, True, 100),
                                                   (3, 40, 2000, 32, 32, True, 60)])
def test_ssm_scan_gives_the_same_bits_every_time(B, H, T, P, N, ragged, runs):
    """The chunked kernel's roles hand over to one another some thirty times a chunk: one that
    went on too early would read what is not there yet, now and then. Every run equal, bit for
    bit, over thousands of chunks, the first against a scan without hand-overs (per token, its
    roundings apart from the chunked kernel's: 2^-7 of the largest output, 2^-16 of the state)."""
    i = ssm_inputs(T + N, B, H, 1, T, P, N, torch.bfloat16, "token", ragged=ragged)
    want = drs.ssm_scan(**{**i, "out": torch.zeros_like(i["out"])}, force_sequential=True)
    out, S = (t.clone() for t in drs.ssm_scan(**{**i, "out": torch.zeros_like(i["out"])}))
    assert float((out.float() - want[0].float()).abs().max()) <= 2.0 ** -7 * float(want[0].float().abs().max())
    assert float((S - want[1]).abs().max()) <= 2.0 ** -16 * float(want[1].abs().max())
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(runs):
        a, b = drs.ssm_scan(**{**i, "out": torch.zeros_like(i["out"])})
        bad += (a != out).any().long() + (b != S).any().long()
    assert int(bad) == 0


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two segmented scans (each with scratch) and two layers' worth of calls on two streams."""
    a, b = (ssm_inputs(s, 1, 2, 1, 6000, 64, 64, t, rate=1e-3)
            for s, t in ((1, torch.bfloat16), (2, torch.float32)))
    want = [tuple(t.clone() for t in drs.ssm_scan(**i)) for i in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k, i in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k].append(drs.ssm_scan(**{**i, "out": torch.empty_like(i["out"])}))
    torch.cuda.synchronize()
    for k in range(2):
        for out, S in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(S, want[k][1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_captured_and_replayed(dtype):
    """Two graphs over the operators, the segmented scan's scratch among them, replayed in turn
    and on two streams, on inputs that changed since the capture."""
    g = gen_of(31)
    sets = [ssm_inputs(40 + k, 1, 1, 1, 3000, 64, 64, dtype, rate=1e-3) for k in range(2)]
    w, conv_w = rnd(g, 64), rnd(g, 64, 4)
    xs = [rnd(g, 1, 3000, 64, dtype=dtype) for _ in range(2)]

    def run(k):
        (x,), _ = drs.short_conv(xs[k], conv_w, splits=[(1, 64)])
        y, S = drs.ssm_scan(**{**sets[k], "x": x, "out": None})
        n = drs.gated_norm(y, xs[k], w)
        return drs.block_norm(n, w, residual=xs[k])[0], S

    run(0), run(1)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run(k))
        graphs.append(gr)
    for k in range(2):
        xs[k].copy_(rnd(g, 1, 3000, 64, dtype=dtype))
    want = [tuple(t.clone() for t in run(k)) for k in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(outs[k], want[k]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_offsets_beyond_int32():
    """Tensors of more than 2^31 elements: the last sequence of a batch of two far apart."""
    T, H, P, N = 70, 2, 64, 64
    step = (1 << 31) + 4096
    big = torch.empty(step + T * 512 + 8192, dtype=torch.bfloat16, device="cuda")
    g = gen_of(13)
    i = ssm_inputs(50, 2, H, 1, T, P, N, torch.bfloat16)

    def far(t, at):
        v = torch.as_strided(big, t.shape, (step, *t.stride()[1:]), at)
        v.copy_(t)
        return v

    x = far(i["x"], 0)
    Bm, Cm = far(i["B"], H * T * P), far(i["C"], H * T * P + T * N)
    out = far(i["out"], H * T * P + 2 * T * N)
    want = drs.ssm_scan(**{**i, "out": None})
    got = drs.ssm_scan(**{**i, "x": x, "B": Bm, "C": Cm, "out": out})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rows = torch.as_strided(big, (2, T, 128), (step, 128, 1), 0)
    rows.copy_(rnd(g, 2, T, 128, dtype=torch.bfloat16))
    w = rnd(g, 128, 4)
    a, sa = drs.short_conv(rows, w)
    b, sb = drs.short_conv(rows.contiguous(), w)
    assert torch.equal(a[0], b[0]) and torch.equal(sa, sb)
    y = rows.unflatten(-1, (2, 64)).transpose(1, 2)
    assert torch.equal(drs.gated_norm(y, rows, w[:, 0].contiguous()),
                       drs.gated_norm(y.contiguous(), rows.contiguous(), w[:, 0].contiguous()))
