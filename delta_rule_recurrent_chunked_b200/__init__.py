"""B200-native forward recurrent-memory scan of delta-rule linear attention.

Thin Python binding over the C-ABI library ``libdrscan.so`` (declared in
``include/drscan.h``). This module only marshals arguments: it checks tensor dtypes,
shapes and devices, passes raw device pointers and the current CUDA stream, and raises
on a non-zero status. Every step of the scan runs in the library's CUDA kernels; there
is no CPU fallback, and a missing library is an error.

    out, S_final = scan(q, k, v, beta, gate, S0=None, mode="gdn")
    out, S_final, u = scan_ex(q, k, v, beta, gate, S0=None, mode="gdn2", erase=b, write=w)
    out, S_final, A_final = vla_scan(q, k, v, u, S0=None, A0=None, lambda0=1.0)
    out = decode_step(q, k, v, beta, gate, S, mode="gdn")     # S updated in place

Around a scan: short_conv / short_conv_step (the causal convolution that makes its inputs),
ssm_scan / ssm_step (the selective state space scan), gated_norm (its output with the gate) and
block_norm (residual and norms between blocks).
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdrscan.so")

DR_LINEAR, DR_DELTANET, DR_GDN, DR_KDA, DR_GDN2 = 0, 1, 2, 3, 4
DR_IN_BF16 = 0x100
DR_FORCE_SEQUENTIAL = 0x200
DR_CHAINED = 0x400
DR_OK, DR_ERR_INVALID_ARG, DR_ERR_UNSUPPORTED, DR_ERR_CUDA, DR_ERR_TIMEOUT, DR_ERR_DEVICE_BOUNDS = (
    0, -1, -2, -3, -4, -5)
DR_ERR_GATE_RANGE = -6
DR_ERR_NOT_SPD = -7
DR_ERR_SCRATCH_LIMIT = -8
VLA_NOALLOC_MAX_FLOATS = 16777216
MODES = {"linear": DR_LINEAR, "deltanet": DR_DELTANET, "gdn": DR_GDN, "kda": DR_KDA,
         "gdn2": DR_GDN2}

CONV_SILU = 0x1000
SSM_DT_SOFTPLUS, SSM_DT_BF16 = 0x1000, 0x2000
NORM_SIGMOID, NORM_GATE_FIRST, NORM_SHARED_WEIGHT = 0x1000, 0x2000, 0x4000
NORM_RESIDUAL_F32 = 0x1000


class DrView(ctypes.Structure):
    """dr_view: a pointer and the element strides of batch, head and token."""
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong),
                ("st", ctypes.c_longlong)]


class ConvSplit(ctypes.Structure):
    """conv_split: where heads x dim channels of a short convolution go."""
    _fields_ = [("out", DrView), ("heads", ctypes.c_int), ("dim", ctypes.c_int),
                ("normalise", ctypes.c_int)]


# Every function the C ABI exports, with its ctypes signature.
_VP, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_PV = _PS = _VP  # addresses of dr_view and conv_split structs
_LL = ctypes.c_longlong
SIGNATURES = {
    "dr_scan_fwd": ([_VP] * 8 + [_I] * 6 + [_VP], _I),
    "dr_scan_fwd_ex": ([_VP] * 11 + [_I] * 6 + [_VP], _I),
    "dr_decode_step": ([_VP] * 7 + [_I] * 5 + [_VP], _I),
    "dr_decode_step_ex": ([_VP] * 10 + [_I] * 5 + [_VP], _I),
    "vla_scan_fwd": ([_VP] * 6 + [_F] + [_VP] * 3 + [_I] * 4 + [_VP], _I),
    "vla_scan_fwd_ex": ([_VP] * 7 + [_F] + [_VP] * 4 + [_I] * 5 + [_VP], _I),
    "vla_scan_fwd_noalloc": ([_VP] * 7 + [_F] + [_VP] * 4 + [_I] * 5 + [_VP], _I),
    "loglinear_scan_fwd": ([_VP] * 5 + [_I] * 7 + [_VP], _I),
    "short_conv_fwd": ([_PV] + [_VP] * 4 + [_PS, _I, _VP, _F] + [_I] * 5 + [_VP], _I),
    "short_conv_step": ([_PV] + [_VP] * 3 + [_PS, _I, _F] + [_I] * 4 + [_VP], _I),
    "ssm_scan_fwd": ([_PV, _PV, _VP, _PV, _PV] + [_VP] * 4 + [_PV, _VP] + [_I] * 7 + [_VP], _I),
    "ssm_step": ([_PV, _PV, _VP, _PV, _PV] + [_VP] * 3 + [_PV] + [_I] * 6 + [_VP], _I),
    "gated_norm_fwd": ([_PV, _PV, _VP, _PV, _F] + [_I] * 6 + [_VP], _I),
    "block_norm_fwd": ([_VP, _LL] + [_VP] * 4 + [_F, _VP, _VP, _F, _LL, _I, _I, _VP], _I),
    "dr_status_string": ([_I], ctypes.c_char_p),
    "dr_poll_error": ([_VP], _I),
    "dr_debug_timeout_probe": ([_I, _VP], _I),
    "dr_debug_wait_limit": ([_LL], _I),
    "dr_chunked_plan": ([_I, ctypes.c_longlong, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "dr_chunked_plan_ex": ([_I, ctypes.c_longlong, _I, _I, _I, ctypes.POINTER(_I),
                            ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "dr_segment_counters": ([ctypes.POINTER(ctypes.c_ulonglong)] * 2, _I),
    "dr_version": ([], _I),
}

_lib = None


class DrScanError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def lib():
    """Load libdrscan.so (built in-tree). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m delta_rule_recurrent_chunked_b200.build` (nvcc, sm_100a)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (argtypes, restype) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().dr_status_string(int(status)).decode()


def _stream_handle(device):
    import torch

    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, shape, dtype, device):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def scan(q, k, v, beta=None, gate=None, S0=None, mode="gdn", want_state=True,
         force_sequential=False, out=None, S_final=None, chained=False):
    """Delta-rule scan on the GPU. q, k: [B,H,T,dk]; v: [B,H,T,dv] (bf16 or fp32, same
    dtype); beta: [B,H,T] fp32; gate: alpha values, [B,H,T] (gdn) or [B,H,T,dk] (kda) fp32;
    S0: [B,H,dv,dk] fp32 or None. chained=True keeps Gated DeltaNet off the segmented scan
    (DR_CHAINED). Returns (out like v, S_final fp32 or None)."""
    import torch

    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q/k/v must be bf16 or fp32")
    _check(q, "q", (B, H, T, dk), q.dtype, dev)
    _check(k, "k", (B, H, T, dk), q.dtype, dev)
    _check(v, "v", (B, H, T, dv), q.dtype, dev)
    if variant != DR_LINEAR:
        _check(beta, "beta", (B, H, T), torch.float32, dev)
    else:
        beta = None
    if variant == DR_GDN:
        _check(gate, "gate", (B, H, T), torch.float32, dev)
    elif variant == DR_KDA:
        _check(gate, "gate", (B, H, T, dk), torch.float32, dev)
    else:
        gate = None
    if S0 is not None:
        _check(S0, "S0", (B, H, dv, dk), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, device=dev)
    _check(out, "out", (B, H, T, dv), q.dtype, dev)
    if want_state and S_final is None:
        S_final = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_final is not None:
        _check(S_final, "S_final", (B, H, dv, dk), torch.float32, dev)
    flags = variant | (DR_IN_BF16 if q.dtype == torch.bfloat16 else 0)
    if force_sequential:
        flags |= DR_FORCE_SEQUENTIAL
    if chained:
        flags |= DR_CHAINED
    rc = lib().dr_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(gate), _ptr(S0), _ptr(out),
                           _ptr(S_final), B, H, T, dk, dv, flags, _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "dr_scan_fwd")
    return out, S_final


def scan_ex(q, k, v, beta=None, gate=None, S0=None, mode="gdn", erase=None, write=None,
            want_state=True, want_u=True, force_sequential=False, out=None, S_final=None,
            u_out=None, chained=False):
    """scan() with Gated DeltaNet-2 and the per-token write values, through dr_scan_fwd_ex.
    mode "gdn2" takes gate [B,H,T] (alpha), erase [B,H,T,dk] (b) and write [B,H,T,dv] (w),
    fp32. Returns (out, S_final or None, u or None): u [B,H,T,dv] like v holds the write
    values beta_t r_t."""
    import torch

    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q/k/v must be bf16 or fp32")
    _check(q, "q", (B, H, T, dk), q.dtype, dev)
    _check(k, "k", (B, H, T, dk), q.dtype, dev)
    _check(v, "v", (B, H, T, dv), q.dtype, dev)
    if variant != DR_LINEAR:
        _check(beta, "beta", (B, H, T), torch.float32, dev)
    else:
        beta = None
    if variant in (DR_GDN, DR_GDN2):
        _check(gate, "gate", (B, H, T), torch.float32, dev)
    elif variant == DR_KDA:
        _check(gate, "gate", (B, H, T, dk), torch.float32, dev)
    else:
        gate = None
    if variant == DR_GDN2:
        _check(erase, "erase", (B, H, T, dk), torch.float32, dev)
        _check(write, "write", (B, H, T, dv), torch.float32, dev)
    else:
        erase = write = None
    if S0 is not None:
        _check(S0, "S0", (B, H, dv, dk), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, device=dev)
    _check(out, "out", (B, H, T, dv), q.dtype, dev)
    if want_state and S_final is None:
        S_final = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_final is not None:
        _check(S_final, "S_final", (B, H, dv, dk), torch.float32, dev)
    if want_u and u_out is None:
        u_out = torch.empty((B, H, T, dv), dtype=q.dtype, device=dev)
    if u_out is not None:
        _check(u_out, "u_out", (B, H, T, dv), q.dtype, dev)
    flags = variant | (DR_IN_BF16 if q.dtype == torch.bfloat16 else 0)
    if force_sequential:
        flags |= DR_FORCE_SEQUENTIAL
    if chained:
        flags |= DR_CHAINED
    rc = lib().dr_scan_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(gate), _ptr(erase),
                              _ptr(write), _ptr(S0), _ptr(out), _ptr(S_final), _ptr(u_out),
                              B, H, T, dk, dv, flags, _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "dr_scan_fwd_ex")
    return out, S_final, u_out


def decode_step_ex(q, k, v, beta=None, gate=None, S=None, mode="gdn", erase=None, write=None,
                   want_u=True, out=None, u_out=None):
    """decode_step() with Gated DeltaNet-2 (erase [B,H,dk], write [B,H,dv]) and the write
    value u [B,H,dv], through dr_decode_step_ex. Returns (out, u or None)."""
    import torch

    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q/k/v must be bf16 or fp32")
    _check(q, "q", (B, H, dk), q.dtype, dev)
    _check(k, "k", (B, H, dk), q.dtype, dev)
    _check(v, "v", (B, H, dv), q.dtype, dev)
    if variant != DR_LINEAR:
        _check(beta, "beta", (B, H), torch.float32, dev)
    else:
        beta = None
    if variant in (DR_GDN, DR_GDN2):
        _check(gate, "gate", (B, H), torch.float32, dev)
    elif variant == DR_KDA:
        _check(gate, "gate", (B, H, dk), torch.float32, dev)
    else:
        gate = None
    if variant == DR_GDN2:
        _check(erase, "erase", (B, H, dk), torch.float32, dev)
        _check(write, "write", (B, H, dv), torch.float32, dev)
    else:
        erase = write = None
    if S is None:
        raise ValueError("decode_step_ex needs the state S (updated in place)")
    _check(S, "S", (B, H, dv, dk), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    _check(out, "out", (B, H, dv), q.dtype, dev)
    if want_u and u_out is None:
        u_out = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    if u_out is not None:
        _check(u_out, "u_out", (B, H, dv), q.dtype, dev)
    flags = variant | (DR_IN_BF16 if q.dtype == torch.bfloat16 else 0)
    rc = lib().dr_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(gate), _ptr(erase),
                                 _ptr(write), _ptr(S), _ptr(out), _ptr(u_out), B, H, dk, dv,
                                 flags, _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "dr_decode_step_ex")
    return out, u_out


def decode_step(q, k, v, beta=None, gate=None, S=None, mode="gdn", out=None):
    """One token of the delta-rule recurrence on a resident state, on the GPU.
    q, k: [B,H,dk]; v: [B,H,dv] (bf16 or fp32, same dtype); beta: [B,H] fp32; gate:
    alpha values, [B,H] (gdn) or [B,H,dk] (kda) fp32; S: [B,H,dv,dk] fp32, updated in
    place. Returns out [B,H,dv] like v."""
    import torch

    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q/k/v must be bf16 or fp32")
    _check(q, "q", (B, H, dk), q.dtype, dev)
    _check(k, "k", (B, H, dk), q.dtype, dev)
    _check(v, "v", (B, H, dv), q.dtype, dev)
    if variant != DR_LINEAR:
        _check(beta, "beta", (B, H), torch.float32, dev)
    else:
        beta = None
    if variant == DR_GDN:
        _check(gate, "gate", (B, H), torch.float32, dev)
    elif variant == DR_KDA:
        _check(gate, "gate", (B, H, dk), torch.float32, dev)
    else:
        gate = None
    if S is None:
        raise ValueError("decode_step needs the state S (updated in place)")
    _check(S, "S", (B, H, dv, dk), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    _check(out, "out", (B, H, dv), q.dtype, dev)
    flags = variant | (DR_IN_BF16 if q.dtype == torch.bfloat16 else 0)
    rc = lib().dr_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(gate), _ptr(S),
                              _ptr(out), B, H, dk, dv, flags, _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "dr_decode_step")
    return out


def vla_scan(q, k, v, u, S0=None, A0=None, lambda0=1.0, want_state=True, out=None,
             sequential=False, two_kernel=False):
    """VLA Sherman-Morrison scan on the GPU (fp32). q, k, v, u: [B,H,T,d];
    S0, A0: [B,H,d,d] or None. Returns (out, S_final, A_final). The chunked scan runs as one
    fused cluster kernel by default; two_kernel=True runs its two phases as separate kernels
    (with pool scratch), sequential=True the per-token kernel."""
    import torch

    B, H, T, d = q.shape
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("u", u)):
        _check(t, name, (B, H, T, d), torch.float32, dev)
    for name, t in (("S0", S0), ("A0", A0)):
        if t is not None:
            _check(t, name, (B, H, d, d), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, T, d), dtype=torch.float32, device=dev)
    _check(out, "out", (B, H, T, d), torch.float32, dev)
    Sf = torch.empty((B, H, d, d), dtype=torch.float32, device=dev) if want_state else None
    Af = torch.empty((B, H, d, d), dtype=torch.float32, device=dev) if want_state else None
    flags = _vla_path_flags(sequential, two_kernel)
    rc = lib().vla_scan_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(S0), _ptr(A0), None,
                               float(lambda0), _ptr(out), _ptr(Sf), _ptr(Af), None, B, H, T,
                               d, flags, _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "vla_scan_fwd_ex")
    return out, Sf, Af


VLA_RATIO_READOUT = 0x1
VLA_SEQUENTIAL = 0x2
VLA_TWO_KERNEL = 0x4


def _vla_path_flags(sequential: bool, two_kernel: bool) -> int:
    return (VLA_SEQUENTIAL if sequential else 0) | (VLA_TWO_KERNEL if two_kernel else 0)


def vla_scan_ratio(q, k, v, u, S0=None, A0=None, n0=None, lambda0=1.0, want_state=True,
                   out=None, sequential=False, two_kernel=False):
    """VLA scan with the ratio readout o_t = S_t q_t / (n_t q_t) (fp32), through
    vla_scan_fwd_ex. q: [B,H,T,d] feature-mapped queries (phi(q)); k: unit-norm
    feature-mapped keys; n0: [B,H,d] or None. Returns (out, S_final, A_final, n_final).
    two_kernel / sequential select the other paths, as in vla_scan."""
    import torch

    B, H, T, d = q.shape
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("u", u)):
        _check(t, name, (B, H, T, d), torch.float32, dev)
    for name, t in (("S0", S0), ("A0", A0)):
        if t is not None:
            _check(t, name, (B, H, d, d), torch.float32, dev)
    if n0 is not None:
        _check(n0, "n0", (B, H, d), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, T, d), dtype=torch.float32, device=dev)
    _check(out, "out", (B, H, T, d), torch.float32, dev)
    Sf = torch.empty((B, H, d, d), dtype=torch.float32, device=dev) if want_state else None
    Af = torch.empty((B, H, d, d), dtype=torch.float32, device=dev) if want_state else None
    nf = torch.empty((B, H, d), dtype=torch.float32, device=dev) if want_state else None
    rc = lib().vla_scan_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(S0), _ptr(A0), _ptr(n0),
                               float(lambda0), _ptr(out), _ptr(Sf), _ptr(Af), _ptr(nf), B, H, T,
                               d, VLA_RATIO_READOUT | _vla_path_flags(sequential, two_kernel),
                               _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "vla_scan_fwd_ex")
    return out, Sf, Af, nf


def loglinear_levels(T: int) -> int:
    """Level weights a log-linear scan of T tokens needs: level 0 plus one per bit of T - 1."""
    return max(1, int(T - 1).bit_length() + 1)


def loglinear_scan(q, k, v, lam, out=None):
    """Log-linear attention over a Fenwick hierarchy of memories, through loglinear_scan_fwd.
    q, k: [B,H,T,dk] bf16; v: [B,H,T,dv] bf16; lam: [B,H,T,L] fp32 level weights
    (L >= loglinear_levels(T)). Returns out [B,H,T,dv] bf16."""
    import torch

    B, H, T, dk = q.shape
    dv = v.shape[-1]
    L = lam.shape[-1]
    dev = q.device
    _check(q, "q", (B, H, T, dk), torch.bfloat16, dev)
    _check(k, "k", (B, H, T, dk), torch.bfloat16, dev)
    _check(v, "v", (B, H, T, dv), torch.bfloat16, dev)
    _check(lam, "lambda", (B, H, T, L), torch.float32, dev)
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=torch.bfloat16, device=dev)
    _check(out, "out", (B, H, T, dv), torch.bfloat16, dev)
    rc = lib().loglinear_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(out), B, H, T, dk,
                                  dv, L, DR_IN_BF16, _stream_handle(dev))
    if rc != DR_OK:
        raise DrScanError(rc, "loglinear_scan_fwd")
    return out


def poll_error(device=None) -> int:
    """Synchronise the current stream and return/clear the device status word."""
    import torch

    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    return int(lib().dr_poll_error(_stream_handle(dev)))


def chunked_plan(mode, BH: int, dk: int, dv: int) -> tuple:
    """(value channels per chain CTA, prep CTAs per head; 0 = unsplit) that dr_scan_fwd uses
    for bf16 inputs on the current device, or None when the chunked kernel does not apply."""
    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    bv, nprep = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().dr_chunked_plan(variant | DR_IN_BF16, int(BH), int(dk), int(dv),
                               ctypes.byref(bv), ctypes.byref(nprep))
    if st == DR_ERR_UNSUPPORTED:
        return None
    if st != DR_OK:
        raise DrScanError(st, "dr_chunked_plan")
    return bv.value, nprep.value


def chunked_plan_ex(mode, BH: int, T: int, dk: int, dv: int, chained=False) -> tuple:
    """(value channels per chain CTA, prep CTAs per head, segments per head) for bf16 inputs
    of length T on the current device, or None when the chunked kernel does not apply. With
    more than one segment the first two describe the launches over B*H*segments sequences."""
    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    bv, nprep, nseg = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    flags = variant | DR_IN_BF16 | (DR_CHAINED if chained else 0)
    st = lib().dr_chunked_plan_ex(flags, int(BH), int(T), int(dk), int(dv), ctypes.byref(bv),
                                  ctypes.byref(nprep), ctypes.byref(nseg))
    if st == DR_ERR_UNSUPPORTED:
        return None
    if st != DR_OK:
        raise DrScanError(st, "dr_chunked_plan_ex")
    return bv.value, nprep.value, nseg.value


def segment_counters(device=None) -> tuple:
    """(segmented scans, chained reruns after a failed hand-off check) on the device since
    the library was loaded; waits for the device's work first."""
    import torch

    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        scans, reruns = ctypes.c_ulonglong(0), ctypes.c_ulonglong(0)
        st = lib().dr_segment_counters(ctypes.byref(scans), ctypes.byref(reruns))
    if st != DR_OK:
        raise DrScanError(st, "dr_segment_counters")
    return scans.value, reruns.value


def chunked_applies(mode, dtype_is_bf16: bool, dk: int, dv: int) -> bool:
    """Whether dr_scan_fwd runs the chunked tensor-core kernel for this request."""
    variant = MODES[mode] if isinstance(mode, str) else int(mode)
    return (dtype_is_bf16 and dk == 128 and dv in (32, 64, 128)
            and variant in (DR_DELTANET, DR_GDN, DR_KDA, DR_GDN2))


# ---- around a scan: short convolution, selective state space scan, norms
#
# These calls are made once per layer and token, where the kernel takes some microseconds: views
# go to the library as one array of 64-bit words (the layout of dr_view and conv_split), pointers
# as plain integers, and a tensor that is as it should be costs one comparison of each property.

_fns = {}


def _call(name, device, *args):
    """Call an entry point with the device's current stream, with that device current."""
    import torch

    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    # (the stream's handle without a Stream object around it, which takes 2 us to make)
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    else:
        rc = fn(*args, stream)
    if rc != DR_OK:
        raise DrScanError(rc, name)


def _rows(t, name, shape, dtype, device):
    """Pointer of a tensor of `shape` with contiguous last dimension, in any layout."""
    if t.dtype is dtype and t.shape == shape and t.device == device and (
            t.stride(-1) == 1 or shape[-1] <= 1):
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous channels")


def _dense(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor, or 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    _check(t, name, shape, dtype, device)
    return t.data_ptr()


def _compute_dtype(t, name):
    import torch

    if t.dtype is torch.bfloat16:
        mode = DR_IN_BF16
    elif t.dtype is torch.float32:
        mode = 0
    else:
        raise ValueError(f"{name} must be bf16 or fp32")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return mode


def _conv_splits(splits, C, outs):
    """(heads, dim, normalised) of each split, checked."""
    if splits is None:
        splits = [(C // 128, 128)]
    splits = [(int(s[0]), int(s[1]), bool(s[2]) if len(s) > 2 else False) for s in splits]
    if sum(s[0] * s[1] for s in splits) != C:
        raise ValueError(f"splits must cover the {C} channels")
    if outs is not None and len(outs) != len(splits):
        raise ValueError(f"outs must hold {len(splits)} tensors")
    return splits


def short_conv(x, weight, bias=None, splits=None, state0=None, lengths=None, silu=True, eps=1e-6,
               outs=None, want_state=True):
    """Causal convolution over tokens, split into heads, through short_conv_fwd.
    x: [B,T,C] bf16 or fp32, contiguous channels; weight: [C,K] fp32; bias: [C] fp32 or None;
    splits: (heads, dim, normalise) for neighbouring channels, together all C (default: heads
    of 128); state0: [B,K-1,C] like x or None; lengths: [B] int32 or None; outs: a
    [B,heads,T,dim] tensor for each split, in any layout with contiguous channels. Returns
    (list of outputs, state_final [B,K-1,C] or None)."""
    import torch

    mode = _compute_dtype(x, "x")
    B, T, C = x.shape
    K = weight.shape[-1]
    dt, dev = x.dtype, x.device
    splits = _conv_splits(splits, C, outs)
    if outs is None:
        outs = [x.new_empty((B, h, T, d)) for h, d, _ in splits]
    words = [_rows(x, "x", x.shape, dt, dev), x.stride(0), 0, x.stride(1)]
    for i, ((h, d, n), o) in enumerate(zip(splits, outs)):
        words += (_rows(o, f"outs[{i}]", (B, h, T, d), dt, dev), *o.stride()[:3], h | d << 32, n)
    arr = (_LL * len(words))(*words)
    at = ctypes.addressof(arr)
    state = x.new_empty((B, K - 1, C)) if want_state else None
    _call("short_conv_fwd", dev, at, _dense(weight, "weight", (C, K), torch.float32, dev),
          _dense(bias, "bias", (C,), torch.float32, dev),
          _dense(state0, "state0", (B, K - 1, C), dt, dev),
          _dense(lengths, "lengths", (B,), torch.int32, dev), at + 32, len(splits),
          0 if state is None else state.data_ptr(), eps, B, T, C, K,
          mode | CONV_SILU if silu else mode)
    return list(outs), state


def short_conv_step(x, weight, bias=None, splits=None, state=None, silu=True, eps=1e-6, outs=None):
    """One token of short_conv on a resident state, through short_conv_step. x: [B,C]; state:
    [B,K-1,C] like x, shifted in place. Returns the outputs, [B,heads,dim] for each split."""
    import torch

    mode = _compute_dtype(x, "x")
    B, C = x.shape
    K = weight.shape[-1]
    dt, dev = x.dtype, x.device
    if state is None:
        raise ValueError("short_conv_step needs the state (updated in place)")
    splits = _conv_splits(splits, C, outs)
    if outs is None:
        outs = [x.new_empty((B, h, d)) for h, d, _ in splits]
    words = [_rows(x, "x", x.shape, dt, dev), x.stride(0), 0, 0]
    for i, ((h, d, n), o) in enumerate(zip(splits, outs)):
        words += (_rows(o, f"outs[{i}]", (B, h, d), dt, dev), *o.stride()[:2], 0, h | d << 32, n)
    arr = (_LL * len(words))(*words)
    at = ctypes.addressof(arr)
    _call("short_conv_step", dev, at, _dense(weight, "weight", (C, K), torch.float32, dev),
          _dense(bias, "bias", (C,), torch.float32, dev),
          _dense(state, "state", (B, K - 1, C), dt, dev), at + 32, len(splits), eps, B, C, K,
          mode | CONV_SILU if silu else mode)
    return list(outs)


def _ssm_views(x, dt, B, C, out, tokens):
    """The words of the views x, dt, B, C, out of a scan (tokens = (T,)) or a step (()), checked;
    with the mode bits of dt's type, G and N."""
    import torch

    dev, ty = x.device, x.dtype
    G, N = B.shape[1], B.shape[-1]
    bshape = (x.shape[0], G, *tokens, N)
    px, po = _rows(x, "x", x.shape, ty, dev), _rows(out, "out", x.shape, ty, dev)
    pb, pc = _rows(B, "B", bshape, ty, dev), _rows(C, "C", bshape, ty, dev)
    if dt.dtype is torch.bfloat16:
        mode = SSM_DT_BF16
    elif dt.dtype is torch.float32:
        mode = 0
    else:
        raise ValueError("dt must be bf16 or fp32")
    if dt.shape != x.shape[:-1] or dt.device != dev:
        raise ValueError(f"dt must have shape {tuple(x.shape[:-1])} on {dev}, got "
                         f"{tuple(dt.shape)} on {dt.device}")
    if tokens:
        arr = (_LL * 20)(px, *x.stride()[:3], dt.data_ptr(), *dt.stride(), pb, *B.stride()[:3], pc,
                         *C.stride()[:3], po, *out.stride()[:3])
    else:
        arr = (_LL * 20)(px, *x.stride()[:2], 0, dt.data_ptr(), *dt.stride(), 0, pb,
                         *B.stride()[:2], 0, pc, *C.stride()[:2], 0, po, *out.stride()[:2], 0)
    return arr, mode, G, N


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=True, S0=None, lengths=None,
             want_state=True, out=None, S_final=None, force_sequential=False):
    """Selective state space scan, through ssm_scan_fwd: S = exp(delta A) S + delta x B^T,
    y = S C + D x, delta = softplus(dt + dt_bias). x: [B,H,T,P]; B, C: [B,G,T,N] (bf16 or fp32
    like x); all in any layout with contiguous channels; dt: [B,H,T] bf16 or fp32, any strides;
    A, D, dt_bias: [H] fp32; S0: [B,H,P,N] fp32 or None; lengths: [B] int32 or None (rows of out
    behind a sequence are left as they were). Returns (out like x, S_final fp32 or None)."""
    import torch

    mode = _compute_dtype(x, "x")
    nb, H, T, P = x.shape
    dev, f32 = x.device, torch.float32
    if out is None:
        out = x.new_empty((nb, H, T, P))
    arr, bits, G, N = _ssm_views(x, dt, B, C, out, (T,))
    mode |= bits | (SSM_DT_SOFTPLUS if dt_softplus else 0)
    if force_sequential:
        mode |= DR_FORCE_SEQUENTIAL
    if want_state and S_final is None:
        S_final = A.new_empty((nb, H, P, N))
    at = ctypes.addressof(arr)
    _call("ssm_scan_fwd", dev, at, at + 32, _dense(A, "A", (H,), f32, dev), at + 64, at + 96,
          _dense(D, "D", (H,), f32, dev), _dense(dt_bias, "dt_bias", (H,), f32, dev),
          _dense(S0, "S0", (nb, H, P, N), f32, dev),
          _dense(lengths, "lengths", (nb,), torch.int32, dev), at + 128,
          _dense(S_final, "S_final", (nb, H, P, N), f32, dev), nb, H, G, T, P, N, mode)
    return out, S_final


def ssm_step(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=True, S=None, out=None):
    """One token of ssm_scan on a resident state, through ssm_step. x: [B,H,P]; dt: [B,H];
    B, C: [B,G,N]; S: [B,H,P,N] fp32, updated in place. Returns out [B,H,P] like x."""
    import torch

    mode = _compute_dtype(x, "x")
    nb, H, P = x.shape
    dev, f32 = x.device, torch.float32
    if S is None:
        raise ValueError("ssm_step needs the state S (updated in place)")
    if out is None:
        out = x.new_empty((nb, H, P))
    arr, bits, G, N = _ssm_views(x, dt, B, C, out, ())
    at = ctypes.addressof(arr)
    _call("ssm_step", dev, at, at + 32, _dense(A, "A", (H,), f32, dev), at + 64, at + 96,
          _dense(D, "D", (H,), f32, dev), _dense(dt_bias, "dt_bias", (H,), f32, dev),
          _dense(S, "S", (nb, H, P, N), f32, dev), at + 128, nb, H, G, P, N,
          mode | bits | (SSM_DT_SOFTPLUS if dt_softplus else 0))
    return out


def gated_norm(y, gate, weight, norm_heads=1, act="silu", gate_first=False, eps=1e-6, out=None):
    """RMS norm of a scan's output with its gate, through gated_norm_fwd. y: [B,H,T,d] in any
    layout with contiguous channels; gate: [B,T,H*d] like y, or None; weight: [H*d] fp32, or [d]
    for every head; norm_heads: neighbouring heads that are normalised together; act: "silu" or
    "sigmoid"; gate_first: the gate before the norm. Returns [B,T,H*d]."""
    import torch

    mode = _compute_dtype(y, "y")
    B, H, T, d = y.shape
    dev, ty = y.device, y.dtype
    row = (B, T, H * d)
    shared = H != 1 and weight.shape == (d,)
    if act not in ("silu", "sigmoid"):
        raise ValueError(f'act must be "silu" or "sigmoid", got {act!r}')
    if out is None:
        out = y.new_empty(row)
    mode |= ((NORM_SIGMOID if act == "sigmoid" else 0) | (NORM_GATE_FIRST if gate_first else 0)
             | (NORM_SHARED_WEIGHT if shared else 0))
    if gate is None:
        g = (0, 0, 0, 0)
    else:
        g = (_rows(gate, "gate", row, ty, dev), gate.stride(0), 0, gate.stride(1))
    arr = (_LL * 12)(_rows(y, "y", y.shape, ty, dev), *y.stride()[:3], *g,
                     _rows(out, "out", row, ty, dev), out.stride(0), 0, out.stride(1))
    at = ctypes.addressof(arr)
    _call("gated_norm_fwd", dev, at, at + 32,
          _dense(weight, "weight", (d,) if shared else (H * d,), torch.float32, dev), at + 64, eps,
          B, H, T, d, norm_heads, mode)
    return out


def block_norm(x, weight, residual=None, scale=1.0, post_weight=None, residual_dtype=None,
               eps=1e-6, out=None, residual_out=None):
    """Residual and norms between two blocks, through block_norm_fwd: z = x (or its RMS norm
    times post_weight), r = residual + scale z, out = RMS norm of r times weight. x: [...,D] bf16
    or fp32, rows at one pitch; residual: the same shape, contiguous, like x or fp32, or None;
    weight, post_weight: [D] fp32; scale: a number or [D] fp32; residual_dtype: of r where there
    is no residual (default: x's). Returns (out like x, r)."""
    import torch

    mode = _compute_dtype(x, "x")
    D, dev, f32 = x.shape[-1], x.device, torch.float32
    rows = x.numel() // D if D else 0
    x2 = x if x.dim() == 2 else x.view(rows, D)
    rt = residual.dtype if residual is not None else residual_dtype or x.dtype
    if rt not in (x.dtype, f32):
        raise ValueError(f"residual must be {x.dtype} or fp32, got {rt}")
    if residual is not None and residual_dtype not in (None, rt):
        raise ValueError(f"residual is {rt}, not {residual_dtype}")
    scale_v = 0
    if isinstance(scale, torch.Tensor):
        scale, scale_v = 1.0, _dense(scale, "scale", (D,), f32, dev)
    if out is None:
        out = x.new_empty(x.shape)
    if residual_out is None:
        residual_out = (x if rt is x.dtype else weight).new_empty(x.shape)
    if mode and rt is f32:
        mode |= NORM_RESIDUAL_F32
    _call("block_norm_fwd", dev, _rows(x2, "x", x2.shape, x.dtype, dev), x2.stride(0),
          _dense(residual, "residual", x.shape, rt, dev), _dense(weight, "weight", (D,), f32, dev),
          _dense(post_weight, "post_weight", (D,), f32, dev), scale_v, scale,
          _dense(out, "out", x.shape, x.dtype, dev),
          _dense(residual_out, "residual_out", x.shape, rt, dev), eps, rows, D, mode)
    return out, residual_out
