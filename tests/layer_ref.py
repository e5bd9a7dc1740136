"""The operators around a scan, from their definitions in fp64 torch on the CPU (test oracle).

Each function also returns, where a tolerance needs it, the sum of the magnitudes that enter an
output: roundings of operands and of partial sums are bounded relative to that."""
from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def conv(x, weight, bias, splits, state0, lengths, eps, silu=True):
    """Outputs [B,h,T,d] per split (rows behind a sequence: NaN), state_final [B,K-1,C], and the
    magnitudes of the sums before the activation, laid out like the outputs."""
    x, weight, bias = f64(x), f64(weight), f64(bias)
    B, T, C = x.shape
    K = weight.shape[1]
    state0 = torch.zeros(B, K - 1, C, dtype=torch.float64) if state0 is None else f64(state0)
    outs = [torch.full((B, h, T, d), float("nan"), dtype=torch.float64) for h, d, _ in splits]
    mags = [torch.zeros(B, h, T, d, dtype=torch.float64) for h, d, _ in splits]
    final = torch.empty(B, K - 1, C, dtype=torch.float64)
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        rows = torch.cat([state0[b], x[b, :n]])
        final[b] = rows[rows.shape[0] - (K - 1):]
        for t in range(n):
            terms = rows[t:t + K].t() * weight
            c = terms.sum(1) + (bias if bias is not None else 0)
            m = terms.abs().sum(1) + (bias.abs() if bias is not None else 0)
            y = c * torch.sigmoid(c) if silu else c
            at = 0
            for i, s in enumerate(splits):
                h, d = s[0], s[1]
                v = y[at:at + h * d].view(h, d)
                mv = m[at:at + h * d].view(h, d)
                if len(s) > 2 and s[2]:
                    r = 1 / torch.sqrt((v * v).sum(1, keepdim=True) + eps)
                    v, mv = v * r, mv * r
                outs[i][b, :, t] = v
                mags[i][b, :, t] = mv
                at += h * d
    return outs, final, mags


def ssm(x, dt, A, Bm, Cm, D, dt_bias, softplus, S0, lengths):
    """(y [B,H,T,P], S [B,H,P,N], magnitudes of both); rows behind a sequence: NaN."""
    x, dt, A, Bm, Cm, D, dt_bias, S0 = (f64(t) for t in (x, dt, A, Bm, Cm, D, dt_bias, S0))
    B, H, T, P = x.shape
    G, N = Bm.shape[1], Bm.shape[3]
    D = torch.zeros(H, dtype=torch.float64) if D is None else D
    S = torch.zeros(B, H, P, N, dtype=torch.float64) if S0 is None else S0.clone()
    M = S.abs()
    y = torch.full((B, H, T, P), float("nan"), dtype=torch.float64)
    my = torch.zeros(B, H, T, P, dtype=torch.float64)
    z = dt if dt_bias is None else dt + dt_bias[:, None]
    delta = torch.logaddexp(z, torch.zeros_like(z)) if softplus else z
    of = torch.arange(H) // (H // G)
    for t in range(T):
        live = torch.ones(B, dtype=torch.bool) if lengths is None else t < f64(lengths)
        a = torch.exp(delta[:, :, t] * A)[..., None, None]
        b, c = Bm[:, of, t], Cm[:, of, t]
        w = (delta[:, :, t, None] * x[:, :, t])[..., None] * b[:, :, None]
        sel = live[:, None, None, None]
        S = torch.where(sel, a * S + w, S)
        M = torch.where(sel, a * M + w.abs(), M)
        sel = live[:, None, None]
        y[:, :, t] = torch.where(sel, (S * c[:, :, None]).sum(-1) + D[:, None] * x[:, :, t],
                                 y[:, :, t])
        my[:, :, t] = torch.where(sel, (M * c[:, :, None].abs()).sum(-1)
                                  + (D[:, None] * x[:, :, t]).abs(), my[:, :, t])
    return y, S, my, M


def act(g, name):
    return g * torch.sigmoid(g) if name == "silu" else torch.sigmoid(g)


def gated(y, gate, weight, heads, name, first, eps):
    y, gate, weight = f64(y), f64(gate), f64(weight)
    B, H, T, d = y.shape
    v = y.transpose(1, 2)
    u = torch.ones_like(v) if gate is None else act(gate.reshape(B, T, H, d), name)
    if first:
        v = v * u
    v = v.reshape(B, T, H // heads, heads * d)
    v = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)).reshape(B, T, H, d)
    v = v * (weight.view(1, d) if weight.numel() == d else weight.view(H, d))
    if not first:
        v = v * u
    return v.reshape(B, T, H * d)


def block(x, weight, residual, scale, post, eps):
    x, weight, residual, post = f64(x), f64(weight), f64(residual), f64(post)
    scale = f64(scale) if torch.is_tensor(scale) else scale
    norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w
    z = (x if post is None else norm(x, post)) * scale
    r = z if residual is None else residual + z
    mag = z.abs() if residual is None else residual.abs() + z.abs()
    return norm(r, weight), r, mag
