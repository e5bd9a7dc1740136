"""The operators around a selective state space layer, as they are measured.

`short_conv` and `short_conv_step` (causal convolution of K taps with SiLU, split into heads,
heads optionally L2-normalised), `ssm_scan` and `ssm_step` (S = exp(delta A) S + delta x B^T,
y = S C + D x), `gated_norm` (RMS norm of a scan's output with its gate) and `block_norm`
(norm after a block, residual with its scale, norm before the next block).

Each case names its operator in "op". The plain forms below work in 32 bits (decays summed in
64) and round once; `exact` goes by the definitions, token by token, in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # q, k, v of a delta-rule layer before its scan: the sizes of the KDA benchmark
        dict(name="conv qkv B8 H16 T4096", op="conv", dtype="bf16", B=8, T=4096, K=4, splits="16x128n,16x128n,16x128",
             lengths=False, state=False),
        # x, B, C of a state space layer: a padded batch of prompts that go on from a cache
        dict(name="conv xBC ragged fp32 T777", op="conv", dtype="fp32", B=3, T=777, K=4, splits="8x64,1x128,1x128",
             lengths=True, state=True),
        # the same for one token of each of 128 sequences
        dict(name="conv step B128", op="conv_step", dtype="bf16", B=128, K=4, splits="32x128,1x128,1x128"),
        # short prompts of several lengths, 32 bits throughout
        dict(name="scan ragged fp32 T301", op="scan", dtype="fp32", B=2, H=4, G=2, T=301, P=32, N=32,
             lengths=True, state=True, rows="head"),
        # a batch of prompts: the sizes of the KDA benchmark, B and C shared by the heads
        dict(name="scan B8 H16 T4096", op="scan", dtype="bf16", B=8, H=16, G=1, T=4096, P=128, N=128,
             lengths=False, state=False, rows="token"),
        # one long prompt over few heads, from a state: the long-context benchmark
        dict(name="scan B1 H16 T32768", op="scan", dtype="bf16", B=1, H=16, G=1, T=32768, P=64, N=128,
             lengths=False, state=True, rows="head"),
        # one sequence's next token: latency
        dict(name="step B1 H16", op="step", dtype="bf16", B=1, H=16, G=1, P=64, N=128),
        # the decode benchmark: 4096 heads whose states do not fit the cache
        dict(name="step B128 H32", op="step", dtype="bf16", B=128, H=32, G=1, P=128, N=128),
        # after a scan of the KDA benchmark's sizes: norm by head, then the gate
        dict(name="gated norm B8 H16 T4096", op="gated", dtype="bf16", B=8, H=16, T=4096, d=128, heads=1,
             first=False, act="silu", shared=True),
        # one token each: gate first, then one norm over all heads
        dict(name="gated norm step B128 fp32", op="gated", dtype="fp32", B=128, H=32, T=1, d=64, heads=32,
             first=True, act="silu", shared=False),
        # between two blocks of a prompt: the residual stream in 32 bits
        dict(name="block norm 32768 x 2048", op="block", dtype="bf16", rows=32768, D=2048, wide=True, post=False,
             vector=False, first=False),
        # one token each: norm after the block, a scale for each channel, norm before the next
        dict(name="block norm 128 x 4096", op="block", dtype="bf16", rows=128, D=4096, wide=False, post=True,
             vector=True, first=False),
    ]


def draw(rng):
    def span(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["conv", "conv", "conv_step", "scan", "scan", "scan", "step", "gated", "block"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("conv", "conv_step"):
        d = rng.choice([32, 64, 128])
        n = rng.choice([32, 64, 128])
        H = span(1, 32)
        g = rng.choice([1, 2])
        splits = rng.choice([f"{H}x{d}n,{H}x{d}n,{H}x{n}", f"{H}x{d},{g}x{n},{g}x{n}", f"{H}x{d}n"])
        width = sum(h * e for h, e, _ in parse(splits))
        K = rng.choice([2, 3, 4, 4])
        if op == "conv_step":
            return dict(op=op, dtype=dtype, B=span(1, 512), K=K, splits=splits)
        B = span(1, 16)
        T = span(1, max(1, min(32768, (1 << 26) // (B * width))))
        return dict(op=op, dtype=dtype, B=B, T=T, K=K, splits=splits, lengths=rng.random() < 0.5,
                    state=rng.random() < 0.5)
    if op in ("scan", "step"):
        P, N = rng.choice([32, 64, 64, 128]), rng.choice([32, 64, 128, 128])
        G = rng.choice([1, 1, 2, 4])
        H = G * span(1, 32 // G)
        if op == "step":
            return dict(op=op, dtype=dtype, B=span(1, 128), H=H, G=G, P=P, N=N)
        B = span(1, 8)
        most = (1 << 19) if dtype == "bf16" else (1 << 16)
        T = span(1, max(1, min(32768, most // (B * H))))
        return dict(op=op, dtype=dtype, B=B, H=H, G=G, T=T, P=P, N=N, lengths=rng.random() < 0.5,
                    state=rng.random() < 0.5, rows=rng.choice(["head", "token"]))
    if op == "gated":
        d, H, B = rng.choice([32, 64, 128]), rng.choice([1, 2, 4, 6, 8, 16, 32]), span(1, 16)
        T = span(1, max(1, min(32768, (1 << 26) // (B * H * d))))
        heads = rng.choice([h for h in (1, 2, 3, H) if H % h == 0])
        return dict(op=op, dtype=dtype, B=B, H=H, T=T, d=d, heads=heads, first=rng.random() < 0.5,
                    act=rng.choice(["silu", "sigmoid"]), shared=rng.random() < 0.5)
    D = 8 * span(4, 1024)
    return dict(op=op, dtype=dtype, rows=span(1, max(1, min(65536, (1 << 26) // D))), D=D, wide=rng.random() < 0.5,
                post=rng.random() < 0.5, vector=rng.random() < 0.5, first=rng.random() < 0.2)


def parse(splits):
    """"16x128n,1x64" -> [(16, 128, True), (1, 64, False)]: heads, width of a head, normalised."""
    got = []
    for s in splits.split(","):
        h, d = s.rstrip("n").split("x")
        got.append((int(h), int(d), s.endswith("n")))
    return got


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, c = case["op"], case
    if op in ("conv", "conv_step"):
        C = sum(h * d for h, d, _ in parse(c["splits"]))
        rows = c["B"] * c.get("T", 1)
        held = c["B"] * (c["K"] - 1) * C * e * (2 if op == "conv_step" or c.get("state") else 1)
        return {"bytes": 2 * rows * C * e + held + C * (c["K"] + 1) * 4, "flops": rows * C * (2 * c["K"] + 6)}
    if op in ("scan", "step"):
        heads = c["B"] * c["H"] * c.get("T", 1)
        pairs = c["B"] * c["G"] * c.get("T", 1)
        states = c["B"] * c["H"] * c["P"] * c["N"] * 4 * (2 if op == "step" or c.get("state") else 1)
        return {"bytes": 2 * heads * c["P"] * e + 2 * pairs * c["N"] * e + 4 * heads + states,
                "flops": heads * (5 * c["P"] * c["N"] + 2 * c["P"] + 10)}
    if op == "gated":
        n = c["B"] * c["H"] * c["T"] * c["d"]
        return {"bytes": 3 * n * e + (c["d"] if c["shared"] else c["H"] * c["d"]) * 4, "flops": 9 * n}
    n = c["rows"] * c["D"]
    r = 4 if c["wide"] else e
    return {"bytes": n * (2 * e + (1 if c["first"] else 2) * r) + 4 * c["D"] * (1 + c["post"] + c["vector"]),
            "flops": n * (6 + 4 * c["post"])}


# ----------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 17)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=gen, device=DEV)

    def lengths(B, T):
        # of a padded batch: any length, one of them the longest, one of them empty where there are three
        n = torch.randint(0, T + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        n[0] = T
        if B > 2:
            n[1] = 0
        return n

    s = dict(case=case, op=case["op"])
    op = case["op"]
    if op in ("conv", "conv_step"):
        B, K, splits = case["B"], case["K"], parse(case["splits"])
        C = sum(h * d for h, d, _ in splits)
        s.update(splits=splits, weight=normal(C, K, std=K ** -0.5, dtype=torch.float32),
                 bias=normal(C, std=0.1, dtype=torch.float32))
        if op == "conv_step":
            s.update(x=normal(B, C), state=normal(B, K - 1, C))
            return s
        T = case["T"]
        # the projection that feeds it makes 64 channels more (steps and gates): rows are not contiguous
        s.update(x=normal(B, T, C + 64)[..., :C], state0=normal(B, K - 1, C) if case["state"] else None,
                 lengths=lengths(B, T) if case["lengths"] else None)
        if case["lengths"]:  # rows behind a sequence stay as they were
            s.update(outs=[normal(B, h, T, d) for h, d, _ in splits])
        return s
    if op in ("scan", "step"):
        B, H, G, P, N = (case[k] for k in "BHGPN")
        rate = torch.exp(uniform(math.log(1e-3), math.log(0.1), H))  # steps between 0.001 and 0.1
        s.update(A=-uniform(1.0, 16.0, H), D=normal(H, dtype=torch.float32), bias=torch.log(torch.expm1(rate)))
        if op == "step":
            s.update(x=normal(B, H, P), dt=normal(B, H, std=0.5, dtype=torch.float32), Bm=normal(B, G, N),
                     Cm=normal(B, G, N), S=normal(B, H, P, N, std=0.1, dtype=torch.float32))
            return s
        T = case["T"]
        if case["rows"] == "token":  # channels of one row after another, as a convolution leaves them
            row = normal(B, T, H * P + 2 * G * N)
            x, Bm, Cm = row.split([H * P, G * N, G * N], dim=-1)
            x = x.unflatten(-1, (H, P)).transpose(1, 2)
            Bm, Cm = (m.unflatten(-1, (G, N)).transpose(1, 2) for m in (Bm, Cm))
            dt = normal(B, T, H, std=0.5).transpose(1, 2)
            out = normal(B, T, H, P).transpose(1, 2)
        else:
            x, Bm, Cm = normal(B, H, T, P), normal(B, G, T, N), normal(B, G, T, N)
            dt = normal(B, H, T, std=0.5, dtype=torch.float32)
            out = normal(B, H, T, P)
        s.update(x=x, Bm=Bm, Cm=Cm, dt=dt, out=out, lengths=lengths(B, T) if case["lengths"] else None,
                 S0=normal(B, H, P, N, std=0.1, dtype=torch.float32) if case["state"] else None)
        return s
    if op == "gated":
        B, H, T, d = (case[k] for k in "BHTd")
        w = 1 + normal(*((d,) if case["shared"] else (H * d,)), std=0.1, dtype=torch.float32)
        s.update(y=normal(B, H, T, d, std=0.5), gate=normal(B, T, H * d), weight=w)
        return s
    R, D = case["rows"], case["D"]
    s.update(x=normal(R, D), weight=1 + normal(D, std=0.1, dtype=torch.float32),
             residual=None if case["first"] else normal(R, D, std=2.0, dtype=torch.float32 if case["wide"] else t),
             post=1 + normal(D, std=0.1, dtype=torch.float32) if case["post"] else None,
             scale=uniform(0.05, 0.5, D) if case["vector"] else 0.7071)
    return s


# -------------------------------------------------------------------------------------- run

EPS = 1e-6


def run(s):
    return kernels(s) if own else plain(s)


def kernels(s):
    import delta_rule_recurrent_chunked_b200 as drs

    op, case = s["op"], s["case"]
    if op == "conv":
        outs, state = drs.short_conv(s["x"], s["weight"], s["bias"], splits=s["splits"], state0=s["state0"],
                                     lengths=s["lengths"], eps=EPS, outs=s.get("outs"))
        return [*outs, state]
    if op == "conv_step":
        outs = drs.short_conv_step(s["x"], s["weight"], s["bias"], splits=s["splits"], state=s["state"], eps=EPS)
        return [*outs, s["state"]]
    if op == "scan":
        return drs.ssm_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], dt_bias=s["bias"],
                            dt_softplus=True, S0=s["S0"], lengths=s["lengths"], out=s["out"])
    if op == "step":
        return drs.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], dt_bias=s["bias"],
                            dt_softplus=True, S=s["S"]), s["S"]
    if op == "gated":
        return drs.gated_norm(s["y"], s["gate"], s["weight"], norm_heads=case["heads"], act=case["act"],
                              gate_first=case["first"], eps=EPS)
    return drs.block_norm(s["x"], s["weight"], residual=s["residual"], scale=s["scale"], post_weight=s["post"],
                          residual_dtype=torch.float32 if case["wide"] else None, eps=EPS)


def plain(s):
    return {"conv": plain_conv, "conv_step": plain_conv_step, "scan": plain_scan, "step": plain_step,
            "gated": plain_gated, "block": plain_block}[s["op"]](s)


def sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def in_heads(y, splits):
    """[B,T,C] in 32 bits -> a [B,heads,T,d] for each split, normalised where it says so."""
    parts = torch.split(y, [h * d for h, d, _ in splits], dim=-1)
    parts = [p.unflatten(-1, (h, d)).transpose(1, 2) for p, (h, d, _) in zip(parts, splits)]
    return [p * torch.rsqrt((p * p).sum(-1, keepdim=True) + EPS) if n else p for p, (_, _, n) in zip(parts, splits)]


def plain_conv(s):
    x, w, K = s["x"], s["weight"], s["weight"].shape[1]
    B, T, C = x.shape
    head = s["state0"] if s["state0"] is not None else x.new_zeros(B, K - 1, C)
    rows = torch.cat([head, x], dim=1)
    f = rows.float()
    c = s["bias"] + f[:, 0:T] * w[:, 0] + f[:, 1:T + 1] * w[:, 1]
    if K > 2:
        c = c + f[:, 2:T + 2] * w[:, 2]
    if K > 3:
        c = c + f[:, 3:T + 3] * w[:, 3]
    outs = [p.to(x.dtype).contiguous() for p in in_heads(c * sigmoid(c), s["splits"])]
    if s["lengths"] is None:
        return [*outs, rows[:, T:].contiguous()]
    n = s["lengths"].long()
    live = (torch.arange(T, device=x.device) < n[:, None])[:, None, :, None]
    at = n[:, None] + torch.arange(K - 1, device=x.device)
    state = torch.gather(rows, 1, at[:, :, None].expand(-1, -1, C))
    return [*(torch.where(live, o, kept) for o, kept in zip(outs, s["outs"])), state]


def plain_conv_step(s):
    rows = torch.cat([s["state"], s["x"][:, None]], dim=1)
    c = s["bias"] + (rows.float() * s["weight"].t()).sum(1)
    outs = [p.squeeze(2).to(s["x"].dtype) for p in in_heads((c * sigmoid(c))[:, None], s["splits"])]
    s["state"].copy_(rows[:, 1:])
    return [*outs, s["state"]]


def plain_scan(s, Q=64):
    """In chunks of Q tokens: inside a chunk by its Q x Q weights, between chunks by their states."""
    x, Bm, Cm = s["x"], s["Bm"], s["Cm"]
    B, H, T, P = x.shape
    G, N = Bm.shape[1], Bm.shape[3]
    R, nc = H // G, -(-T // Q)
    dev = x.device
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=dev)
    live = torch.arange(nc * Q, device=dev) < n[:, None]  # [B, nc Q]

    def chunks(v, heads):  # [B,heads,T,w] -> [B,G,heads/G,nc,Q,w] in 32 bits, zeros behind the sequence
        v = torch.nn.functional.pad(v.float(), (0, 0, 0, nc * Q - T))
        v = torch.where(live[:, None, :, None], v, torch.zeros((), device=dev))
        return v.reshape(B, G, heads // G, nc, Q, v.shape[-1])

    delta = softplus(s["dt"].float() + s["bias"][:, None])
    delta = chunks(delta[..., None], H)[..., 0]                       # [B,G,R,nc,Q]
    xs, bs, cs = chunks(x, H), chunks(Bm, G), chunks(Cm, G)
    la = (delta * s["A"].reshape(G, R, 1, 1)).double()
    cum = la.cumsum(-1)
    tri = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    w = torch.where(tri, cum[..., :, None] - cum[..., None, :], -math.inf)
    w = torch.exp(w).float() * delta[..., None, :]
    y = (torch.matmul(cs, bs.transpose(-1, -2)) * w) @ xs             # [B,G,R,nc,Q,P]
    scaled = xs * (delta * torch.exp(cum[..., -1:] - cum).float())[..., None]
    add = torch.matmul(scaled.transpose(-1, -2), bs)                  # [B,G,R,nc,P,N]
    ends = torch.nn.functional.pad(cum[..., -1].cumsum(-1), (1, 0))   # decay before each chunk, and at the end
    over = ends[..., :, None] - ends[..., None, 1:]
    over = torch.where(torch.ones(nc + 1, nc, dtype=torch.bool, device=dev).tril(-1), over, -math.inf)
    S = torch.matmul(torch.exp(over).float(), add.reshape(B, G, R, nc, P * N)).reshape(B, G, R, nc + 1, P, N)
    if s["S0"] is not None:
        S = S + torch.exp(ends).float()[..., None, None] * s["S0"].reshape(B, G, R, 1, P, N)
    y = y + torch.exp(cum).float()[..., None] * torch.matmul(cs, S[..., :-1, :, :].transpose(-1, -2))
    y = y.reshape(B, H, nc * Q, P)[:, :, :T] + s["D"][:, None, None] * x.float()
    out = torch.where(live[:, None, :T, None], y.to(x.dtype), s["out"])
    return out, S[..., -1, :, :].reshape(B, H, P, N).contiguous()


def plain_step(s):
    x, S = s["x"].float(), s["S"]
    R = x.shape[1] // s["Bm"].shape[1]
    Bm, Cm = (m.float().repeat_interleave(R, dim=1) for m in (s["Bm"], s["Cm"]))
    delta = softplus(s["dt"] + s["bias"])
    S.mul_(torch.exp(delta * s["A"])[..., None, None])
    S.add_((delta[..., None] * x)[..., None] * Bm[:, :, None, :])
    y = torch.matmul(S, Cm[..., None])[..., 0] + s["D"][:, None] * x
    return y.to(s["x"].dtype), S


def plain_gated(s):
    y, case = s["y"], s["case"]
    B, H, T, d = y.shape
    v, g = y.transpose(1, 2).float(), s["gate"].float().unflatten(-1, (H, d))
    g = g * sigmoid(g) if case["act"] == "silu" else sigmoid(g)
    v = v * g if case["first"] else v
    v = v.reshape(B, T, H // case["heads"], case["heads"] * d)
    v = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)).reshape(B, T, H, d)
    v = v * (s["weight"] if case["shared"] else s["weight"].reshape(H, d))
    v = v if case["first"] else v * g
    return v.to(y.dtype).reshape(B, T, H * d)


def plain_block(s):
    v = s["x"].float()
    if s["post"] is not None:
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["post"]
    v = v * s["scale"]
    if s["residual"] is not None:
        v = v + s["residual"].float()
    out = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"]).to(s["x"].dtype)
    return out, v.to(torch.float32 if s["case"]["wide"] else s["x"].dtype)


# ------------------------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"conv": exact_conv, "conv_step": exact_conv, "scan": exact_scan, "step": exact_scan,
            "gated": exact_gated, "block": exact_block}[case["op"]](case, s, f)


def exact_conv(case, s, f):
    step = case["op"] == "conv_step"
    x = f["x"][:, None] if step else f["x"]
    past = f["state"] if step else f["state0"]
    B, T, C = x.shape
    K = case["K"]
    n = [T] * B if s.get("lengths") is None else s["lengths"].tolist()
    held = torch.zeros(B, K - 1, C, dtype=torch.float64, device=DEV) if past is None else past.clone()
    got = [torch.empty(B, h, T, d, dtype=torch.float64, device=DEV) if s.get("outs") is None else o.double()
           for (h, d, _), o in zip(s["splits"], s.get("outs") or s["splits"])]
    for b in range(B):
        if n[b] == 0:
            continue
        line = torch.cat([held[b], x[b, :n[b]]])                      # [K - 1 + n, C]
        c = torch.einsum("tck,ck->tc", line.unfold(0, K, 1), f["weight"]) + f["bias"]
        c = c / (1 + torch.exp(-c))
        at = 0
        for i, (h, d, normed) in enumerate(s["splits"]):
            for j in range(h):
                v = c[:, at:at + d]
                got[i][b, j, :n[b]] = v / torch.sqrt(v.square().sum(1, keepdim=True) + EPS) if normed else v
                at += d
        held[b] = line[-(K - 1):]
    return [*(o[:, :, 0] if step else o for o in got), held]


def exact_scan(case, s, f):
    step = case["op"] == "step"
    x, dt, Bm, Cm = ((f[k][:, :, None] for k in ("x", "dt", "Bm", "Cm")) if step
                     else (f[k] for k in ("x", "dt", "Bm", "Cm")))
    B, H, T, P = x.shape
    group = torch.arange(H, device=DEV) // (H // Bm.shape[1])
    S = f["S"].clone() if step else torch.zeros(B, H, P, case["N"], dtype=torch.float64, device=DEV) \
        if f["S0"] is None else f["S0"].clone()
    delta = torch.nn.functional.softplus(dt + f["bias"][:, None], threshold=1000.0)
    if s.get("lengths") is not None:  # a step of zero keeps the state
        delta = delta * (torch.arange(T, device=DEV) < s["lengths"][:, None])[:, None]
    a = torch.exp(delta * f["A"][:, None])
    y = torch.empty(B, H, T, P, dtype=torch.float64, device=DEV)
    scaled = x * delta[..., None]
    for t in range(T):
        b, c = Bm[:, group, t], Cm[:, group, t]
        S.mul_(a[:, :, t, None, None]).addcmul_(scaled[:, :, t, :, None], b[:, :, None, :])
        torch.matmul(S, c[..., None], out=y[:, :, t, :, None])
    y += f["D"][:, None, None] * x
    if s.get("lengths") is not None:
        for b, n in enumerate(s["lengths"].tolist()):
            y[b, :, n:] = f["out"][b, :, n:]
    return (y[:, :, 0] if step else y), S


def exact_gated(case, s, f):
    y, g, H, d, m = f["y"], f["gate"], case["H"], case["d"], case["heads"]
    B, _, T, _ = y.shape
    out = torch.empty(B, T, H * d, dtype=torch.float64, device=DEV)
    weight = f["weight"].repeat(H) if case["shared"] else f["weight"]
    for at in range(0, H, m):  # one normalised group of heads after another
        cols = slice(at * d, (at + m) * d)
        v = y[:, at:at + m].permute(0, 2, 1, 3).reshape(B, T, m * d)
        u = 1 / (1 + torch.exp(-g[..., cols]))
        u = u * g[..., cols] if case["act"] == "silu" else u
        if case["first"]:
            v = v * u
        v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * weight[cols]
        out[..., cols] = v if case["first"] else v * u
    return out


def exact_block(case, s, f):
    def norm(v, w):
        return v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS) * w

    r = (norm(f["x"], f["post"]) if case["post"] else f["x"]) * f["scale"]
    r = r if f["residual"] is None else r + f["residual"]
    return norm(r, f["weight"]), r
