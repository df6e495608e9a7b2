"""What is measured of the operators that complete a block around a recurrent
mixer: the residual layer norm with its gradients, the gated feed-forward
projection with its gradients, and the selective state space scan with its short
causal convolution, for prompts (dense and packed) and for single tokens.

A case names one operator and its sizes.  `run` computes it either in elementary
torch operations in 32 bits (own = False) or through gated_delta_rule_34_amd.
Widths of 1024 are the layer benchmark's 8 heads of 128 channels, 32768 rows its
8 x 4096 tokens; a scan of 2048 channels is that width expanded twice.
"""
import math

import torch

own = False

EPS = 1e-5
F8MAX = 448.0  # largest finite e4m3 value
F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": F8}
SIZE = {"bf16": 2, "f32": 4, "f8": 1}
ACTS = ("silu", "silu", "gelu", "relu")

#: the most a drawn case may cost: the largest listed case of its kind
MOST_ELEMENTS = 32768 * 1024
MOST_FLOPS = 4 * 32768 * 4096 * 1024
MOST_CONV = 32768 * 2048
MOST_SCAN = 32768 * 2048 * 16
MOST_STATE = 128 * 4096 * 16


def listed():
    return [
        # the norm of a few decode tokens of the layer benchmark's width: latency
        {"name": "ln_token", "op": "ln", "rows": 4, "D": 1024, "dtype": "bf16", "rdtype": "bf16", "out": "bf16",
         "residual": True, "bias": True, "stats": False},
        # a training or prefill batch entering an 8-bit product, residual stream in fp32
        {"name": "ln8_prefill", "op": "ln", "rows": 32768, "D": 1024, "dtype": "bf16", "rdtype": "f32", "out": "f8",
         "residual": True, "bias": True, "stats": True},
        # the backward of the norm over a training batch, gradient of the residual stream joined in
        {"name": "ln_bwd_train", "op": "ln_bwd", "rows": 32768, "D": 1024, "dtype": "bf16", "rdtype": "bf16",
         "dr": True},
        # one decode token through the gate and up projections: reads both weights once
        {"name": "glu_token", "op": "glu", "M": 1, "N": 4096, "K": 1024, "dtype": "bf16", "out": "bf16", "act": "silu",
         "bias": False, "preact": False},
        # the gated projection of a training batch; both arguments are kept for the backward
        {"name": "glu_train", "op": "glu", "M": 32768, "N": 4096, "K": 1024, "dtype": "bf16", "out": "bf16",
         "act": "silu", "bias": False, "preact": True},
        # a ragged prefill chunk in 8 bits, odd row and column counts
        {"name": "glu8_ragged", "op": "glu", "M": 1037, "N": 2731, "K": 1024, "dtype": "f8", "out": "bf16",
         "act": "gelu", "bias": True, "preact": False},
        # gradients of the gated projection of a training batch
        {"name": "glu_bwd_train", "op": "glu_bwd", "M": 16384, "N": 4096, "K": 1024, "dy": "bf16", "grad": "bf16",
         "act": "silu", "bias": False},
        # the convolution before the scan over a batch of prompts
        {"name": "conv_prompt", "op": "conv", "B": 8, "T": 4096, "C": 2048, "W": 4, "dtype": "bf16", "state": False,
         "seqs": ""},
        # the same for one token of each of 64 sequences, carried inputs in and out: latency
        {"name": "conv_token", "op": "conv", "B": 64, "T": 1, "C": 2048, "W": 4, "dtype": "bf16", "state": True,
         "seqs": ""},
        # the scan over a batch of prompts, with the skip and the output gate
        {"name": "scan_prompt", "op": "scan", "B": 8, "T": 4096, "D": 2048, "N": 16, "dtype": "bf16", "z": True,
         "h0": False, "seqs": ""},
        # a ragged packed batch that goes on from carried states
        {"name": "scan_packed", "op": "scan", "B": 9, "T": 6000, "D": 1024, "N": 16, "dtype": "bf16", "z": True,
         "h0": True, "seqs": "2500,1,777,64,1300,200,33,1000,125"},
        # one token of each of 64 sequences: reads and writes their states
        {"name": "scan_token", "op": "step", "B": 64, "D": 2048, "N": 16, "dtype": "bf16", "z": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(rng, total):
    """total cut into a few ragged lengths."""
    n = min(total, _log(rng, 1, 24))
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(("ln", "ln_bwd", "glu", "glu", "glu_bwd", "conv", "scan", "scan", "step"))
    if op in ("ln", "ln_bwd"):
        D = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            D = max(8, D // 8 * 8)
        rows = max(1, min(_log(rng, 1, 32768), MOST_ELEMENTS // D))
        c = {"op": op, "rows": rows, "D": D, "dtype": rng.choice(("bf16", "bf16", "f32"))}
        c["rdtype"] = "f32" if c["dtype"] == "f32" else rng.choice(("bf16", "f32"))
        if op == "ln_bwd":
            c["dr"] = rng.random() < 0.6
            return c
        c["out"] = rng.choice((c["dtype"], c["dtype"], "f8"))
        c["residual"] = rng.random() < 0.75
        if not c["residual"]:
            c["rdtype"] = c["dtype"]
        c["bias"] = rng.random() < 0.7
        c["stats"] = rng.random() < 0.5
        return c
    if op in ("glu", "glu_bwd"):
        M, N, K = _log(rng, 1, 32768), _log(rng, 1, 8192), 16 * _log(rng, 1, 512)
        if rng.random() < 0.5:
            N = max(8, N // 8 * 8)
        per = 8 if op == "glu_bwd" else 4
        while per * M * N * K > MOST_FLOPS:
            M = max(1, M // 2)
        c = {"op": op, "M": M, "N": N, "K": K, "act": rng.choice(ACTS), "bias": rng.random() < 0.5}
        if op == "glu":
            c["dtype"] = rng.choice(("bf16", "bf16", "f8"))
            c["out"] = rng.choice(("bf16", "bf16", "f32"))
            c["preact"] = rng.random() < 0.5
        else:
            c["dy"] = rng.choice(("bf16", "bf16", "f32"))
            c["grad"] = rng.choice(("bf16", "bf16", "f32"))
        return c
    D = _log(rng, 64, 4096)
    if rng.random() < 0.7:
        D = max(8, D // 8 * 8)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "step":
        N = rng.choice((8, 16, 16, 32, 64))
        B = max(1, min(_log(rng, 1, 256), MOST_STATE // (D * N)))
        return {"op": op, "B": B, "D": D, "N": N, "dtype": dtype, "z": rng.random() < 0.7}
    T, B = _log(rng, 1, 8192), _log(rng, 1, 16)
    packed = rng.random() < 0.4
    if op == "conv":
        T = max(1, min(T, MOST_CONV // (D * B)))
        c = {"op": op, "B": B, "T": T, "C": D, "W": rng.choice((2, 3, 4, 4)), "dtype": dtype,
             "state": rng.random() < 0.5, "seqs": ""}
    else:
        N = rng.choice((8, 16, 16, 16, 32, 64))
        T = max(1, min(T, MOST_SCAN // (D * N * B)))
        c = {"op": op, "B": B, "T": T, "D": D, "N": N, "dtype": dtype, "z": rng.random() < 0.7,
             "h0": rng.random() < 0.5, "seqs": ""}
    if packed:  # B sequences of T tokens in all
        lens = _lengths(rng, T)
        c["B"], c["seqs"] = len(lens), ",".join(str(n) for n in lens)
    return c


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _to_f8(x):
    """Rows of x as e4m3 values and one fp32 scale a row."""
    s = x.abs().amax(dim=1) / F8MAX
    return (x / s[:, None]).clamp(-F8MAX, F8MAX).to(F8), s


def _lens(case):
    return [int(n) for n in case["seqs"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = case
    s = {"case": c}
    if c["op"] in ("ln", "ln_bwd"):
        rows, D = c["rows"], c["D"]
        s["x"] = _randn(gen, rows, D).to(DT[c["dtype"]])  # the norm's input, or its output's gradient
        s["weight"] = 1.0 + 0.1 * _randn(gen, D)
        if c["op"] == "ln":
            s["bias"] = 0.1 * _randn(gen, D) if c["bias"] else None
            s["residual"] = (0.5 + 2.0 * _randn(gen, rows, D)).to(DT[c["rdtype"]]) if c["residual"] else None
            return s
        s["r"] = (0.5 + 2.0 * _randn(gen, rows, D)).to(DT[c["rdtype"]])
        r = s["r"].float()
        s["mean"] = r.mean(dim=1)
        s["rstd"] = torch.rsqrt((r - s["mean"][:, None]).square().mean(dim=1) + EPS)
        s["dr"] = _randn(gen, rows, D).to(DT[c["rdtype"]]) if c["dr"] else None
        return s
    if c["op"] in ("glu", "glu_bwd"):
        M, N, K = c["M"], c["N"], c["K"]
        x, w = _randn(gen, M, K), _randn(gen, 2 * N, K) * K ** -0.5  # gate rows, then up rows
        s["bias"] = 0.1 * _randn(gen, 2 * N) if c["bias"] else None
        if c["op"] == "glu":
            s["xs"] = s["ws"] = None
            if c["dtype"] == "f8":
                (s["x"], s["xs"]), (s["w"], s["ws"]) = _to_f8(x), _to_f8(w)
            else:
                s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
            return s
        s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
        s["dy"] = _randn(gen, M, N).to(DT[c["dy"]])
        s["z"] = s["x"] @ s["w"].t()
        if c["bias"]:
            s["z"] = s["z"] + s["bias"].to(torch.bfloat16)
        return s
    dt = DT[c["dtype"]]
    packed = bool(c.get("seqs"))
    if packed:
        cu = [0]
        for n in _lens(c):
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    lead = (c["B"],) if c["op"] == "step" else (c["T"],) if packed else (c["B"], c["T"])
    if c["op"] == "conv":
        C, W = c["C"], c["W"]
        s["x"] = _randn(gen, *lead, C).to(dt)
        s["weight"] = W ** -0.5 * _randn(gen, C, W)
        s["bias"] = 0.1 * _randn(gen, C)
        s["state"] = _randn(gen, c["B"], W - 1, C) if c["state"] else None
        return s
    D, N = c["D"], c["N"]
    x = _randn(gen, *lead, D)
    s["x"] = (x * torch.sigmoid(x)).to(dt)
    s["dt"] = (0.5 * _randn(gen, *lead, D)).to(dt)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=gen, device="cuda"))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it: steps between 0.001 and 0.1
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * _randn(gen, D, N))
    s["B"], s["C"] = _randn(gen, *lead, N).to(dt), _randn(gen, *lead, N).to(dt)
    s["D"] = 1.0 + 0.1 * _randn(gen, D)
    s["z"] = _randn(gen, *lead, D).to(dt) if c["z"] else None
    s["h"] = _randn(gen, c["B"], D, N) if c["op"] == "step" or c["h0"] else None
    return s


# ---- the operators in elementary operations ---------------------------------


def _act(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))))


def _act_grad(act, z):
    """Derivative of the activation at z."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _ln_plain(s):
    c = s["case"]
    u = s["x"].float()
    out = {}
    if s["residual"] is not None:
        u = u + s["residual"].float()
        out["r"] = u.to(DT[c["rdtype"]])
    mean = u.mean(dim=1)
    d = u - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(dim=1) + EPS)
    y = d * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["out"] == "f8":
        scale = y.abs().amax(dim=1) / F8MAX
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        out["y"], out["scale"] = (y / scale[:, None]).clamp(-F8MAX, F8MAX).to(F8), scale
    else:
        out["y"] = y.to(DT[c["out"]])
    if c["stats"]:
        out["mean"], out["rstd"] = mean, rstd
    return out


def _ln_bwd_plain(s):
    dy, xhat = s["x"].float(), (s["r"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["weight"]
    dx = s["rstd"][:, None] * (a - a.mean(dim=1, keepdim=True) - xhat * (a * xhat).mean(dim=1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {"dx": dx.to(s["r"].dtype), "dweight": (dy * xhat).sum(dim=0), "dbias": dy.sum(dim=0)}


def _glu_plain(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        z = z * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        z = z + s["bias"]
    g, u = z[:, :c["N"]], z[:, c["N"]:]
    out = {"y": (_act(c["act"], g) * u).to(DT[c["out"]])}
    if c["preact"]:
        out["z"] = z.to(torch.bfloat16)
    return out


def _glu_bwd_plain(s):
    c = s["case"]
    dy, z = s["dy"].float(), s["z"].float()
    g, u = z[:, :c["N"]], z[:, c["N"]:]
    dz = torch.cat([dy * u * _act_grad(c["act"], g), dy * _act(c["act"], g)], dim=1)
    out = {"dx": (dz @ s["w"].float()).to(DT[c["grad"]]), "dw": (dz.t() @ s["x"].float()).to(DT[c["grad"]])}
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


def _conv_one(x, w, bias, state):
    """x [B, T, C], state [B, W-1, C] or None: (y, new state)."""
    B, T, C = x.shape
    W = w.shape[1]
    if state is None:
        state = torch.zeros(B, W - 1, C, device=x.device)
    xs = torch.cat([state, x.float()], dim=1)
    y = bias.expand(B, T, C)
    for j in range(W):
        y = y + w[:, j] * xs[:, j:j + T]
    return _act("silu", y).to(x.dtype), xs[:, T:].contiguous()


def _conv_plain(s):
    c = s["case"]
    if not c["seqs"]:
        y, state = _conv_one(s["x"], s["weight"], s["bias"], s["state"])
        return {"y": y, "state": state}
    ys, states, at = [], [], 0
    for i, n in enumerate(_lens(c)):
        st = None if s["state"] is None else s["state"][i:i + 1]
        y, st = _conv_one(s["x"][at:at + n][None], s["weight"], s["bias"], st)
        ys.append(y[0])
        states.append(st)
        at += n
    return {"y": torch.cat(ys), "state": torch.cat(states)}


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _padded(t, lens):
    """Packed rows [total, ...] as [sequences, longest, ...], zero behind each sequence."""
    out = torch.zeros(len(lens), max(lens), *t.shape[1:], dtype=t.dtype, device=t.device)
    at = 0
    for i, n in enumerate(lens):
        out[i, :n] = t[at:at + n]
        at += n
    return out


def _scan_plain(s):
    c = s["case"]
    x, dt, Bm, Cm = (s[n].float() for n in ("x", "dt", "B", "C"))
    d = _softplus(dt + s["dt_bias"])
    lens = _lens(c) if c["seqs"] else None
    u = d * x
    if lens:  # behind a sequence's end d and u are zero: its state stays
        d, u, Bm, Cm = (_padded(t, lens) for t in (d, u, Bm, Cm))
    h = torch.zeros(c["B"], c["D"], c["N"], device=x.device) if s["h"] is None else s["h"]
    y = torch.empty_like(u)
    for t in range(u.shape[1]):
        h = torch.exp(d[:, t, :, None] * s["A"]) * h + u[:, t, :, None] * Bm[:, t, None, :]
        y[:, t] = (h * Cm[:, t, None, :]).sum(dim=-1)
    if lens:
        y = torch.cat([y[i, :n] for i, n in enumerate(lens)])
    y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _act("silu", s["z"].float())
    return {"y": y.to(s["x"].dtype), "h": h}


def _step_plain(s):
    x = s["x"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(d[..., None] * s["A"]) * s["h"] + (d * x)[..., None] * s["B"].float()[:, None, :]
    y = (h * s["C"].float()[:, None, :]).sum(dim=-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _act("silu", s["z"].float())
    return {"y": y.to(s["x"].dtype), "h": h}


PLAIN = {"ln": _ln_plain, "ln_bwd": _ln_bwd_plain, "glu": _glu_plain, "glu_bwd": _glu_bwd_plain, "conv": _conv_plain,
         "scan": _scan_plain, "step": _step_plain}


# ---- the framework's calls ----------------------------------------------------


def _own(s):
    import gated_delta_rule_34_amd as gdn
    c = s["case"]
    if c["op"] == "ln":
        y, r, mean, rstd, scale = gdn.gdn_add_layernorm(s["x"], s["weight"], bias=s["bias"], residual=s["residual"],
                                                        eps=EPS, out_dtype=DT[c["out"]], return_stats=c["stats"])
        out = {"y": y}
        if r is not None:
            out["r"] = r
        if scale is not None:
            out["scale"] = scale
        if mean is not None:
            out["mean"], out["rstd"] = mean, rstd
        return out
    if c["op"] == "ln_bwd":
        dx, dweight, dbias = gdn.gdn_add_layernorm_bwd(s["x"], s["r"], s["weight"], s["mean"], s["rstd"], dr=s["dr"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if c["op"] == "glu":
        y, z = gdn.gdn_gated_linear(s["x"], s["w"], bias=s["bias"], act=c["act"], x_scale=s["xs"], w_scale=s["ws"],
                                    out_dtype=DT[c["out"]], return_preact=c["preact"])
        return {"y": y} if z is None else {"y": y, "z": z}
    if c["op"] == "glu_bwd":
        dx, dw, dbias = gdn.gdn_gated_linear_bwd(s["dy"], s["x"], s["w"], s["z"], act=c["act"], bias=c["bias"],
                                                 grad_dtype=DT[c["grad"]])
        return {"dx": dx, "dw": dw} if dbias is None else {"dx": dx, "dw": dw, "dbias": dbias}
    if c["op"] == "conv":
        kw = dict(bias=s["bias"], act="silu", conv_state=s["state"])
        if c["seqs"]:
            y, state = gdn.gdn_causal_conv_varlen(s["x"], s["weight"], s["cu"], **kw)
        else:
            y, state = gdn.gdn_causal_conv(s["x"], s["weight"], **kw)
        return {"y": y, "state": state}
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if c["op"] == "step":
        y, h = gdn.gdn_selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h"],
                                      state_out=torch.empty_like(s["h"]), **kw)
    elif c["seqs"]:
        y, h = gdn.gdn_selective_scan_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], h0=s["h"], **kw)
    else:
        y, h = gdn.gdn_selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], h0=s["h"], **kw)
    return {"y": y, "h": h}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] in ("ln", "ln_bwd"):
        n, es, rs = c["rows"] * c["D"], SIZE[c["dtype"]], SIZE[c["rdtype"]]
        if c["op"] == "ln_bwd":
            return {"bytes": n * (es + 2 * rs + (rs if c["dr"] else 0)) + 12 * c["D"] + 8 * c["rows"], "flops": 13 * n}
        b = n * (es + SIZE[c["out"]] + (2 * rs if c["residual"] else 0)) + (8 if c["bias"] else 4) * c["D"]
        b += 4 * c["rows"] * ((1 if c["out"] == "f8" else 0) + (2 if c["stats"] else 0))
        return {"bytes": b, "flops": 8 * n}
    if c["op"] in ("glu", "glu_bwd"):
        M, N, K = c["M"], c["N"], c["K"]
        if c["op"] == "glu":
            es = SIZE[c["dtype"]]
            b = (M * K + 2 * N * K) * es + M * N * SIZE[c["out"]] + (4 * M * N if c["preact"] else 0)
            b += (8 * N if c["bias"] else 0) + (4 * (M + 2 * N) if c["dtype"] == "f8" else 0)
            return {"bytes": b, "flops": 4 * M * N * K}
        b = M * N * (SIZE[c["dy"]] + 4) + (M * K + 2 * N * K) * (2 + SIZE[c["grad"]])
        return {"bytes": b + (8 * N if c["bias"] else 0), "flops": 8 * M * N * K}
    es = SIZE[c["dtype"]]
    tokens = c["B"] if c["op"] == "step" else c["T"] if c["seqs"] else c["B"] * c["T"]
    if c["op"] == "conv":
        carried = 4 * c["B"] * (c["W"] - 1) * c["C"]
        return {"bytes": 2 * tokens * c["C"] * es + 4 * c["C"] * (c["W"] + 1) + carried * (2 if c["state"] else 1),
                "flops": tokens * c["C"] * (2 * c["W"] + 5)}
    state = 4 * c["B"] * c["D"] * c["N"]
    b = tokens * es * (c["D"] * (4 if c["z"] else 3) + 2 * c["N"]) + 4 * c["D"] * (c["N"] + 2)
    b += state * (2 if c["op"] == "step" or c["h0"] else 1)
    # a product and an exponential for the decay, a product and two multiply-adds
    return {"bytes": b, "flops": 7 * tokens * c["D"] * c["N"]}


# ---- the definitions in 64 bits -------------------------------------------------


def _e4m3_nearest(v):
    """The e4m3 values nearest to v (|v| <= 448), ties to the even significand: steps of 2^(e-3) for 2^e <= |v| < 2^(e+1),
    not below 2^-9."""
    _, e = torch.frexp(v.abs())  # |v| = m 2^e with 1/2 <= m < 1
    step = torch.exp2((e.to(torch.float64) - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _recurrence(a, b, h):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling: after a turn with distance k every entry stands for
    the 2 k steps that end there."""
    a, b = a.clone(), b.clone()
    if h is not None:
        b[0] += a[0] * h
    k = 1
    while k < a.shape[0]:
        b[k:] = b[k:] + a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = lambda t: None if t is None else t.to(torch.float64)  # noqa: E731

    def activated(g):  # the activation's value and derivative
        if c["act"] == "relu":
            return torch.maximum(g, torch.zeros_like(g)), torch.where(g > 0, torch.ones_like(g), torch.zeros_like(g))
        if c["act"] == "silu":
            p = torch.sigmoid(g)
            return g * p, p + g * p * torch.sigmoid(-g)
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)

    if c["op"] == "ln":
        u = d(s["x"]) if s["residual"] is None else d(s["x"]) + d(s["residual"])
        var, mean = torch.var_mean(u, dim=1, correction=0)
        inv = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(torch.zeros_like(u) if s["bias"] is None else d(s["bias"]).expand_as(u),
                          (u - mean.unsqueeze(1)) * inv.unsqueeze(1), d(s["weight"]).expand_as(u))
        out = {"y": y}
        if s["residual"] is not None:
            out["r"] = u
        if c["out"] == "f8":
            amax = y.abs().max(dim=1).values
            scale = torch.where(amax > 0, amax / F8MAX, torch.ones_like(amax))
            out["y"], out["scale"] = _e4m3_nearest(y / scale.unsqueeze(1)), scale
        if c["stats"]:
            out["mean"], out["rstd"] = mean, inv
        return out
    if c["op"] == "ln_bwd":
        # y_j = w_j (r_j - m) s: dL/dr_i = s w_i dy_i - s/D sum_j w_j dy_j - s^3 (r_i - m) / D sum_j dy_j w_j (r_j - m)
        dy, inv, w = d(s["x"]), d(s["rstd"]), d(s["weight"])
        r = d(s["r"]) - d(s["mean"]).unsqueeze(1)
        dot, plain = torch.einsum("ij,ij,j->i", dy, r, w), torch.einsum("ij,j->i", dy, w)
        dx = inv.unsqueeze(1) * w * dy - (inv * plain / c["D"]).unsqueeze(1) - r * (inv ** 3 * dot / c["D"]).unsqueeze(1)
        if s["dr"] is not None:
            dx = dx + d(s["dr"])
        return {"dx": dx, "dweight": torch.einsum("ij,ij,i->j", dy, r, inv), "dbias": torch.einsum("ij->j", dy)}
    if c["op"] == "glu":
        x, w = d(s["x"]), d(s["w"])
        if s["xs"] is not None:
            x, w = x * d(s["xs"]).unsqueeze(1), w * d(s["ws"]).unsqueeze(1)
        g, u = (torch.mm(x, half.t().contiguous()) for half in w.split(c["N"]))
        if s["bias"] is not None:
            bg, bu = d(s["bias"]).split(c["N"])
            g, u = g + bg, u + bu
        out = {"y": activated(g)[0] * u}
        if c["preact"]:
            out["z"] = torch.cat([g, u], dim=1)
        return out
    if c["op"] == "glu_bwd":
        dy, x = d(s["dy"]), d(s["x"])
        (g, u), (wg, wu) = d(s["z"]).split(c["N"], dim=1), d(s["w"]).split(c["N"])
        f, df = activated(g)
        dg, du = dy * df * u, dy * f
        out = {"dx": torch.mm(dg, wg.contiguous()) + torch.mm(du, wu.contiguous()),
               "dw": torch.cat([torch.mm(t.t().contiguous(), x) for t in (dg, du)])}
        if c["bias"]:
            out["dbias"] = torch.cat([torch.einsum("ij->j", t) for t in (dg, du)])
        return out
    lens = _lens(c) if c.get("seqs") else None
    ends = [0]
    for n in lens or [c.get("T", 1)] * c["B"]:
        ends.append(ends[-1] + n)
    flat = lambda t: None if t is None else d(t).reshape(-1, t.shape[-1])  # noqa: E731
    if c["op"] == "conv":
        x, w, C, W = flat(s["x"]), d(s["weight"]), c["C"], c["W"]
        ys, states = [], []
        for i, (a, b) in enumerate(zip(ends, ends[1:])):
            old = x.new_zeros(W - 1, C) if s["state"] is None else d(s["state"][i])
            line = torch.cat([old, x[a:b]])
            v = d(s["bias"]) + torch.einsum("tcj,cj->tc", line.unfold(0, W, 1), w)
            ys.append(v * torch.sigmoid(v))
            states.append(line[b - a:])
        return {"y": torch.cat(ys).reshape(s["x"].shape), "state": torch.stack(states)}
    x, dt, Bm, Cm, z = (flat(s[n]) for n in ("x", "dt", "B", "C", "z"))
    v = dt + d(s["dt_bias"])
    step = torch.where(v > 0, v + torch.log1p(torch.exp(-v)), torch.log1p(torch.exp(v)))
    A = d(s["A"])
    y, h = torch.empty_like(x), torch.empty(c["B"], c["D"], c["N"], dtype=torch.float64, device=x.device)
    for i, (a, b) in enumerate(zip(ends, ends[1:])):
        per = max(1, (1 << 28) // ((b - a) * c["N"]))  # channels at a time
        for k in range(0, c["D"], per):
            ch = slice(k, min(k + per, c["D"]))
            decay = torch.exp(step[a:b, ch].unsqueeze(2) * A[ch])
            put = (step[a:b, ch] * x[a:b, ch]).unsqueeze(2) * Bm[a:b].unsqueeze(1)
            hs = _recurrence(decay, put, None if s["h"] is None else d(s["h"][i, ch]))
            y[a:b, ch] = torch.matmul(hs, Cm[a:b].unsqueeze(2)).squeeze(2)
            h[i, ch] = hs[-1]
    y = y + x * d(s["D"])
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return {"y": y.reshape(s["x"].shape), "h": h}
