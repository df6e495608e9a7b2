"""What is measured of the operators at the two ends of the layer: the residual
addition with its RMS norm (and an 8-bit output), the row quantiser, and the
layer's matrix products with their epilogue, forward and backward.

A case names one operator and its sizes.  `run` computes it either in elementary
torch operations in 32 bits (own = False) or through gated_delta_rule_34_amd.
Hidden sizes of 1024 are the layer benchmark's 8 heads of 128 channels, 32768
rows its 8 x 4096 tokens.
"""
import math

import torch

own = False

EPS = 1e-5
F8MAX = 448.0  # largest finite e4m3 value
F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": F8}
SIZE = {"bf16": 2, "f32": 4, "f8": 1}
ACTS = ("none", "relu", "silu", "gelu")

#: the most a drawn case may cost: the largest listed case of its kind
MOST_FLOPS = 2 * 32768 * 4096 * 1024
MOST_ELEMENTS = 32768 * 1024


def listed():
    return [
        # the norm of a few decode tokens of the layer benchmark's width: latency
        {"name": "norm_decode", "op": "norm", "rows": 4, "D": 1024, "dtype": "bf16", "rdtype": "bf16", "out": "bf16",
         "residual": True, "rstd": False},
        # a training or prefill batch entering an 8-bit product, residual stream in fp32
        {"name": "norm8_prefill", "op": "norm", "rows": 32768, "D": 1024, "dtype": "bf16", "rdtype": "f32",
         "out": "f8", "residual": True, "rstd": True},
        # the backward of the same norm over a training batch, gradient of the residual stream joined in
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 32768, "D": 1024, "dtype": "bf16", "rdtype": "bf16",
         "dr": True},
        # a short ragged batch of a wide model, width without a power of two, no gradient from above
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "rows": 777, "D": 5125, "dtype": "f32", "rdtype": "f32",
         "dr": False},
        # the weights of a projection, quantised once for serving
        {"name": "quant_weight", "op": "quant", "rows": 4096, "D": 4096, "dtype": "bf16"},
        # the activations of a ragged prefill chunk before an 8-bit product
        {"name": "quant_rows_ragged", "op": "quant", "rows": 333, "D": 1368, "dtype": "f32"},
        # one decode token through an up projection: reads the weights once
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 1024, "dtype": "bf16", "out": "bf16",
         "act": "silu", "bias": True, "residual": False, "preact": False},
        # the up projection of a training batch; the pre-activation is kept for the backward
        {"name": "linear_train", "op": "linear", "M": 32768, "N": 4096, "K": 1024, "dtype": "bf16", "out": "bf16",
         "act": "silu", "bias": True, "residual": False, "preact": True},
        # a decode batch through a wide 8-bit projection, fp32 out, odd row and column counts
        {"name": "linear8_decode", "op": "linear", "M": 17, "N": 4099, "K": 4096, "dtype": "f8", "out": "f32",
         "act": "none", "bias": False, "residual": True, "preact": False},
        # the down projection of a prefill batch in 8 bits, added to the residual stream
        {"name": "linear8_prefill", "op": "linear", "M": 32768, "N": 1024, "K": 4096, "dtype": "f8", "out": "bf16",
         "act": "none", "bias": True, "residual": True, "preact": False},
        # gradients of a small ragged projection, kept in fp32 for the optimiser
        {"name": "linear_bwd_ragged", "op": "linear_bwd", "M": 1037, "N": 515, "K": 1024, "dy": "bf16",
         "grad": "f32", "act": "none", "bias": True},
        # gradients of the up projection of a training batch
        {"name": "linear_bwd_train", "op": "linear_bwd", "M": 16384, "N": 4096, "K": 1024, "dy": "bf16",
         "grad": "bf16", "act": "silu", "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "quant", "linear", "linear", "linear_bwd"))
    if op in ("norm", "norm_bwd", "quant"):
        D = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            D = max(8, D // 8 * 8)
        rows = max(1, min(_log(rng, 1, 32768), MOST_ELEMENTS // D))
        c = {"op": op, "rows": rows, "D": D, "dtype": rng.choice(("bf16", "bf16", "f32"))}
        if op == "quant":
            return c
        c["rdtype"] = "f32" if c["dtype"] == "f32" else rng.choice(("bf16", "f32"))
        if op == "norm":
            c["out"] = rng.choice((c["dtype"], c["dtype"], "f8"))
            c["residual"] = rng.random() < 0.75
            if not c["residual"]:
                c["rdtype"] = c["dtype"]
            c["rstd"] = rng.random() < 0.5
        else:
            c["dr"] = rng.random() < 0.6
        return c
    M, N, K = _log(rng, 1, 32768), _log(rng, 1, 8192), 16 * _log(rng, 1, 512)
    if rng.random() < 0.5:
        N = max(8, N // 8 * 8)
    per = 4 if op == "linear_bwd" else 2
    while per * M * N * K > MOST_FLOPS:
        M = max(1, M // 2)
    if op == "linear":
        c = {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(("bf16", "bf16", "f8")),
             "out": rng.choice(("bf16", "bf16", "f32")), "act": rng.choice(ACTS), "bias": rng.random() < 0.6,
             "residual": rng.random() < 0.4}
        c["preact"] = c["act"] != "none" and rng.random() < 0.5
        return c
    return {"op": op, "M": M, "N": N, "K": K, "dy": rng.choice(("bf16", "bf16", "f32")),
            "grad": rng.choice(("bf16", "f32")), "act": rng.choice(ACTS), "bias": rng.random() < 0.6}


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _to_f8(x):
    """Rows of x as e4m3 values and one fp32 scale a row."""
    s = x.abs().amax(dim=1) / F8MAX
    return (x / s[:, None]).clamp(-F8MAX, F8MAX).to(F8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = case
    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd", "quant"):
        rows, D = c["rows"], c["D"]
        s["x"] = _randn(gen, rows, D).to(DT[c["dtype"]])  # the norm's input, or its output's gradient
        if c["op"] == "quant":
            return s
        s["weight"] = 1.0 + 0.1 * _randn(gen, D)
        if c["op"] == "norm":
            s["residual"] = (2.0 * _randn(gen, rows, D)).to(DT[c["rdtype"]]) if c["residual"] else None
            return s
        s["r"] = (2.0 * _randn(gen, rows, D)).to(DT[c["rdtype"]])
        s["rstd"] = torch.rsqrt(s["r"].float().square().mean(dim=1) + EPS)
        s["dr"] = _randn(gen, rows, D).to(DT[c["rdtype"]]) if c["dr"] else None
        return s
    M, N, K = c["M"], c["N"], c["K"]
    x, w = _randn(gen, M, K), _randn(gen, N, K) * K ** -0.5
    s["bias"] = 0.1 * _randn(gen, N) if c["bias"] else None
    if c["op"] == "linear":
        s["xs"] = s["ws"] = None
        if c["dtype"] == "f8":
            (s["x"], s["xs"]), (s["w"], s["ws"]) = _to_f8(x), _to_f8(w)
        else:
            s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
        s["residual"] = _randn(gen, M, N).to(DT[c["out"]]) if c["residual"] else None
        return s
    s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
    s["dy"] = _randn(gen, M, N).to(DT[c["dy"]])
    s["z"] = None
    if c["act"] != "none":
        s["z"] = s["x"] @ s["w"].t()
        if c["bias"]:
            s["z"] = s["z"] + s["bias"].to(torch.bfloat16)
    return s


# ---- the operators in elementary operations ---------------------------------


def _act(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))))
    return z


def _act_grad(act, z):
    """Derivative of the activation at z."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _quant_plain(y):
    scale = y.abs().amax(dim=1) / F8MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (y / scale[:, None]).clamp(-F8MAX, F8MAX).to(F8), scale


def _norm_plain(s):
    c = s["case"]
    r = s["x"].float()
    out = {}
    if s["residual"] is not None:
        r = r + s["residual"].float()
        out["r"] = r.to(DT[c["rdtype"]])
    rstd = torch.rsqrt((r * r).mean(dim=1) + EPS)
    y = r * rstd[:, None] * s["weight"]
    if c["out"] == "f8":
        out["y"], out["scale"] = _quant_plain(y)
    else:
        out["y"] = y.to(DT[c["out"]])
    if c["rstd"]:
        out["rstd"] = rstd
    return out


def _norm_bwd_plain(s):
    dy, xhat = s["x"].float(), s["r"].float() * s["rstd"][:, None]
    wdy = dy * s["weight"]
    dx = s["rstd"][:, None] * (wdy - xhat * (wdy * xhat).mean(dim=1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {"dx": dx.to(s["r"].dtype), "dweight": (dy * xhat).sum(dim=0)}


def _linear_plain(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        z = z * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(DT[c["out"]])}
    if c["preact"]:
        out["z"] = z.to(torch.bfloat16)
    return out


def _linear_bwd_plain(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(c["act"], s["z"].float())
    out = {"dx": (dz @ s["w"].float()).to(DT[c["grad"]]), "dw": (dz.t() @ s["x"].float()).to(DT[c["grad"]])}
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


# ---- the framework's calls ----------------------------------------------------


def _own(s):
    import gated_delta_rule_34_amd as gdn
    c = s["case"]
    if c["op"] == "norm":
        y, r, rstd, scale = gdn.gdn_add_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                                out_dtype=DT[c["out"]], return_rstd=c["rstd"])
        out = {"y": y}
        if r is not None:
            out["r"] = r
        if scale is not None:
            out["scale"] = scale
        if rstd is not None:
            out["rstd"] = rstd
        return out
    if c["op"] == "norm_bwd":
        dx, dweight = gdn.gdn_add_rmsnorm_bwd(s["x"], s["r"], s["weight"], s["rstd"], dr=s["dr"])
        return {"dx": dx, "dweight": dweight}
    if c["op"] == "quant":
        q, scale = gdn.gdn_quantize_rows(s["x"])
        return {"q": q, "scale": scale}
    if c["op"] == "linear":
        y, z = gdn.gdn_linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=c["act"], x_scale=s["xs"],
                              w_scale=s["ws"], out_dtype=DT[c["out"]], return_preact=c["preact"])
        return {"y": y} if z is None else {"y": y, "z": z}
    dx, dw, dbias = gdn.gdn_linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=c["act"], bias=c["bias"],
                                       grad_dtype=DT[c["grad"]])
    return {"dx": dx, "dw": dw} if dbias is None else {"dx": dx, "dw": dw, "dbias": dbias}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "quant":
        q, scale = _quant_plain(state["x"].float())
        return {"q": q, "scale": scale}
    return _linear_plain(state) if op == "linear" else _linear_bwd_plain(state)


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd", "quant"):
        n, es = c["rows"] * c["D"], SIZE[c["dtype"]]
        if c["op"] == "quant":
            return {"bytes": n * (es + 1) + 4 * c["rows"], "flops": 3 * n}
        rs = SIZE[c["rdtype"]]
        if c["op"] == "norm":
            b = n * (es + SIZE[c["out"]] + (2 * rs if c["residual"] else 0)) + 4 * c["D"]
            b += 4 * c["rows"] * ((1 if c["out"] == "f8" else 0) + (1 if c["rstd"] else 0))
            return {"bytes": b, "flops": 6 * n}
        return {"bytes": n * (es + 2 * rs + (rs if c["dr"] else 0)) + 8 * c["D"] + 4 * c["rows"], "flops": 10 * n}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "linear":
        es = SIZE[c["dtype"]]
        b = (M * K + N * K) * es + M * N * SIZE[c["out"]] * (2 if c["residual"] else 1)
        b += (4 * N if c["bias"] else 0) + (2 * M * N if c["preact"] else 0) + (4 * (M + N) if c["dtype"] == "f8" else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    b = M * N * (SIZE[c["dy"]] + (2 if c["act"] != "none" else 0)) + (M * K + N * K) * (2 + SIZE[c["grad"]])
    return {"bytes": b + (4 * N if c["bias"] else 0), "flops": 4 * M * N * K}


# ---- the definitions in 64 bits -------------------------------------------------


def _e4m3_nearest(v):
    """The e4m3 values nearest to v (|v| <= 448), ties to the even significand: steps of 2^(e-3) for 2^e <= |v| < 2^(e+1),
    not below 2^-9."""
    _, e = torch.frexp(v.abs())  # |v| = m 2^e with 1/2 <= m < 1
    step = torch.exp2((e.to(torch.float64) - 4).clamp(min=-9))
    return torch.round(v / step) * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = lambda t: None if t is None else t.to(torch.float64)  # noqa: E731

    def eight(y):
        amax = y.abs().max(dim=1).values
        scale = torch.where(amax > 0, amax / F8MAX, torch.ones_like(amax))
        return _e4m3_nearest(y / scale.unsqueeze(1)), scale

    def phi(z):  # the normal distribution function
        return torch.special.ndtr(z)

    if c["op"] == "quant":
        q, scale = eight(d(s["x"]))
        return {"q": q, "scale": scale}
    if c["op"] == "norm":
        u = d(s["x"]) if s["residual"] is None else d(s["x"]) + d(s["residual"])
        inv = 1 / torch.sqrt(torch.einsum("ij,ij->i", u, u) / c["D"] + EPS)
        y = u * d(s["weight"]) * inv.unsqueeze(1)
        out = {"y": y}
        if c["out"] == "f8":
            out["y"], out["scale"] = eight(y)
        if s["residual"] is not None:
            out["r"] = u
        if c["rstd"]:
            out["rstd"] = inv
        return out
    if c["op"] == "norm_bwd":
        # y_j = w_j r_j s with s = (mean r^2 + eps)^(-1/2): dL/dr_i = s w_i dy_i - s^3 r_i / D sum_j dy_j w_j r_j
        dy, r, inv, w = d(s["x"]), d(s["r"]), d(s["rstd"]), d(s["weight"])
        dot = torch.einsum("ij,ij,j->i", dy, r, w)
        dx = inv.unsqueeze(1) * w * dy - r * (inv ** 3 * dot / c["D"]).unsqueeze(1)
        if s["dr"] is not None:
            dx = dx + d(s["dr"])
        return {"dx": dx, "dweight": torch.einsum("ij,ij,i->j", dy, r, inv)}
    if c["op"] == "linear":
        x, w = d(s["x"]), d(s["w"])
        if s["xs"] is not None:
            x, w = x * d(s["xs"]).unsqueeze(1), w * d(s["ws"]).unsqueeze(1)
        z = torch.mm(x, w.t().contiguous())
        if s["bias"] is not None:
            z += d(s["bias"])
        a = c["act"]
        y = torch.maximum(z, torch.zeros_like(z)) if a == "relu" else z * torch.sigmoid(z) if a == "silu" else \
            z * phi(z) if a == "gelu" else z
        out = {"y": y if s["residual"] is None else y + d(s["residual"])}
        if c["preact"]:
            out["z"] = z
        return out
    dz, a = d(s["dy"]), c["act"]
    if a != "none":
        z = d(s["z"])
        if a == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif a == "silu":
            dz = dz * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
        else:
            dz = dz * (phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    out = {"dx": torch.mm(dz, d(s["w"])), "dw": torch.mm(dz.t().contiguous(), d(s["x"]))}
    if c["bias"]:
        out["dbias"] = torch.einsum("ij->j", dz)
    return out
