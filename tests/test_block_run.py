"""The operators at the ends of the layer together with the layer itself, as a
model runs them: a block's forward (norm, projections, prologue, rule, gated
norm, output projection into the residual stream), its 8-bit form, prefill
against single tokens, and a training step of a feed-forward pair."""
import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H, D, E = 2, 64, 256     # heads, head size, width of the block


def _params(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = {"norm": 1 + 0.1 * r(E), "gnorm": 1 + 0.1 * r(D), "A_log": torch.zeros(H, device="cuda"),
         "dt_bias": 0.1 * r(H), "wo": (H * D) ** -0.5 * r(E, H * D)}
    for n in ("q", "k", "v", "z"):
        p["w" + n] = E ** -0.5 * r(H * D, E)
    for n in ("a", "b"):
        p["w" + n] = E ** -0.5 * r(H, E)
    for n in ("q", "k", "v"):
        p["c" + n] = 0.5 * r(H * D, 4)
    return p


def _mul(x, w, eight, xs, **kw):
    """x @ w^T, in 8 bits where x already is."""
    if eight:
        q, s = gdn.gdn_quantize_rows(w.to(BF))
        return gdn.gdn_linear(x, q, x_scale=xs, w_scale=s, **kw)[0]
    return gdn.gdn_linear(x, w.to(BF), **kw)[0]


def _block(p, x, stream, conv=None, state=None, eight=False):
    """One block on x [B, T, E] (the previous block's output) and the residual stream.  Returns (out, stream, conv
    state, rule state)."""
    B, T, _ = x.shape
    y, r, _, xs = gdn.gdn_add_rmsnorm(x, p["norm"], residual=stream, out_dtype=F8 if eight else BF)
    xq, xk, xv, z = (_mul(y, p["w" + n], eight, xs).view(B, T, H, D) for n in ("q", "k", "v", "z"))
    a, b = (_mul(y, p["w" + n], eight, xs, out_dtype=F32) for n in ("a", "b"))
    q, k, v, g, beta, conv = gdn.gdn_prologue(xq, xk, xv, a, b, p["cq"], p["ck"], p["cv"], p["A_log"], p["dt_bias"],
                                              conv_state=conv)
    if T == 1 and state is not None:
        o = gdn.gdn_recurrent_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], state)[:, None]
    else:
        o, state = gdn.gdn_chunk_fwd(q, k, v, g, beta, h0=state)
    u = gdn.gdn_gated_rmsnorm(o.contiguous(), z, p["gnorm"]).view(B, T, H * D)
    us = None
    if eight:
        u, us = gdn.gdn_quantize_rows(u)
    return _mul(u, p["wo"], eight, us, residual=r.to(BF)), r, conv, state


def _block64(p, x, stream):
    """The same in 64 bits with torch operations."""
    p = {k: v.double() for k, v in p.items()}
    x = x.double() + stream.double()
    B, T, _ = x.shape
    y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-5) * p["norm"]

    def conv(n):
        t = torch.nn.functional.pad((y @ p["w" + n].t()).transpose(1, 2), (3, 0))
        t = torch.nn.functional.conv1d(t, p["c" + n][:, None], groups=H * D).transpose(1, 2)
        return torch.nn.functional.silu(t).view(B, T, H, D)

    q, k, v = conv("q"), conv("k"), conv("v")
    q, k = (t * torch.rsqrt(t.pow(2).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    g = -p["A_log"].exp() * torch.nn.functional.softplus(y @ p["wa"].t() + p["dt_bias"])
    beta = torch.sigmoid(y @ p["wb"].t())
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device=x.device)
    o = []
    for t in range(T):
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        o.append(D ** -0.5 * (S * q[:, t, :, :, None]).sum(-2))
    o = torch.stack(o, 1)
    z = (y @ p["wz"].t()).view(B, T, H, D)
    o = o * torch.rsqrt(o.pow(2).mean(-1, keepdim=True) + 1e-5) * p["gnorm"] * torch.nn.functional.silu(z)
    return o.reshape(B, T, H * D) @ p["wo"].t() + x


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("eight,bar", [(False, 2.0 ** -7), (True, 2.0 ** -4)])
def test_block_forward(eight, bar):
    """Each step rounds its output once (2^-8 of it at most in bf16, 2^-4 in e4m3, of independent signs) and the block's
    branch is less than half of its output, the rest being the residual stream: four such roundings in sequence,
    averaged over K products in each projection, stay within one unit of the type's half step doubled for bf16,
    and within the half step for e4m3, in the 2-norm."""
    p = _params(1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randn(2, 100, E, generator=gen, device="cuda").to(BF)
    stream = (2 * torch.randn(2, 100, E, generator=gen, device="cuda"))
    out, r, _, _ = _block(p, x, stream, eight=eight)
    assert torch.equal(r, x.float() + stream)
    ref = _block64(p, x, stream)
    assert _rel(out, ref) <= bar


def test_prefill_then_tokens_equals_the_whole_sequence():
    """31 tokens at once and 3 one by one, through the carried convolution and rule states, against 34 at once: the
    same arithmetic up to the chunked and the recurrent form of the rule (bf16 path against fp32 step)."""
    p = _params(3)
    torch.manual_seed(4)
    x = torch.randn(2, 34, E, device="cuda").to(BF)
    stream = torch.randn(2, 34, E, device="cuda")
    whole = _block(p, x, stream)[0]
    part, _, conv, state = _block(p, x[:, :31].contiguous(), stream[:, :31].contiguous())
    outs = [part]
    for t in range(31, 34):
        o, _, conv, state = _block(p, x[:, t:t + 1].contiguous(), stream[:, t:t + 1].contiguous(), conv, state)
        outs.append(o)
    assert _rel(torch.cat(outs, 1), whole.double()) <= 2.0 ** -7


def test_training_step_of_a_feed_forward_pair():
    """norm -> up projection with SiLU -> down projection, forward and backward, against autograd in 64 bits.  Every
    gradient passes at most five roundings to bf16 (2^-8 each, of independent signs), so its 2-norm is within
    3 * 2^-8; the rounding of the sums themselves is far below."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    M, F = 333, 640
    x, res = r(M, E).to(BF), r(M, E)
    wn, w1, b1, w2 = 1 + 0.1 * r(E), (E ** -0.5 * r(F, E)).to(BF), 0.1 * r(F), (F ** -0.5 * r(E, F)).to(BF)
    dout = r(M, E).to(BF)
    y, rs, rstd, _ = gdn.gdn_add_rmsnorm(x, wn, residual=res, return_rstd=True)
    h, z = gdn.gdn_linear(y, w1, bias=b1, act="silu", return_preact=True)
    out, _ = gdn.gdn_linear(h, w2)
    dh, dw2, _ = gdn.gdn_linear_bwd(dout, h, w2, grad_dtype=BF)
    dy, dw1, db1 = gdn.gdn_linear_bwd(dh, y, w1, z=z, act="silu", bias=True)
    dx, dwn = gdn.gdn_add_rmsnorm_bwd(dy, rs, wn, rstd, dr=dout.float())     # out + stream: the stream's gradient joins
    leaves = [t.double().requires_grad_() for t in (x, wn, w1, b1, w2)]
    X, WN, W1, B1, W2 = leaves
    U = X + res.double()
    Y = U * torch.rsqrt(U.pow(2).mean(-1, keepdim=True) + 1e-5) * WN
    OUT = torch.nn.functional.silu(Y @ W1.t() + B1) @ W2.t()
    ((OUT + U) * dout.double()).sum().backward()
    assert _rel(out, OUT.detach()) <= 2.0 ** -7
    for got, t in ((dx, X), (dwn, WN), (dw1, W1), (db1, B1), (dw2, W2)):
        assert _rel(got, t.grad) <= 3 * 2.0 ** -8


def test_eight_bit_weights_stand_for_their_values():
    """quantise -> multiply equals multiplying the dequantised values."""
    torch.manual_seed(6)
    x, w = torch.randn(50, 512, device="cuda").to(BF), torch.randn(96, 512, device="cuda").to(BF)
    (xq, xs), (wq, ws) = gdn.gdn_quantize_rows(x), gdn.gdn_quantize_rows(w)
    y, _ = gdn.gdn_linear(xq, wq, x_scale=xs, w_scale=ws, out_dtype=F32)
    f = lambda q, s: q.float().double() * s.double()[:, None]  # noqa: E731
    ref, _ = ob.linear(f(xq, xs).cpu().numpy(), f(wq, ws).cpu().numpy())
    bar = 514 * 2.0 ** -24 * (np.abs(f(xq, xs).cpu().numpy()) @ np.abs(f(wq, ws).cpu().numpy()).T)
    assert (np.abs(y.double().cpu().numpy() - ref) <= bar).all()
