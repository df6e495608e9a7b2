"""Plain fp64 definitions of the short causal convolution and the selective state space scan -- TEST INFRASTRUCTURE
ONLY (tests; the product path never imports this module)."""
from __future__ import annotations

import numpy as np


def silu(v):
    return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def causal_conv(x, w, b=None, state=None, act="silu"):
    """(y, new state) of x [B, T, C], w [C, W], state [B, W-1, C]."""
    B, T, C = x.shape
    W = w.shape[1]
    if state is None:
        state = np.zeros((B, W - 1, C))
    line = np.concatenate([state, x], axis=1)
    y = np.zeros_like(x) if b is None else np.broadcast_to(b, x.shape).copy()
    for j in range(W):
        y = y + w[:, j] * line[:, j:j + T]
    return (silu(y) if act == "silu" else y), line[:, T:]


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, per_step=0.0):
    """(y, h, bar of y, bar of h) of x, dt, z [batch, T, ch], B, C [batch, T, N], A [ch, N], h0 [batch, ch, N].

    The bars bound what fp32 arithmetic may be off by.  Per step: d is within 2^-20 of itself, the exponent d A within
    2^-20 of itself (and per_step more, relatively, for sums of d over a part of the sequence), exp2 within 2^-22, the
    input d x B within 2^-19, the multiply-add within 2^-24; errors decay as the state does."""
    n, T, ch = x.shape
    N = A.shape[1]
    h = np.zeros((n, ch, N)) if h0 is None else h0.astype(np.float64)
    e = np.zeros_like(h)
    d = softplus(dt if dt_bias is None else dt + dt_bias)
    y, ey = np.zeros_like(x), np.zeros_like(x)
    for t in range(T):
        arg = d[:, t, :, None] * A
        a = np.exp(arg)
        put = (d[:, t] * x[:, t])[..., None] * B[:, t, None, :]
        e = a * e + (np.abs(arg) * (2.0 ** -20 + per_step) + 2.0 ** -22) * a * np.abs(h) + 2.0 ** -19 * np.abs(put)
        h = a * h + put
        e = e + 2.0 ** -24 * np.abs(h)
        c = C[:, t, None, :]
        y[:, t] = (c * h).sum(axis=-1)
        ey[:, t] = (np.abs(c) * e).sum(axis=-1) + (N / 4 + 6) * 2.0 ** -24 * (np.abs(c * h)).sum(axis=-1)
    if D is not None:
        y = y + D * x
        ey = ey + 2.0 ** -23 * (np.abs(D * x) + np.abs(y))
    if z is not None:
        g = silu(z)
        y, ey = y * g, ey * np.abs(g)
        ey = ey * (1 + 2.0 ** -18) + (2.0 ** -22 * np.abs(z) + 2.0 ** -20) * np.abs(y)
    return y, h, ey, e
