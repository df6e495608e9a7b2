"""Plain fp64 definitions of the operations at the two ends of the layer --
TEST INFRASTRUCTURE ONLY (tests; the product path never imports this module):
the residual addition with its RMS norm, the 8-bit rounding of a row, the
matrix product with its epilogue, and their gradients.

GatedDeltaNet walkthrough (yfxerp.com), data-flow overview: the token mixer is
projections -> short convolution -> gates -> rule -> gated norm -> output
projection inside a residual block whose input is RMS-normalised.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erf

F8MAX = 448.0


def e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even: 3 significand bits after the leading one, smallest normal
    2^-6, steps of 2^-9 below it; beyond 448 + half a step there is no value (NaN)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    e = np.where(2.0 ** e > a, e - 1, e)          # log2 may round up across a power of two
    e = np.where(2.0 ** (e + 1) <= a, e + 1, e)
    step = 2.0 ** np.maximum(e - 3, -9)
    q = np.round(v / step) * step
    return np.where(np.abs(q) > F8MAX, np.nan, q)


def quantize_rows(y):
    """(codes' values, scale per row): scale = max|y| / 448, 1 for a row of zeros."""
    amax = np.max(np.abs(y), axis=-1)
    scale = np.where(amax == 0, 1.0, amax / F8MAX)
    with np.errstate(invalid="ignore"):
        return e4m3(y / scale[..., None]), scale


def add_rmsnorm(x, w, residual=None, eps=1e-5):
    """(y, u, rstd)."""
    u = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(u * u, axis=-1) + eps)
    return u * rstd[..., None] * w, u, rstd


def add_rmsnorm_bwd(dy, r, w, rstd, dr=None):
    """(dx, dw) at the given r and rstd."""
    xhat = r * rstd[..., None]
    g = dy * w
    dx = rstd[..., None] * (g - xhat * np.mean(g * xhat, axis=-1, keepdims=True))
    dw = (dy * xhat).reshape(-1, r.shape[-1]).sum(axis=0)
    return (dx if dr is None else dx + dr), dw


def act(name, z):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return z * 0.5 * (1.0 + erf(z / np.sqrt(2.0)))
    assert name == "none"
    return z


def act_grad(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        p = 1.0 / (1.0 + np.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if name == "gelu":
        return 0.5 * (1.0 + erf(z / np.sqrt(2.0))) + z * np.exp(-z * z / 2.0) / np.sqrt(2.0 * np.pi)
    assert name == "none"
    return np.ones_like(z)


def linear(x, w, bias=None, residual=None, name="none", x_scale=None, w_scale=None):
    """(y, z): z = (x w^T) x_scale w_scale + bias, y = act(z) + residual."""
    z = x @ w.T
    if x_scale is not None:
        z = z * x_scale[:, None] * w_scale
    if bias is not None:
        z = z + bias
    y = act(name, z)
    return (y if residual is None else y + residual), z


def linear_bwd(dy, x, w, z=None, name="none"):
    """(dx, dw, dbias, dz)."""
    dz = dy if name == "none" else dy * act_grad(name, z)
    return dz @ w, dz.T @ x, dz.sum(axis=0), dz


def add_layernorm(x, w, b=None, residual=None, eps=1e-5):
    """(y, u, mean, rstd)."""
    u = x if residual is None else x + residual
    mean = np.mean(u, axis=-1)
    d = u - mean[..., None]
    rstd = 1.0 / np.sqrt(np.mean(d * d, axis=-1) + eps)
    y = d * rstd[..., None] * w
    return (y if b is None else y + b), u, mean, rstd


def add_layernorm_bwd(dy, r, w, mean, rstd, dr=None):
    """(dx, dw, db) at the given r, mean and rstd."""
    xhat = (r - mean[..., None]) * rstd[..., None]
    a = dy * w
    dx = rstd[..., None] * (a - np.mean(a, axis=-1, keepdims=True) - xhat * np.mean(a * xhat, axis=-1, keepdims=True))
    D = r.shape[-1]
    return (dx if dr is None else dx + dr), (dy * xhat).reshape(-1, D).sum(axis=0), dy.reshape(-1, D).sum(axis=0)


def gated_linear(x, w, bias=None, name="silu", x_scale=None, w_scale=None):
    """(y, z): z = (g, u) = (x w^T) x_scale w_scale + bias with the gate's rows of w first, y = act(g) u."""
    _, z = linear(x, w, bias, None, "none", x_scale, w_scale)
    N = w.shape[0] // 2
    return act(name, z[:, :N]) * z[:, N:], z


def gated_linear_bwd(dy, x, w, z, name="silu"):
    """(dx, dw, dbias, dz) with dz = (dg, du)."""
    N = w.shape[0] // 2
    g, u = z[:, :N], z[:, N:]
    dz = np.concatenate([dy * u * act_grad(name, g), dy * act(name, g)], axis=1)
    return dz @ w, dz.T @ x, dz.sum(axis=0), dz
