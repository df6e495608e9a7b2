"""GPU parity of the residual RMS norm, its backward and the row quantiser,
through the public calls, against the fp64 definitions in oracle/block.py.

Tolerances.  The kernels compute in fp32 and round each output once.
  - r = x + residual is one correctly rounded fp32 addition: 2^-24 |r|, plus
    2^-8 |r| where r is bf16.
  - y = u s w: a thread adds at most 32 squares in order, then at most 6 + 16
    partial sums, all positive, so the mean is within 54 * 2^-24 of its value
    relatively and s within half of that; u, s and the two products add four
    roundings: (27 + 4) 2^-24 < 2^-19.  fp32 bar 2^-18; bf16 bar 2^-8 + 2^-16.
  - 8 bits: scale within 2^-18 relatively (its y's error, a product and its constant's rounding);
    a code stands for its y within half a step, 2^-4 |y| or 2^-10 of the scale
    below the normal range, plus the 2^-17 by which y / scale may be off.
  - dx = s (w dy - xhat m) + dr with m a mean of 64-term thread sums: absolute
    bar 2^-17 (s |w dy| + s |xhat| mean|w dy xhat| + |dr|), plus 2^-8 |dx| where
    dx is bf16.
  - dweight: at most 64 + 4 + 32 + 32 sequential additions at these sizes:
    absolute bar 2^-16 sum|dy xhat|."""
import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 0.0}
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
WIDTHS = [1, 3, 8, 63, 512, 513, 1024, 1031, 2048, 2049, 4096, 4099, 8192, 8200, 16384, 16391, 32768]


def _t(rng, shape, dt, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _h(t):
    return t.detach().float().cpu().double().numpy()


def _close(x, ref, bar, what):
    bad = np.abs(x - ref) - bar
    assert np.isfinite(x).all() and bad.max() <= 0, f"{what}: worst excess {bad.max():.3e}"


def _check_f8(q, scale, y, what):
    s = np.max(np.abs(y), axis=-1) / 448.0
    s = np.where(s == 0, 1.0, s)
    _close(_h(scale), s, 2.0 ** -18 * s, what + " scale")
    got = _h(q) * s[..., None]
    _close(got, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[..., None]) + 2.0 ** -17 * np.abs(y), what + " codes")


@pytest.mark.parametrize("xd,rd", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_norm_every_width(D, xd, rd):
    rng = np.random.default_rng(D)
    rows = 5
    x, res, w = _t(rng, (rows, D), xd), _t(rng, (rows, D), rd, 2.0), _t(rng, (D,), F32, 0.1) + 1.0
    ref, u, rstd = ob.add_rmsnorm(_h(x), _h(w), _h(res))
    y, r, s, sc = gdn.gdn_add_rmsnorm(x, w, residual=res, return_rstd=True)
    assert y.dtype == xd and r.dtype == rd and sc is None
    _close(_h(r), u, (2.0 ** -24 + HALF[rd]) * np.abs(u), "r")
    _close(_h(s), rstd, 2.0 ** -18 * rstd, "rstd")
    _close(_h(y), ref, (2.0 ** -18 + HALF[xd] * (1 + 2.0 ** -8)) * np.abs(ref), "y")
    q, r8, none, scale = gdn.gdn_add_rmsnorm(x, w, residual=res, out_dtype=F8)
    assert none is None and torch.equal(r8, r)
    _check_f8(q, scale, ref, "y8")


@pytest.mark.parametrize("xd", [BF, F32])
@pytest.mark.parametrize("D", [1, 40, 1024, 2056, 5125])
def test_norm_without_residual_and_quantiser(D, xd):
    rng = np.random.default_rng(100 + D)
    x, w = _t(rng, (2, 3, D), xd), _t(rng, (D,), F32, 0.1) + 1.0
    y, r, s, sc = gdn.gdn_add_rmsnorm(x, w, eps=0.5)
    assert r is None and s is None and sc is None and y.shape == x.shape
    ref, _, _ = ob.add_rmsnorm(_h(x), _h(w), eps=0.5)
    _close(_h(y), ref, (2.0 ** -18 + HALF[xd] * (1 + 2.0 ** -8)) * np.abs(ref), "y")
    q, scale = gdn.gdn_quantize_rows(x)
    assert scale.shape == (2, 3)
    _check_f8(q, scale, _h(x), "q")


def test_quantiser_rounds_as_a_division_does():
    """x / scale in fp32, rounded to nearest even: the codes of torch's division and conversion, ties included
    (quotients of bf16 values fall on midpoints).  The scale is max|x| times the fp32 number nearest to 1 / 448."""
    x = _t(np.random.default_rng(7), (64, 1024), BF)
    q, scale = gdn.gdn_quantize_rows(x)
    s = x.float().abs().amax(dim=1) * (torch.ones(1, device="cuda") / torch.full((1,), 448.0, device="cuda"))
    assert torch.equal(scale, s)
    ref = (x.float() / s[:, None]).to(F8)
    assert torch.equal(q.view(torch.uint8), ref.view(torch.uint8))


def test_special_rows_stay_in_their_row():
    """Rows of zeros, of the smallest numbers, with an infinity and with a NaN: the others are as without them."""
    rng = np.random.default_rng(8)
    x, w = _t(rng, (9, 1000), F32), torch.ones(1000, device="cuda")
    plain_q, plain_s = gdn.gdn_quantize_rows(x)
    plain_y = gdn.gdn_add_rmsnorm(x, w)[0]
    x[1] = 0
    x[3, 17] = float("inf")
    x[5, 999] = float("nan")
    x[7] = 1e-44
    q, s = gdn.gdn_quantize_rows(x)
    keep = [0, 2, 4, 6, 8]
    assert torch.equal(q[keep].view(torch.uint8), plain_q[keep].view(torch.uint8)) and torch.equal(s[keep], plain_s[keep])
    assert (q[1].float() == 0).all() and s[1] == 1
    assert torch.isnan(q[3].float()[17]) and torch.isinf(s[3])
    assert torch.isnan(q[5].float()).all() and torch.isnan(s[5])
    assert torch.isfinite(q[7].float()).all() and torch.isfinite(s[7])
    y = gdn.gdn_add_rmsnorm(x, w)[0]
    assert torch.equal(y[keep], plain_y[keep]) and (y[1] == 0).all() and torch.isnan(y[5]).all()
    y8, _, _, s8 = gdn.gdn_add_rmsnorm(x, w, out_dtype=F8)
    assert (y8[1].float() == 0).all() and s8[1] == 1 and torch.isnan(y8[5].float()).all() and torch.isnan(s8[3])
    assert torch.isfinite(y8[keep].float()).all()


@pytest.mark.parametrize("D", [24, 1000, 3001])
def test_in_place_and_rows_behind(D):
    """r over residual, and buffers that go on behind the last row: nothing there changes."""
    rng = np.random.default_rng(9)
    x, res, w = _t(rng, (6, D), BF), _t(rng, (6, D), F32), _t(rng, (D,), F32)
    y0, r0, _, _ = gdn.gdn_add_rmsnorm(x, w, residual=res)
    big_r, big_y = torch.full((8, D), 7.0, device="cuda"), torch.full((8, D), 7.0, device="cuda", dtype=BF)
    big_r[:6] = res
    y, r, _, _ = gdn.gdn_add_rmsnorm(x, w, residual=big_r[:6], residual_out=big_r[:6], out=big_y[:6])
    assert torch.equal(r, r0) and torch.equal(y, y0)
    assert (big_r[6:] == 7).all() and (big_y[6:] == 7).all()


@pytest.mark.parametrize("xd,rd", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 65), (700, 512), (37, 1024), (5, 2047), (1030, 2048), (9, 4096), (3, 8192),
                                    (4, 16384), (2, 32767), (1500, 8), (600, 5125), (3, 6143)])
def test_norm_bwd(rows, D, xd, rd):
    rng = np.random.default_rng(rows + D)
    dy, r, dr = _t(rng, (rows, D), xd), _t(rng, (rows, D), rd, 2.0), _t(rng, (rows, D), rd)
    w = _t(rng, (D,), F32, 0.1) + 1.0
    rstd = torch.from_numpy(ob.add_rmsnorm(_h(r), _h(w))[2].astype(np.float32)).cuda()
    for d in (None, dr):
        dx, dw = gdn.gdn_add_rmsnorm_bwd(dy, r, w, rstd, dr=d)
        rx, rw = ob.add_rmsnorm_bwd(_h(dy), _h(r), _h(w), _h(rstd), None if d is None else _h(d))
        xhat, s = _h(r) * _h(rstd)[:, None], _h(rstd)[:, None]
        g = np.abs(_h(dy) * _h(w))
        mag = s * g + s * np.abs(xhat) * np.mean(g * np.abs(xhat), axis=1, keepdims=True)
        if d is not None:
            mag = mag + np.abs(_h(d))
        _close(_h(dx), rx, 2.0 ** -17 * mag + HALF[rd] * np.abs(rx), "dx")
        _close(_h(dw), rw, 2.0 ** -16 * np.sum(np.abs(_h(dy) * xhat), axis=0), "dweight")
    again = gdn.gdn_add_rmsnorm_bwd(dy, r, w, rstd, dr=dr)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)      # repeats bit for bit
    dx2, none = gdn.gdn_add_rmsnorm_bwd(dy, r, w, rstd, dr=dr, need_dweight=False)
    assert none is None and torch.equal(dx2, dx)


def test_norm_captured_and_replayed():
    """Forward and backward in a captured graph, replayed on new inputs with eager work between."""
    rng = np.random.default_rng(11)
    rows, D = 300, 1024
    x, res, dy = (_t(rng, (rows, D), BF) for _ in range(3))
    w = _t(rng, (D,), F32, 0.1) + 1.0

    def step():
        y, r, s, _ = gdn.gdn_add_rmsnorm(x, w, residual=res, return_rstd=True)
        q, _, _, sc = gdn.gdn_add_rmsnorm(x, w, residual=res, out_dtype=F8)
        dx, dw = gdn.gdn_add_rmsnorm_bwd(dy, r, w, s)
        return y, r, q.view(torch.uint8), sc, dx, dw

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(_t(rng, (rows, D), BF))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
