"""GPU parity of the residual layer norm and its backward, through the public
calls, against the fp64 definitions in oracle/block.py.

Tolerances.  The kernels compute in fp32 and round each output once.
  - r = x + residual: one correctly rounded addition, 2^-24 |r| (2^-8 for bf16).
  - m: a thread adds at most 32 values, then at most 6 + 16 partial sums, and
    divides: 55 * 2^-24 of mean|u|, below 2^-18 A with A = mean|u|.
  - s: the differences d = u - m are all off by the same 2^-18 A and by 2^-24 of
    themselves; a common shift c adds c^2 to their mean square, which is below
    2^-19 of it where A <= 2^8 sigma (the test data); the squares add up like
    those of the RMS norm: 2^-18 relatively.
  - y = d s w + b: s |w| 2^-18 A, 2^-17 of |d s w| (s and four roundings), 2^-24 |y|;
    plus 2^-8 |y| where y is bf16.
  - 8 bits: scale within the bar of the largest y; a code within half a step.
  - dx at the given m and s: means of 64-term thread sums, absolute bar
    2^-17 s (|a| + mean|a| + |xhat| mean|a xhat|) + 2^-17 |dr|, plus 2^-8 |dx|
    in bf16; dweight, dbias: at most 132 sequential additions at these sizes,
    2^-16 sum|dy xhat| and 2^-16 sum|dy|."""
import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 0.0}
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
WIDTHS = [2, 3, 8, 63, 512, 513, 1024, 1031, 2048, 2049, 4096, 4099, 8192, 8200, 16384, 16391, 32768]


def _t(rng, shape, dt, scale=1.0, shift=0.0):
    return torch.from_numpy((shift + scale * rng.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _h(t):
    return t.detach().float().cpu().double().numpy()


def _close(x, ref, bar, what):
    bad = np.abs(x - ref) - bar
    assert np.isfinite(x).all() and bad.max() <= 0, f"{what}: worst excess {bad.max():.3e}"


def _bar(ref, u, b, s, w):
    """Bar of y before its rounding."""
    A = np.mean(np.abs(u), axis=-1, keepdims=True)
    b = 0.0 if b is None else b
    return s[..., None] * np.abs(w) * 2.0 ** -18 * A + 2.0 ** -17 * np.abs(ref - b) + 2.0 ** -24 * np.abs(ref)


def _check_f8(q, scale, y, bar, what):
    top = np.argmax(np.abs(y), axis=-1)
    amax = np.take_along_axis(np.abs(y), top[..., None], -1)[..., 0]
    s = np.where(amax == 0, 1.0, amax / 448.0)
    slack = bar.max(axis=-1) / 448.0 + 2.0 ** -22 * s
    _close(_h(scale), s, slack, what + " scale")
    got = _h(q) * _h(scale)[..., None]
    _close(got, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[..., None]) + 2 * bar + 2.0 ** -20 * np.abs(y),
           what + " codes")


@pytest.mark.parametrize("xd,rd", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_layernorm_every_width(D, xd, rd):
    rng = np.random.default_rng(D)
    rows = 5
    x, res = _t(rng, (rows, D), xd), _t(rng, (rows, D), rd, 2.0, 3.0)
    w, b = _t(rng, (D,), F32, 0.1, 1.0), _t(rng, (D,), F32)
    ref, u, mean, rstd = ob.add_layernorm(_h(x), _h(w), _h(b), _h(res))
    y, r, m, s, sc = gdn.gdn_add_layernorm(x, w, bias=b, residual=res, return_stats=True)
    assert y.dtype == xd and r.dtype == rd and sc is None
    _close(_h(r), u, (2.0 ** -24 + HALF[rd]) * np.abs(u), "r")
    _close(_h(m), mean, 2.0 ** -18 * np.mean(np.abs(u), axis=-1), "mean")
    _close(_h(s), rstd, 2.0 ** -17 * rstd, "rstd")
    bar = _bar(ref, u, _h(b), rstd, _h(w))
    _close(_h(y), ref, bar + HALF[xd] * (np.abs(ref) + bar), "y")
    q, r8, none, none2, scale = gdn.gdn_add_layernorm(x, w, bias=b, residual=res, out_dtype=F8)
    assert none is None and none2 is None and torch.equal(r8, r)
    _check_f8(q, scale, ref, bar, "y8")


@pytest.mark.parametrize("xd", [BF, F32])
@pytest.mark.parametrize("D", [1, 40, 1024, 2056, 5125])
def test_layernorm_without_residual_or_bias(D, xd):
    rng = np.random.default_rng(100 + D)
    x, w = _t(rng, (2, 3, D), xd), _t(rng, (D,), F32, 0.1, 1.0)
    y, r, m, s, sc = gdn.gdn_add_layernorm(x, w, eps=0.5)
    assert r is None and m is None and s is None and sc is None and y.shape == x.shape
    ref, u, _, rstd = ob.add_layernorm(_h(x), _h(w), eps=0.5)
    bar = _bar(ref, u, None, rstd, _h(w))
    _close(_h(y), ref, bar + HALF[xd] * (np.abs(ref) + bar), "y")


def test_a_large_mean_leaves_the_spread():
    """A row of 4096 + k / 16: fp32 holds every sum and difference to the mean, the difference of the moments would
    not hold the variance."""
    x = (4096.0 + torch.arange(1024, device="cuda") % 64 / 16.0)[None].contiguous()
    y, _, m, s, _ = gdn.gdn_add_layernorm(x, torch.ones(1024, device="cuda"), return_stats=True)
    ref, _, mean, rstd = ob.add_layernorm(_h(x), np.ones(1024))
    _close(_h(m), mean, 2.0 ** -24 * mean, "mean")
    _close(_h(s), rstd, 2.0 ** -17 * rstd, "rstd")
    _close(_h(y), ref, 2.0 ** -17 * np.abs(ref) + 2.0 ** -23 * mean * rstd, "y")


def test_the_mean_is_kept_beyond_its_rounding():
    """Rows whose mean fp32 rounds (values around 1e4 + 1/3): the differences' own sum takes the rounding out again, so
    y is as near as the differences themselves allow, 2^-24 of the values' size each."""
    rng = np.random.default_rng(12)
    x = _t(rng, (7, 4099), F32, 1.0) + 10000.0 + 1.0 / 3.0
    y, _, m, s, _ = gdn.gdn_add_layernorm(x, torch.ones(4099, device="cuda"), return_stats=True)
    ref, _, mean, rstd = ob.add_layernorm(_h(x), np.ones(4099))
    _close(_h(m), mean, 2.0 ** -23 * mean, "mean")
    _close(_h(s), rstd, 2.0 ** -17 * rstd, "rstd")
    # x - m is exact here (both within a factor of two, multiples of 2^-10); off by at most 2^-18 of itself after the
    # correction, whose sum has the error of 4099 additions of differences
    _close(_h(y), ref, 2.0 ** -16 * np.maximum(np.abs(ref), 1.0), "y")


def test_special_rows_stay_in_their_row():
    """Rows of one value, with an infinity and with a NaN: the others are as without them."""
    rng = np.random.default_rng(8)
    x, w = _t(rng, (9, 1000), F32), torch.ones(1000, device="cuda")
    plain = gdn.gdn_add_layernorm(x, w)[0]
    x[1] = 0
    x[2] = 3.0
    x[3, 17] = float("inf")
    x[5, 999] = float("nan")
    keep = [0, 4, 6, 7, 8]
    y = gdn.gdn_add_layernorm(x, w)[0]
    assert torch.equal(y[keep], plain[keep]) and (y[1:3] == 0).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    q, _, _, _, s = gdn.gdn_add_layernorm(x, w, out_dtype=F8)
    assert (q[1:3].float() == 0).all() and (s[1:3] == 1).all() and torch.isnan(s[3]) and torch.isnan(q[5].float()).all()
    assert torch.isfinite(q[keep].float()).all()


@pytest.mark.parametrize("D", [24, 1000, 3001])
def test_in_place_and_rows_behind(D):
    """r over residual, and buffers that go on behind the last row: nothing there changes."""
    rng = np.random.default_rng(9)
    x, res, w = _t(rng, (6, D), BF), _t(rng, (6, D), F32), _t(rng, (D,), F32)
    y0, r0 = gdn.gdn_add_layernorm(x, w, residual=res)[:2]
    big_r, big_y = torch.full((8, D), 7.0, device="cuda"), torch.full((8, D), 7.0, device="cuda", dtype=BF)
    big_r[:6] = res
    y, r = gdn.gdn_add_layernorm(x, w, residual=big_r[:6], residual_out=big_r[:6], out=big_y[:6])[:2]
    assert torch.equal(r, r0) and torch.equal(y, y0)
    assert (big_r[6:] == 7).all() and (big_y[6:] == 7).all()


@pytest.mark.parametrize("xd,rd", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 65), (700, 512), (37, 1024), (5, 2047), (1030, 2048), (9, 4096), (3, 8192),
                                    (4, 16384), (2, 32767), (1500, 8), (600, 5125), (3, 6143)])
def test_layernorm_bwd(rows, D, xd, rd):
    rng = np.random.default_rng(rows + D)
    dy, r, dr = _t(rng, (rows, D), xd), _t(rng, (rows, D), rd, 2.0, 1.0), _t(rng, (rows, D), rd)
    w = _t(rng, (D,), F32, 0.1, 1.0)
    _, _, m, s = ob.add_layernorm(_h(r), _h(w))
    mean, rstd = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (m, s))
    for d in (None, dr):
        dx, dw, db = gdn.gdn_add_layernorm_bwd(dy, r, w, mean, rstd, dr=d)
        rx, rw, rb = ob.add_layernorm_bwd(_h(dy), _h(r), _h(w), _h(mean), _h(rstd), None if d is None else _h(d))
        xhat, sc = np.abs((_h(r) - _h(mean)[:, None]) * _h(rstd)[:, None]), _h(rstd)[:, None]
        a = np.abs(_h(dy) * _h(w))
        mag = sc * (a + np.mean(a, axis=1, keepdims=True) + xhat * np.mean(a * xhat, axis=1, keepdims=True))
        if d is not None:
            mag = mag + np.abs(_h(d))
        _close(_h(dx), rx, 2.0 ** -17 * mag + HALF[rd] * np.abs(rx), "dx")
        _close(_h(dw), rw, 2.0 ** -16 * np.sum(np.abs(_h(dy)) * xhat, axis=0), "dweight")
        _close(_h(db), rb, 2.0 ** -16 * np.sum(np.abs(_h(dy)), axis=0), "dbias")
    again = gdn.gdn_add_layernorm_bwd(dy, r, w, mean, rstd, dr=dr)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))      # repeats bit for bit
    for nw, nb in ((False, False), (True, False), (False, True)):
        x2, w2, b2 = gdn.gdn_add_layernorm_bwd(dy, r, w, mean, rstd, dr=dr, need_dweight=nw, need_dbias=nb)
        assert torch.equal(x2, dx) and (w2 is None) == (not nw) and (b2 is None) == (not nb)
        assert w2 is None or torch.equal(w2, dw)
        assert b2 is None or torch.equal(b2, db)


def test_layernorm_captured_and_replayed():
    """Forward and backward in a captured graph, replayed on new inputs with eager work between."""
    rng = np.random.default_rng(11)
    rows, D = 300, 1024
    x, res, dy = (_t(rng, (rows, D), BF) for _ in range(3))
    w, b = _t(rng, (D,), F32, 0.1, 1.0), _t(rng, (D,), F32)

    def step():
        y, r, m, s, _ = gdn.gdn_add_layernorm(x, w, bias=b, residual=res, return_stats=True)
        q, _, _, _, sc = gdn.gdn_add_layernorm(x, w, bias=b, residual=res, out_dtype=F8)
        return (y, r, q.view(torch.uint8), sc) + gdn.gdn_add_layernorm_bwd(dy, r, w, m, s)

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
        for a, c in zip(out, step()):
            assert torch.equal(a, c)
        torch.cuda.synchronize()


def test_the_binding_refuses():
    x, w = torch.zeros(4, 64, device="cuda", dtype=BF), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_add_layernorm(x.t(), w)
    with pytest.raises(ValueError):
        gdn.gdn_add_layernorm(x, w, bias=torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        gdn.gdn_add_layernorm(x, w.to(BF))
    with pytest.raises(ValueError):
        gdn.gdn_add_layernorm(x, w, residual_out=x)
    with pytest.raises(RuntimeError):
        gdn.gdn_add_layernorm(x, w, eps=0.0)
    with pytest.raises(RuntimeError):
        gdn.gdn_add_layernorm(x, w, out_dtype=F32)
    with pytest.raises(ValueError):
        gdn.gdn_add_layernorm_bwd(x, x, w, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"))
