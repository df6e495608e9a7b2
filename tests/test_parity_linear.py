"""GPU parity of gdn_linear and gdn_linear_bwd, through the public calls,
against the fp64 definitions in oracle/block.py.

Most shapes run on small whole numbers, whose products and sums are exact in
fp32 in any order (all partial sums stay below 2^24): fp32 outputs have to be
equal, bf16 outputs equal to the rounded exact value.  A missing, doubled or
misplaced product cannot hide in a tolerance.

Random values.  fp32 sums of K products: |error| <= K 2^-24 sum|x w| (one
rounding per addition), dz likewise.  Activations: sigmoid's exponent argument
is off by 2^-23 |z|, its exp2, sum, reciprocal and product by five roundings
of at most 2 ulp (2^-22): bar (2^-22 |z| + 2^-20) |act(z)| and, for the
error of z itself, |act'| <= 1.13 times it; erf within 2^-21 absolutely, that is
2^-21 |z| for gelu.  Rounding to bf16: 2^-8 of the value."""
import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 0.0}
ACTS = ("none", "relu", "silu", "gelu")


def _ints(rng, shape, top, dt):
    return torch.from_numpy(rng.integers(-top, top + 1, shape).astype(np.float32)).to(dt).cuda()


def _t(rng, shape, dt, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _h(t):
    return t.detach().float().cpu().double().numpy()


def _rounded(ref, dt):
    return torch.from_numpy(ref).float().to(dt).float().double().numpy()


def _close(x, ref, bar, what):
    bad = np.abs(x - ref) - bar
    assert np.isfinite(x).all() and bad.max() <= 0, f"{what}: worst excess {bad.max():.3e}"


# one row, one column, one slab; each kernel's tile edge and both sides of it; sums split in parts; whole large tiles
SHAPES = [(1, 1, 8), (1, 5, 64), (2, 64, 72), (3, 129, 1024), (15, 16, 520), (16, 4096, 64), (17, 255, 136), (31, 33, 4096),
          (33, 1000, 256), (64, 64, 8192), (65, 130, 64), (127, 128, 192), (128, 127, 128), (129, 257, 1024), (255, 300, 48),
          (256, 256, 64), (3000, 16, 264), (5000, 17, 64), (257, 513, 1032), (1000, 8, 1024), (8, 1031, 1024), (640, 4104, 160), (4097, 4099, 56),
          (4096, 4096, 128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_exact_in_bf16(M, N, K):
    rng = np.random.default_rng(M + N + K)
    x, w = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF)
    b, res = _ints(rng, (N,), 9, F32), _ints(rng, (M, N), 9, F32)
    ref, z = ob.linear(_h(x), _h(w), _h(b), _h(res), "relu")
    y, zz = gdn.gdn_linear(x, w, bias=b, residual=res, act="relu", out_dtype=F32, return_preact=True)
    np.testing.assert_array_equal(_h(y), ref)
    np.testing.assert_array_equal(_h(zz), _rounded(z, BF))
    y, none = gdn.gdn_linear(x, w)
    assert none is None and y.dtype == BF
    np.testing.assert_array_equal(_h(y), _rounded(_h(x) @ _h(w).T, BF))


@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[2] % 16 == 0])
def test_linear_exact_in_8_bits(M, N, K):
    rng = np.random.default_rng(M + N + K)
    x, w = _ints(rng, (M, K), 3, F32).to(F8), _ints(rng, (N, K), 3, F32).to(F8)
    xs = torch.from_numpy(2.0 ** rng.integers(-3, 4, M)).float().cuda()
    ws = torch.from_numpy(2.0 ** rng.integers(-3, 4, N)).float().cuda()
    ref, _ = ob.linear(_h(x), _h(w), None, None, "none", _h(xs), _h(ws))
    y, _ = gdn.gdn_linear(x, w, x_scale=xs, w_scale=ws, out_dtype=F32)
    np.testing.assert_array_equal(_h(y), ref)
    res = _ints(rng, (M, N), 9, BF)
    y, _ = gdn.gdn_linear(x, w, x_scale=xs, w_scale=ws, residual=res)
    np.testing.assert_array_equal(_h(y), _rounded(ref + _h(res), BF))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_bwd_exact(M, N, K):
    rng = np.random.default_rng(M + N + K)
    x, w, dy = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF), _ints(rng, (M, N), 3, BF)
    rx, rw, rb, _ = ob.linear_bwd(_h(dy), _h(x), _h(w))
    dx, dw, db = gdn.gdn_linear_bwd(dy, x, w, bias=True, grad_dtype=F32)
    np.testing.assert_array_equal(_h(dx), rx)
    np.testing.assert_array_equal(_h(dw), rw)
    np.testing.assert_array_equal(_h(db), rb)
    dx, dw, db = gdn.gdn_linear_bwd(dy, x, w)
    assert db is None
    np.testing.assert_array_equal(_h(dx), _rounded(rx, BF))
    np.testing.assert_array_equal(_h(dw), _rounded(rw, BF))


@pytest.mark.parametrize("M,N,K", [(1, 3, 8), (70, 130, 136), (300, 515, 264), (2000, 24, 64)])
def test_linear_bwd_keeps_fp32_gradients_of_an_inexact_dz(M, N, K):
    """dy in fp32 with 23 significant bits: three bf16 parts carry it (one number per row of dy, so that sums are
    exact too), through a relu whose argument decides the sign."""
    rng = np.random.default_rng(M)
    x, w = _ints(rng, (M, K), 1, BF), torch.zeros(N, K, dtype=BF, device="cuda")
    w[:, 0] = 1
    z = _ints(rng, (M, N), 2, BF)
    dy = torch.zeros(M, N, device="cuda")
    col = torch.from_numpy(rng.integers(0, N, M)).cuda()
    dy[torch.arange(M), col] = torch.from_numpy((2.0 ** 22 + rng.integers(0, 2 ** 22, M)).astype(np.float32)).cuda()
    z[torch.arange(M), col] = torch.from_numpy(np.where(rng.random(M) < 0.5, 1.0, -1.0)).to(BF).cuda()
    rx, rw, rb, _ = ob.linear_bwd(_h(dy), _h(x), _h(w), _h(z), "relu")
    dx, dw, db = gdn.gdn_linear_bwd(dy, x, w, z=z, act="relu", bias=True, grad_dtype=F32)
    np.testing.assert_array_equal(_h(dx), rx)
    bar = M * 2.0 ** -24 * (np.abs(_h(dy)).T @ np.abs(_h(x)))
    _close(_h(dw), rw, bar, "dw")
    _close(_h(db), rb, M * 2.0 ** -24 * np.abs(_h(dy)).sum(0), "dbias")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (33, 77, 264), (300, 640, 512)])
def test_linear_random(M, N, K, out, act):
    rng = np.random.default_rng(M + N)
    x, w = _t(rng, (M, K), BF, 2.0), _t(rng, (N, K), BF, K ** -0.5)
    b, res = _t(rng, (N,), F32), _t(rng, (M, N), out)
    ref, z = ob.linear(_h(x), _h(w), _h(b), _h(res), act)
    y, zz = gdn.gdn_linear(x, w, bias=b, residual=res, act=act, out_dtype=out, return_preact=True)
    ez = (K + 2) * 2.0 ** -24 * (np.abs(_h(x)) @ np.abs(_h(w)).T + np.abs(_h(b)))
    _close(_h(zz), z, ez + 2.0 ** -8 * np.abs(z), "z")
    a = np.abs(ob.act(act, z))
    ea = 1.13 * ez + (2.0 ** -22 * np.abs(z) + 2.0 ** -20) * a + 2.0 ** -21 * np.abs(z)
    _close(_h(y), ref, ea + 2.0 ** -23 * np.abs(ref) + HALF[out] * np.abs(ref), "y")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dyt,grad", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("M,N,K", [(1, 512, 64), (33, 77, 264), (300, 640, 512)])
def test_linear_bwd_random(M, N, K, dyt, grad, act):
    """dz is off by its own arithmetic (about ten roundings, 2^-20 (1 + |z|) of |dy|), and by 2^-8 |dz| where it is rounded to bf16; the three
    bf16 parts of an fp32 dz leave 2^-24 of it."""
    rng = np.random.default_rng(M + N)
    x, w, dy = _t(rng, (M, K), BF), _t(rng, (N, K), BF, K ** -0.5), _t(rng, (M, N), dyt)
    z = _t(rng, (M, N), BF, 2.0) if act != "none" else None
    rx, rw, rb, dz = ob.linear_bwd(_h(dy), _h(x), _h(w), None if z is None else _h(z), act)
    dx, dw, db = gdn.gdn_linear_bwd(dy, x, w, z=z, act=act, bias=True, grad_dtype=grad)
    e0 = 2.0 ** -20 * np.abs(_h(dy)) * (1 + (0 if z is None else np.abs(_h(z)))) if act != "none" else 0 * dz
    exact = act == "none" and dyt == BF
    e = e0 + (0 if exact else (2.0 ** -8 if grad == BF else 2.0 ** -23) * np.abs(dz))
    n = 3 * 2.0 ** -24
    _close(_h(dx), rx, e @ np.abs(_h(w)) + n * N * (np.abs(dz) @ np.abs(_h(w))) + HALF[grad] * np.abs(rx), "dx")
    _close(_h(dw), rw, e.T @ np.abs(_h(x)) + n * M * (np.abs(dz).T @ np.abs(_h(x))) + HALF[grad] * np.abs(rw), "dw")
    _close(_h(db), rb, e0.sum(0) + M * 2.0 ** -24 * np.abs(dz).sum(0), "dbias")


def test_gradients_equal_differences_of_the_forward():
    """Central differences of the fp32-output forward in one direction per operand.  Steps h on values of order 1 in
    bf16: the perturbed operands are exact (multiples of 2^-6 below 2), so a difference of losses is off by the
    forward's fp32 error over h, and by h^2 / 6 times the third derivative (silu: below 0.5 |direction|^3)."""
    rng = np.random.default_rng(21)
    M, N, K = 24, 40, 64
    grid = lambda shape, s: (torch.from_numpy(rng.integers(-24, 25, shape) / 64.0 * s).float()).to(BF).cuda()  # noqa: E731
    x, w, b = grid((M, K), 1.0), grid((N, K), 1.0), _t(rng, (N,), F32)
    dy = _t(rng, (M, N), F32)
    loss = lambda x_, w_, b_: float((gdn.gdn_linear(x_, w_, bias=b_, act="silu", out_dtype=F32)[0].double() * dy.double()).sum())  # noqa: E731
    _, z = gdn.gdn_linear(x, w, bias=b, act="silu", out_dtype=F32, return_preact=True)
    dx, dw, db = gdn.gdn_linear_bwd(dy, x, w, z=z, act="silu", bias=True, grad_dtype=F32)
    h = 2.0 ** -6
    zf = ob.linear(_h(x), _h(w), _h(b))[1]
    for which, g, t in (("x", dx, x), ("w", dw, w), ("b", db, b)):
        d = torch.zeros_like(t)
        i = tuple(int(rng.integers(0, n)) for n in t.shape)
        d[i] = h
        args = lambda s: [t + s * d if k == which else v for k, v in (("x", x), ("w", w), ("b", b))]  # noqa: E731
        diff = (loss(*args(1)) - loss(*args(-1))) / (2 * h)
        dzd = {"x": _h(w)[:, i[-1]][None, :] * (np.arange(M) == i[0])[:, None] if which == "x" else 0,
               "w": _h(x)[:, i[-1]][:, None] * (np.arange(N) == i[0])[None, :] if which == "w" else 0,
               "b": (np.arange(N) == i[0])[None, :] * np.ones((M, 1))}[which]
        a = np.abs(_h(dy) * dzd)
        # z is kept in bf16: the derivative is taken 2^-8 |z| away, |silu''| <= 1/2
        bar = (a * 2.0 ** -8 * np.abs(zf) / 2).sum() + h * h / 6 * 0.5 * (np.abs(_h(dy)) * np.abs(dzd) ** 3).sum()
        bar += 2.0 ** -20 * (np.abs(_h(dy)) * (dzd != 0) * (1 + np.abs(zf))).sum() / h + 2.0 ** -18 * a.sum()
        assert abs(diff - float(g[i])) <= bar, (which, diff, float(g[i]), bar)


def test_infinities_and_nan_stay_in_their_row_and_column():
    rng = np.random.default_rng(22)
    M, N, K = 150, 140, 200
    x, w = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF)
    clean = gdn.gdn_linear(x, w, out_dtype=F32)[0]
    x[7, 199] = float("nan")
    x[149, 0] = float("inf")
    w[139, 100] = float("nan")
    y = gdn.gdn_linear(x, w, out_dtype=F32)[0]
    keep_i = [i for i in range(M) if i not in (7, 149)]
    assert torch.equal(y[keep_i][:, :139], clean[keep_i][:, :139])
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 139]).all() and not torch.isfinite(y[149]).any()


@pytest.mark.parametrize("M,out", [(20, BF), (20, F32), (200, BF), (200, F32)])
def test_infinities_and_nan_in_8_bits(M, out):
    """A NaN code spoils its row (its column, in the weights) and nothing else; an infinite scale gives infinities."""
    rng = np.random.default_rng(27)
    N, K = 150, 208
    x, w = _ints(rng, (M, K), 3, F32), _ints(rng, (N, K), 3, F32)
    xs, ws = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    x[:, 0] = 1
    clean = gdn.gdn_linear(x.to(F8), w.to(F8), x_scale=xs, w_scale=ws, out_dtype=out)[0]
    x[7, 207], w[149, 100] = float("nan"), float("nan")
    xs[11] = float("inf")
    y = gdn.gdn_linear(x.to(F8), w.to(F8), x_scale=xs, w_scale=ws, out_dtype=out)[0]
    keep = [i for i in range(M) if i not in (7, 11)]
    assert torch.equal(y[keep][:, :149], clean[keep][:, :149])
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 149]).all() and not torch.isfinite(y[11]).any()


@pytest.mark.parametrize("M,N", [(5, 37), (130, 136), (600, 1100)])
def test_in_place_and_rows_behind(M, N):
    rng = np.random.default_rng(23)
    K = 256
    x, w, res = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF), _ints(rng, (M, N), 9, F32)
    want = gdn.gdn_linear(x, w, residual=res, out_dtype=F32)[0]
    big = torch.full((M + 3, N), 7.0, device="cuda")
    big[:M] = res
    y, _ = gdn.gdn_linear(x, w, residual=big[:M], out_dtype=F32, out=big[:M])
    assert torch.equal(y, want) and (big[M:] == 7).all()


def test_repeats_bit_for_bit_and_captured():
    """Split sums, both tile sizes and the backward: the same bits each time, eager and in replays of a captured
    graph on new inputs."""
    rng = np.random.default_rng(24)
    x, w, w2 = _t(rng, (200, 1024), BF), _t(rng, (520, 1024), BF, 0.03), _t(rng, (1024, 520), BF, 0.03)
    b = _t(rng, (520,), F32)

    def step():
        h, z = gdn.gdn_linear(x, w, bias=b, act="silu", return_preact=True)
        y, _ = gdn.gdn_linear(h, w2, residual=x)
        dh, dw2, _ = gdn.gdn_linear_bwd(y, h, w2)
        dx, dw, db = gdn.gdn_linear_bwd(dh, x, w, z=z, act="silu", bias=True, grad_dtype=F32)
        return h, z, y, dh, dw2, dx, dw, db

    first = step()
    for a, c in zip(first, step()):
        assert torch.equal(a, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(_t(rng, (200, 1024), BF))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, step()):
            assert torch.equal(a, c)
        torch.cuda.synchronize()


def test_another_stream():
    rng = np.random.default_rng(25)
    x, w = _ints(rng, (300, 512), 3, BF), _ints(rng, (260, 512), 3, BF)
    want = gdn.gdn_linear(x, w, out_dtype=F32)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = gdn.gdn_linear(x, w, out_dtype=F32)[0]
        dx = gdn.gdn_linear_bwd(y, x, w, need_dw=False)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    assert torch.equal(dx, gdn.gdn_linear_bwd(want, x, w, need_dw=False)[0])


def test_two_streams_at_once():
    """Split sums and paired gradients on two streams, each call with its own workspace."""
    rng = np.random.default_rng(27)
    work = []
    for _ in range(2):
        x, w, dy = _ints(rng, (200, 4096), 2, BF), _ints(rng, (520, 4096), 2, BF), _ints(rng, (200, 520), 2, BF)
        work.append((x, w, dy, gdn.gdn_linear(x, w, out_dtype=F32)[0], gdn.gdn_linear_bwd(dy, x, w, bias=True)))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k, (x, w, dy, _, _) in enumerate(work):
            with torch.cuda.stream(side[k]):
                got[k].append((gdn.gdn_linear(x, w, out_dtype=F32)[0], gdn.gdn_linear_bwd(dy, x, w, bias=True)))
    torch.cuda.synchronize()
    for k, (_, _, _, y, grads) in enumerate(work):
        for a, b in got[k]:
            assert torch.equal(a, y) and all(torch.equal(u, v) for u, v in zip(b, grads))


@pytest.mark.parametrize("M,N,K", [(5, 4105, 64), (5, 8203, 1024), (16, 9001, 2064), (30, 4105, 1040), (30, 8203, 528),
                                   (50, 4105, 1040), (50, 8203, 528), (64, 8192, 1024), (3, 70, 16400)])
def test_few_rows_of_many_columns(M, N, K):
    """Each cut of the kernel for few rows, with whole and partial last pieces, exactly."""
    rng = np.random.default_rng(28)
    x, w = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF)
    want = _h(x) @ _h(w).T
    assert np.array_equal(_h(gdn.gdn_linear(x, w, out_dtype=F32)[0]), want)
    if K % 16 == 0:
        one = lambda n: torch.ones(n, device="cuda")
        y, _ = gdn.gdn_linear(x.to(F8), w.to(F8), x_scale=one(M), w_scale=one(N), out_dtype=F32)
        assert np.array_equal(_h(y), want)


@pytest.mark.parametrize("M,N", [(1_100_003, 2056), (2056, 1_100_003)])
def test_offsets_past_2_to_the_31(M, N):
    """Outputs of 2.26e9 values: the corners against the same rows and columns computed alone."""
    need = M * N * 2 * 1.1
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs %.0f GB of device memory" % (need / 1e9))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    K = 64
    x = torch.randint(-3, 4, (M, K), generator=gen, device="cuda").to(BF)
    w = torch.randint(-3, 4, (N, K), generator=gen, device="cuda").to(BF)
    y = gdn.gdn_linear(x, w)[0]
    for i in (0, M // 2, M - 40):
        for j in (0, N // 2, N - 40):
            ref = x[i:i + 40].float() @ w[j:j + 40].float().t()
            assert torch.equal(y[i:i + 40, j:j + 40], ref.to(BF))
