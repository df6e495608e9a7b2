"""The fp64 definitions of the convolution and the scan against forms that share nothing with them: numpy's
convolution, the closed sum of the recurrence, and the two halves of a sequence."""
import numpy as np

from oracle import scan as os_


def test_conv_is_a_convolution():
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((2, 9, 3)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    y, state = os_.causal_conv(x, w, b, act="none")
    for i in range(2):
        for c in range(3):
            np.testing.assert_allclose(y[i, :, c], b[c] + np.convolve(x[i, :, c], w[c, ::-1])[:9], atol=1e-12)
    np.testing.assert_array_equal(state, x[:, -3:])
    y1, s1 = os_.causal_conv(x[:, :2], w, b, act="none")
    y2, s2 = os_.causal_conv(x[:, 2:], w, b, s1, act="none")
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, atol=1e-12)
    np.testing.assert_array_equal(s2, state)


def test_scan_is_its_closed_sum():
    rng = np.random.default_rng(1)
    T, ch, N = 7, 3, 2
    x, dt = rng.standard_normal((1, T, ch)), rng.standard_normal((1, T, ch))
    B, C = rng.standard_normal((1, T, N)), rng.standard_normal((1, T, N))
    A, h0 = -np.exp(rng.standard_normal((ch, N))), rng.standard_normal((1, ch, N))
    y, h, _, _ = os_.selective_scan(x, dt, A, B, C, h0=h0)
    d = np.log(1 + np.exp(dt))[0]
    for t in range(T):
        want = np.exp(A * d[:t + 1].sum(axis=0)[:, None]) * h0[0]
        for s in range(t + 1):
            decay = np.exp(A * d[s + 1:t + 1].sum(axis=0)[:, None])
            want = want + decay * (d[s] * x[0, s])[:, None] * B[0, s]
        np.testing.assert_allclose(y[0, t], want @ C[0, t], atol=1e-10)
    np.testing.assert_allclose(h[0], want, atol=1e-10)


def test_scan_in_two_halves_with_skip_and_gate():
    rng = np.random.default_rng(2)
    n, T, ch, N = 2, 8, 5, 4
    x, dt, z = (rng.standard_normal((n, T, ch)) for _ in range(3))
    B, C = rng.standard_normal((n, T, N)), rng.standard_normal((n, T, N))
    A, D, b = -np.exp(rng.standard_normal((ch, N))), rng.standard_normal(ch), rng.standard_normal(ch)
    y, h, _, _ = os_.selective_scan(x, dt, A, B, C, D, z, b)
    f = lambda s, h0: os_.selective_scan(x[:, s], dt[:, s], A, B[:, s], C[:, s], D, z[:, s], b, h0)  # noqa: E731
    y1, h1, _, _ = f(slice(0, 3), None)
    y2, h2, _, _ = f(slice(3, T), h1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, atol=1e-12)
    np.testing.assert_allclose(h2, h, atol=1e-12)
