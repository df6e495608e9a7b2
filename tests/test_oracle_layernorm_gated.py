"""The fp64 definitions of the layer norm and the gated projection: the
gradients against central differences, and the forms that have to agree."""
import numpy as np
import pytest

from oracle import block as ob


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_layernorm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, res, dy, dr = (rng.standard_normal((3, 7)) for _ in range(4))
    w, b = 1 + 0.3 * rng.standard_normal(7), rng.standard_normal(7)

    def loss(x, w, b):
        y, u, _, _ = ob.add_layernorm(x, w, b, res)
        return np.sum(dy * y) + np.sum(dr * u)

    _, u, mean, rstd = ob.add_layernorm(x, w, b, res)
    dx, dw, db = ob.add_layernorm_bwd(dy, u, w, mean, rstd, dr)
    np.testing.assert_allclose(dx, _differences(lambda t: loss(t, w, b), x), atol=1e-7)
    np.testing.assert_allclose(dw, _differences(lambda t: loss(x, t, b), w), atol=1e-7)
    np.testing.assert_allclose(db, _differences(lambda t: loss(x, w, t), b), atol=1e-7)


def test_layernorm_of_a_centred_row_is_the_rms_norm():
    x = np.random.default_rng(1).standard_normal((4, 9))
    x -= x.mean(axis=1, keepdims=True)
    w = np.arange(1.0, 10.0)
    np.testing.assert_allclose(ob.add_layernorm(x, w)[0], ob.add_rmsnorm(x, w)[0], rtol=1e-12)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_gated_gradients_against_differences(name):
    rng = np.random.default_rng(2)
    x, w, b, dy = rng.standard_normal((4, 5)), rng.standard_normal((6, 5)), rng.standard_normal(6), rng.standard_normal((4, 3))
    loss = lambda x, w, b: np.sum(dy * ob.gated_linear(x, w, b, name)[0])  # noqa: E731
    _, z = ob.gated_linear(x, w, b, name)
    dx, dw, db, _ = ob.gated_linear_bwd(dy, x, w, z, name)
    np.testing.assert_allclose(dx, _differences(lambda t: loss(t, w, b), x), atol=1e-6)
    np.testing.assert_allclose(dw, _differences(lambda t: loss(x, t, b), w), atol=1e-6)
    np.testing.assert_allclose(db, _differences(lambda t: loss(x, w, t), b), atol=1e-6)
