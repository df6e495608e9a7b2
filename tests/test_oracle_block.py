"""Pins of oracle/block.py: against torch float64 operations and autograd, and
against differences of the forward definitions."""
import numpy as np
import pytest
import torch

from oracle import block as ob

ACTS = ("none", "relu", "silu", "gelu")


def test_e4m3_equals_torchs_rounding_over_every_step():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = np.unique(codes[np.isfinite(codes)])
    mids = (codes[1:] + codes[:-1]) / 2
    v = np.concatenate([codes, mids, np.nextafter(mids, 1e9), np.nextafter(mids, -1e9),
                        np.random.default_rng(1).uniform(-448, 448, 4000)]).astype(np.float32)
    got = ob.e4m3(v.astype(np.float64))
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, ref)


def test_norm_and_gradients_equal_autograd():
    rng = np.random.default_rng(2)
    x, res, dy, dr = (rng.standard_normal((5, 33)) for _ in range(4))
    w = 1 + 0.1 * rng.standard_normal(33)
    tx, tr, tw = (torch.tensor(a, requires_grad=True) for a in (x, res, w))
    u = tx + tr
    y = u * torch.rsqrt(u.pow(2).mean(-1, keepdim=True) + 1e-5) * tw
    (y * torch.tensor(dy)).sum().add((u * torch.tensor(dr)).sum()).backward()
    oy, ou, rstd = ob.add_rmsnorm(x, w, res)
    np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-12)
    dx, dw = ob.add_rmsnorm_bwd(dy, ou, w, rstd, dr)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(dx, tr.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-10, atol=1e-13)


@pytest.mark.parametrize("name", ACTS)
def test_linear_and_gradients_equal_autograd(name):
    rng = np.random.default_rng(3)
    x, w, b, res, dy = (rng.standard_normal(s) for s in ((4, 6), (5, 6), (5,), (4, 5), (4, 5)))
    f = {"none": lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu}[name]
    tx, tw, tb, tr = (torch.tensor(a, requires_grad=True) for a in (x, w, b, res))
    y = f(torch.nn.functional.linear(tx, tw, tb)) + tr
    (y * torch.tensor(dy)).sum().backward()
    oy, z = ob.linear(x, w, b, res, name)
    np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-12)
    dx, dw, db, _ = ob.linear_bwd(dy, x, w, z, name)
    for got, t in ((dx, tx), (dw, tw), (db, tb)):
        np.testing.assert_allclose(got, t.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_array_equal(dy, tr.grad.numpy())


def test_gradients_equal_differences():
    """Central differences with step h in 64 bits: error h^2 |f'''| / 6 + 2^-52 |f| / h, about 1e-9 at h = 1e-5."""
    rng = np.random.default_rng(4)
    r, w, dy = rng.standard_normal((2, 7)), 1 + 0.1 * rng.standard_normal(7), rng.standard_normal((2, 7))
    _, _, rstd = ob.add_rmsnorm(r, w)
    dx, dw = ob.add_rmsnorm_bwd(dy, r, w, rstd)
    h = 1e-5
    loss = lambda r_, w_: float((ob.add_rmsnorm(r_, w_)[0] * dy).sum())  # noqa: E731
    for i in np.ndindex(r.shape):
        e = np.zeros_like(r)
        e[i] = h
        assert abs((loss(r + e, w) - loss(r - e, w)) / (2 * h) - dx[i]) < 1e-7
    for j in range(7):
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(r, w + e) - loss(r, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_scales_of_the_8_bit_product_are_a_diagonal_on_each_side():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((3, 8)), rng.standard_normal((4, 8))
    sx, sw = rng.uniform(0.5, 2, 3), rng.uniform(0.5, 2, 4)
    _, z = ob.linear(x, w, x_scale=sx, w_scale=sw)
    np.testing.assert_allclose(z, (np.diag(sx) @ x) @ (np.diag(sw) @ w).T, rtol=1e-13)
