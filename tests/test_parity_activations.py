"""GPU parity of the activations in gdn_linear's epilogue and of their
derivatives, in relative terms over the whole range: a product of zeros leaves
z = bias, so y is act(bias) with nothing else in the way.

Phi(z) = exp(-z^2/2) R(|z|) for z <= 0, R a polynomial of degree 8 in
a / (a + 2.875).  Evaluated step by step in fp32 it is within 4.3e-7 of itself
relatively; the hardware's reciprocal and exp2 may each be a unit (1.2e-7)
further off, and the product with z rounds once more: below 2^-20 for fp32
outputs.  bf16 outputs leave out the exponent's correction: 2^-24 |z|^2 more,
7.6e-6 in all at -13, below 2^-16, beside the output's own rounding of 2^-8.
The derivative Phi(z) + z phi(z) is within 2^-20 of the sum of its terms'
magnitudes.  z sigmoid(z): the exponent's argument is rounded twice, 2^-23 |z|,
the rest are five roundings of at most 2 units: 2^-22 |z| + 2^-20."""
import numpy as np
import pytest
from scipy.special import ndtr

import gated_delta_rule_34_amd as gdn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _apply(z, act, out, rows):
    x, w = torch.zeros(rows, 8, dtype=BF, device="cuda"), torch.zeros(len(z), 8, dtype=BF, device="cuda")
    y, _ = gdn.gdn_linear(x, w, bias=torch.from_numpy(z).cuda(), act=act, out_dtype=out)
    assert torch.equal(y, y[:1].expand_as(y))
    return y[0].double().cpu().numpy()


def _slope(z, act):
    """act'(z) at bf16 z, as dbias of a single row with dy = 1."""
    x, w = torch.zeros(1, 8, dtype=BF, device="cuda"), torch.zeros(z.numel(), 8, dtype=BF, device="cuda")
    dy = torch.ones(1, z.numel(), device="cuda")
    return gdn.gdn_linear_bwd(dy, x, w, z=z[None], act=act, bias=True, need_dx=False, need_dw=False)[2].double().cpu().numpy()


@pytest.mark.parametrize("rows", [1, 200])    # the kernel for few rows, and tiles
@pytest.mark.parametrize("out,bar", [(F32, 2.0 ** -20), (BF, 2.0 ** -8 + 2.0 ** -16)])
def test_gelu_is_accurate_relatively(out, bar, rows):
    z = np.linspace(-12.5, 10.0, 9001, dtype=np.float32)
    ref = z.astype(np.float64) * ndtr(z.astype(np.float64))
    err = np.abs(_apply(z, "gelu", out, rows) - ref)
    worst = np.argmax(err - bar * np.abs(ref))
    assert (err <= bar * np.abs(ref)).all(), f"gelu({z[worst]}): off by {err[worst] / abs(ref[worst]):.2e} of itself"


def test_gelu_derivative_is_accurate_relatively():
    t = torch.linspace(-12.5, 10.0, 9001).to(BF).cuda()
    z = t.double().cpu().numpy()
    phi = np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    err = np.abs(_slope(t, "gelu") - (ndtr(z) + z * phi))
    bar = 2.0 ** -20 * (ndtr(z) + np.abs(z) * phi)
    worst = np.argmax(err - bar)
    assert (err <= bar).all(), f"gelu'({z[worst]}): off by {err[worst]:.2e}, bar {bar[worst]:.2e}"


@pytest.mark.parametrize("out,half", [(F32, 0.0), (BF, 2.0 ** -8)])
def test_silu_is_accurate_relatively(out, half):
    z = np.linspace(-80.0, 20.0, 9001, dtype=np.float32)
    z64 = z.astype(np.float64)
    ref = z64 / (1 + np.exp(-z64))
    bar = (2.0 ** -22 * np.abs(z64) + 2.0 ** -20 + half) * np.abs(ref)
    assert (np.abs(_apply(z, "silu", out, 1) - ref) <= bar).all()


def test_activations_far_out():
    """Where exp overflows or vanishes: 0 on the left, z on the right; a NaN stays."""
    z = np.array([-3e38, -1e30, -1e5, -200.0, -40.0, 40.0, 1e5, 1e30, 3e38, np.nan], dtype=np.float32)
    for out in (F32, BF):
        for act in ("gelu", "silu"):
            y = _apply_one(z, act, out)
            ref = torch.from_numpy(z).to(out).double().numpy()
            np.testing.assert_array_equal(y[5:], ref[5:])
            assert (np.abs(y[:4]) <= 1e-30).all() and abs(y[4]) <= 1e-15
    t = torch.from_numpy(z).to(BF).cuda()
    for act in ("gelu", "silu"):
        s = _slope(t, act)
        np.testing.assert_array_equal(s[5:9], 1.0)
        assert (np.abs(s[:4]) <= 1e-30).all() and abs(s[4]) <= 1e-15 and np.isnan(s[9])


def _apply_one(z, act, out):
    x, w = torch.zeros(1, 8, dtype=BF, device="cuda"), torch.zeros(len(z), 8, dtype=BF, device="cuda")
    return gdn.gdn_linear(x, w, bias=torch.from_numpy(z).cuda(), act=act, out_dtype=out)[0][0].double().cpu().numpy()
