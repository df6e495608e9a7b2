"""The residual layer norm on values and sizes at its limits."""
import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import block as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


def _t(rng, shape, dt, scale=1.0, shift=0.0):
    return torch.from_numpy((shift + scale * rng.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _h(t):
    return t.detach().float().cpu().double().numpy()


@pytest.mark.parametrize("xd,rd", TYPES)
@pytest.mark.parametrize("D", [5, 24, 64, 256, 1000, 1001, 2056, 4104, 16392])
def test_gradients_of_a_row_of_one_large_value(D, xd, rd):
    """mean rstd is beyond fp32 and xhat zero: dx = rstd (a - mean(a)) is finite, dweight gets nothing from the row.
    Bars as in test_parity_layernorm.py: 2^-17 rstd (|a| + mean|a|), plus 2^-8 |dx| in bf16."""
    rng = np.random.default_rng(D)
    dy, w = _t(rng, (3, D), xd), _t(rng, (D,), F32, 0.1, 1.0)
    r = _t(rng, (3, D), rd)
    r[1] = 2.0 ** 120
    _, _, m, s = ob.add_layernorm(_h(r), _h(w))
    mean, rstd = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (m, s))
    assert np.isfinite(_h(mean)).all() and not torch.isfinite(mean[1] * rstd[1])
    dx, dw, db = gdn.gdn_add_layernorm_bwd(dy, r, w, mean, rstd)
    rx, rw, rb = ob.add_layernorm_bwd(_h(dy), _h(r), _h(w), _h(mean), _h(rstd))
    a, xhat = np.abs(_h(dy) * _h(w)), np.abs((_h(r) - _h(mean)[:, None]) * _h(rstd)[:, None])
    mag = _h(rstd)[:, None] * (a + a.mean(1, keepdims=True) + xhat * np.mean(a * xhat, axis=1, keepdims=True))
    assert np.isfinite(_h(dx)).all()
    assert (np.abs(_h(dx) - rx) <= 2.0 ** -17 * mag + (2.0 ** -8 if rd == BF else 0) * np.abs(rx)).all()
    assert (np.abs(_h(dw) - rw) <= 2.0 ** -16 * (np.abs(_h(dy)) * xhat).sum(0)).all()
    assert (np.abs(_h(db) - rb) <= 2.0 ** -16 * np.abs(_h(dy)).sum(0)).all()


@pytest.mark.parametrize("xd", [BF, F32])
@pytest.mark.parametrize("D", [1, 2, 4, 8, 64])
def test_8_bits_of_a_row_of_one_large_value(D, xd):
    """The differences are zero, the mean times rstd is beyond fp32: codes of zero with scale 1."""
    x = torch.full((5, D), 2.0 ** 60, dtype=xd, device="cuda")
    q, _, mean, rstd, scale = gdn.gdn_add_layernorm(x, torch.ones(D, device="cuda"), eps=1e-44, out_dtype=F8,
                                                    return_stats=True)
    assert (mean == 2.0 ** 60).all() and not torch.isfinite(mean * rstd).any()
    assert (q.float() == 0).all() and (scale == 1).all()
