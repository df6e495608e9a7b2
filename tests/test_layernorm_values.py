"""The residual layer norm on values and sizes at its limits: rows whose mean
times 1 / deviation leaves fp32, infinities and NaN in the backward, and rows
that take more than one launch."""
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


@pytest.mark.parametrize("xd,rd", TYPES)
@pytest.mark.parametrize("rows,D", [(9, 5), (9, 256), (700, 1000), (9, 1001), (40, 2055), (9, 4104), (9, 8201)])
def test_special_values_stay_in_their_row_and_column(rows, D, xd, rd):
    """An infinity or NaN of dy, r or dr: dx of that row only, dweight and dbias of that column only (dr: neither)."""
    rng = np.random.default_rng(rows + D)
    dy, r, dr = _t(rng, (rows, D), xd), _t(rng, (rows, D), rd), _t(rng, (rows, D), rd)
    w = _t(rng, (D,), F32, 0.1, 1.0)
    mean, rstd = r.float().mean(1), 1 / r.float().std(1)
    px, pw, pb = gdn.gdn_add_layernorm_bwd(dy, r, w, mean, rstd, dr=dr)
    cols = [0, D // 2, D - 3, D - 1]      # the last ones are columns that two threads hold where D is odd
    for bad in (float("nan"), float("inf")):
        d2, r2, e2 = dy.clone(), r.clone(), dr.clone()
        d2[1, cols[0]], d2[4, cols[3]] = bad, bad
        r2[6, cols[1]], e2[7, cols[2]] = bad, bad
        dx, dw, db = gdn.gdn_add_layernorm_bwd(d2, r2, w, mean, rstd, dr=e2)
        same = [i for i in range(rows) if i not in (1, 4, 6, 7)]
        assert torch.equal(dx[same], px[same])
        assert not torch.isfinite(dx[[1, 4, 6]].float()).any()
        assert not torch.isfinite(dx[7, cols[2]].float())
        others = [c for c in range(D) if c != cols[2]]
        assert torch.equal(dx[7, others], px[7, others])
        for got, plain, hit in ((dw, pw, (cols[0], cols[3], cols[1])), (db, pb, (cols[0], cols[3]))):
            keep = [c for c in range(D) if c not in hit]
            assert not torch.isfinite(got[list(hit)]).any() and torch.equal(got[keep], plain[keep])


def test_rows_beyond_one_launch():
    """Rows of eight columns go four to a workgroup, 2^21 workgroups to a launch: the rows of the second launch, with
    every output, against the same rows alone."""
    rows, D = (1 << 23) + 5, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(rows, D, generator=gen, device="cuda", dtype=BF)
    res = torch.randn(rows, D, generator=gen, device="cuda", dtype=BF)
    w, b = torch.rand(D, generator=gen, device="cuda"), torch.rand(D, generator=gen, device="cuda")
    for out in (BF, F8):
        got = gdn.gdn_add_layernorm(x, w, bias=b, residual=res, return_stats=True, out_dtype=out)
        for at in (slice(0, 9), slice((1 << 23) - 7, (1 << 23) + 5)):
            want = gdn.gdn_add_layernorm(x[at].contiguous(), w, bias=b, residual=res[at].contiguous(), return_stats=True,
                                         out_dtype=out)
            for g, e in zip(got, want):
                assert (g is None) == (e is None)
                if g is not None:
                    assert torch.equal(g[at].float(), e.float())
