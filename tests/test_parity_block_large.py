"""Sizes whose element offsets pass 2^31: the last rows and tokens against the
same rows and tokens alone."""
import pytest

import gated_delta_rule_34_amd as gdn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _room(nbytes):
    if torch.cuda.mem_get_info()[0] < 1.1 * nbytes:
        pytest.skip("needs %.0f GB of device memory" % (1.1 * nbytes / 1e9))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF)


def _gen():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    return gen


def test_layernorm_past_2_31():
    rows, D, n = (1 << 21) + 5, 1032, 300
    _room(5 * rows * D * 2)
    gen = _gen()
    x, res = _randn(gen, rows, D), _randn(gen, rows, D)
    w, b = torch.rand(D, generator=gen, device="cuda"), torch.rand(D, generator=gen, device="cuda")
    y, r, m, s, _ = gdn.gdn_add_layernorm(x, w, bias=b, residual=res, return_stats=True)
    for at in (slice(0, n), slice(rows - n, rows)):
        yy, rr, mm, ss, _ = gdn.gdn_add_layernorm(x[at], w, bias=b, residual=res[at], return_stats=True)
        assert torch.equal(y[at], yy) and torch.equal(r[at], rr) and torch.equal(m[at], mm) and torch.equal(s[at], ss)
    del y, res
    dx, _, _ = gdn.gdn_add_layernorm_bwd(x, r, w, m, s)
    for at in (slice(0, n), slice(rows - n, rows)):
        assert torch.equal(dx[at], gdn.gdn_add_layernorm_bwd(x[at], r[at], w, m[at], s[at])[0])


def test_gated_past_2_31():
    """z, dz and y beyond 2^31 elements; the rows' own products are the same in any tile, K in one part."""
    M, N, K, n = (1 << 20) + 300, 1032, 64, 512
    _room(4 * M * 2 * N * 2)
    gen = _gen()
    x, w = _randn(gen, M, K), _randn(gen, 2 * N, K)
    y, z = gdn.gdn_gated_linear(x, w, return_preact=True)
    for at in (slice(0, n), slice(M - n, M)):
        yy, zz = gdn.gdn_gated_linear(x[at].contiguous(), w, return_preact=True)
        assert torch.equal(y[at], yy) and torch.equal(z[at], zz)
    dx = gdn.gdn_gated_linear_bwd(y, x, w, z, need_dw=False)[0]
    for at in (slice(0, n), slice(M - n, M)):
        ref = gdn.gdn_gated_linear_bwd(y[at].contiguous(), x[at].contiguous(), w, z[at].contiguous(), need_dw=False,
                                       grad_dtype=torch.float32)[0]
        # dz and dx rounded to bf16: each at most 2^-8 in the 2-norm
        assert float((dx[at].float() - ref).norm() / ref.norm()) <= 2 * 2.0 ** -8


def test_conv_past_2_31():
    T, C, n = (1 << 20) + 77, 2056, 100
    _room(2 * T * C * 2)
    gen = _gen()
    x, w = _randn(gen, 1, T, C), torch.randn(C, 4, generator=gen, device="cuda")
    y, state = gdn.gdn_causal_conv(x, w)
    last = x[:, T - n - 3:T].contiguous()
    yy, ss = gdn.gdn_causal_conv(last[:, 3:].contiguous(), w, conv_state=last[:, :3].float().contiguous())
    assert torch.equal(y[:, T - n:], yy) and torch.equal(state, ss)
    cu = torch.tensor([0, 5, T - n, T], dtype=torch.int32, device="cuda")
    y, state = gdn.gdn_causal_conv_varlen(x[0], w, cu)
    yy, ss = gdn.gdn_causal_conv(x[:, T - n:].contiguous(), w)
    assert torch.equal(y[T - n:], yy[0]) and torch.equal(state[2:], ss)


def test_scan_past_2_31():
    """Many sequences; the last one alone is cut differently, so states agree to fp32 steps (200 of them, each within
    2^-20 of what it adds or decays) and outputs to a bf16 rounding beside that."""
    B, T, ch, N = 1320, 200, 8200, 16
    _room(4 * B * T * ch * 2)
    gen = _gen()
    x, dt = _randn(gen, B, T, ch), _randn(gen, B, T, ch)
    Bm, Cm = _randn(gen, B, T, N), _randn(gen, B, T, N)
    A = -torch.rand(ch, N, generator=gen, device="cuda") - 0.1
    db = torch.full((ch,), -3.0, device="cuda")
    y, h = gdn.gdn_selective_scan(x, dt, A, Bm, Cm, dt_bias=db)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    flat = [t.view(B * T, -1) for t in (x, dt, Bm, Cm)]
    yv, hv = gdn.gdn_selective_scan_varlen(flat[0], flat[1], A, flat[2], flat[3], cu, dt_bias=db)
    for got, hg in ((y, h), (yv.view(B, T, ch), hv)):
        for i in (0, B - 1):
            yy, hh = gdn.gdn_selective_scan(x[i:i + 1], dt[i:i + 1], A, Bm[i:i + 1], Cm[i:i + 1], dt_bias=db)
            assert float((hg[i:i + 1] - hh).norm() / hh.norm()) <= 200 * 2.0 ** -20
            assert float((got[i:i + 1].float() - yy.float()).norm() / yy.float().norm()) <= 2.0 ** -8
