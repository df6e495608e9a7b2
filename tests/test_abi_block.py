"""Host checks of the norm, quantiser and linear entry points: bad arguments
come back as a status before the GPU is touched (fake, never-dereferenced
addresses; needs no GPU)."""
import ctypes
import os

import pytest

import gated_delta_rule_34_amd as gdn

pytestmark = pytest.mark.skipif(not os.path.exists(gdn.lib_path), reason="libgdn.so not built")

FAKE = 0x7F0000000000
F32, BF16, F8 = 0, 1, 2


def _p(x):
    return ctypes.c_void_p(x) if x else None


def _ptrs(n):
    return [FAKE + (i << 36) for i in range(n)]


def test_add_rmsnorm_rejects_bad_arguments():
    lib = gdn.load()
    base = _ptrs(7)   # x residual weight y r rstd y_scale

    def f(ptrs=None, rows=10, D=128, dt=BF16, rdt=BF16, odt=BF16, eps=1e-5, **at):
        p = list(base if ptrs is None else ptrs)
        if odt != F8 and "y_scale" not in at:
            p[6] = None
        for k, v in at.items():
            p[("x", "residual", "weight", "y", "r", "rstd", "y_scale").index(k)] = v
        return lib.gdn_add_rmsnorm(*[_p(x) for x in p], rows, D, dt, rdt, odt, eps, None)

    assert f(x=None) == 1 and f(weight=None) == 1 and f(y=None) == 1
    assert f(rows=0) == 1 and f(rows=-3) == 1 and f(D=0) == 1 and f(eps=0.0) == 1 and f(eps=float("nan")) == 1
    assert f(D=32769) == 2
    assert f(dt=F32, rdt=BF16, odt=F32) == 2 and f(dt=F8) == 2 and f(dt=BF16, odt=F32) == 2 and f(rdt=F8) == 2
    assert f(dt=7) == 2 and f(odt=9) == 2
    assert f(odt=F8, y_scale=None) == 1               # 8 bits need a scale
    assert f(y_scale=base[6]) == 1                    # and only they
    assert f(residual=None) == 1                      # r without residual
    assert f(x=base[0] + 8) == 1 and f(residual=base[1] + 2) == 1 and f(r=base[4] + 4) == 1 and f(y=base[3] + 8) == 1
    assert f(weight=base[2] + 2) == 1 and f(rstd=base[5] + 1) == 1
    assert f(odt=F8, y=base[3] + 4) == 1
    assert f(y=base[0]) == 1 and f(y=base[1]) == 1    # y over x, over residual
    assert f(r=base[1] + 16) == 1                     # r partly over residual
    assert f(r=base[0]) == 1 and f(rstd=base[3]) == 1


def test_add_rmsnorm_bwd_rejects_bad_arguments():
    lib = gdn.load()
    base = _ptrs(7)   # dy r weight rstd dr dx dweight
    ws = FAKE + (9 << 36)
    need = lib.gdn_add_rmsnorm_bwd_workspace(10, 128)
    assert need > 0 and need % 256 == 0
    assert lib.gdn_add_rmsnorm_bwd_workspace(0, 128) == 0 and lib.gdn_add_rmsnorm_bwd_workspace(10, 32769) == 0

    def f(rows=10, D=128, dt=BF16, rdt=BF16, w=ws, nbytes=need, **at):
        p = list(base)
        for k, v in at.items():
            p[("dy", "r", "weight", "rstd", "dr", "dx", "dweight").index(k)] = v
        return lib.gdn_add_rmsnorm_bwd(*[_p(x) for x in p], rows, D, dt, rdt, _p(w), nbytes, None)

    for k in ("dy", "r", "weight", "rstd", "dx"):
        assert f(**{k: None}) == 1
    assert f(rows=0) == 1 and f(D=-1) == 1 and f(D=40000) == 2 and f(dt=F8) == 2 and f(dt=F32, rdt=BF16) == 2
    assert f(w=None) == 3 and f(w=ws + 64) == 3 and f(nbytes=need - 1) == 3
    assert f(dx=base[0]) == 1 and f(dx=base[1]) == 1 and f(dx=base[4]) == 1 and f(dweight=base[5]) == 1
    assert f(dweight=base[2]) == 1 and f(w=base[5]) == 1 and f(dx=base[5] + 2) == 1


def test_quantize_rows_rejects_bad_arguments():
    lib = gdn.load()
    x, q, s = _ptrs(3)

    def f(x=x, q=q, s=s, rows=10, D=128, dt=BF16):
        return lib.gdn_quantize_rows(_p(x), _p(q), _p(s), rows, D, dt, None)

    assert f(x=None) == 1 and f(q=None) == 1 and f(s=None) == 1 and f(rows=0) == 1 and f(D=0) == 1
    assert f(D=32769) == 2 and f(dt=F8) == 2
    assert f(x=x + 2) == 1 and f(q=q + 4) == 1 and f(q=x) == 1 and f(s=q) == 1


def test_linear_rejects_bad_arguments():
    lib = gdn.load()
    base = _ptrs(8)   # x w x_scale w_scale bias residual y z
    ws = FAKE + (12 << 36)
    names = ("x", "w", "x_scale", "w_scale", "bias", "residual", "y", "z")
    assert lib.gdn_linear_workspace(100, 100, 8192, BF16) > 0          # few tiles, long sum: partial sums
    assert lib.gdn_linear_workspace(100, 100, 12, BF16) == 0 and lib.gdn_linear_workspace(0, 100, 64, BF16) == 0

    def f(M=100, N=100, K=8192, dt=BF16, odt=BF16, act=0, w_=ws, nbytes=None, **at):
        p = list(base)
        if dt != F8:
            p[2] = p[3] = None
        for k, v in at.items():
            p[names.index(k)] = v
        if nbytes is None:
            nbytes = lib.gdn_linear_workspace(M, N, K, dt)
        return lib.gdn_linear(*[_p(x) for x in p], M, N, K, dt, odt, act, _p(w_), nbytes, None)

    for k in ("x", "w", "y"):
        assert f(**{k: None}) == 1
    assert f(M=0) == 1 and f(N=-1) == 1 and f(K=0) == 1
    assert f(K=12) == 2 and f(K=8200, dt=F8) == 2 and f(K=(1 << 22) + 8) == 2 and f(N=(1 << 22) + 1) == 2
    assert f(M=2 ** 31 - 1, N=1 << 20) == 2
    assert f(dt=F32) == 2 and f(dt=5) == 2 and f(odt=F8) == 2 and f(act=4) == 2 and f(act=-1) == 2
    assert f(dt=F8, x_scale=None) == 1 and f(dt=F8, w_scale=None) == 1 and f(x_scale=base[2]) == 1
    for k in ("x", "w", "residual", "y", "z"):
        assert f(**{k: base[names.index(k)] + 8}) == 1
    assert f(bias=base[4] + 2) == 1
    assert f(w_=None) == 3 and f(w_=ws + 16) == 3 and f(nbytes=64) == 3
    assert f(y=base[0]) == 1 and f(y=base[5] + 16) == 1 and f(z=base[6]) == 1 and f(z=base[5]) == 1 and f(w_=base[6]) == 1


def test_linear_bwd_rejects_bad_arguments():
    lib = gdn.load()
    base = _ptrs(7)   # dy x w z dx dw dbias
    ws = FAKE + (12 << 36)
    names = ("dy", "x", "w", "z", "dx", "dw", "dbias")

    def size(M=100, N=100, K=64, dyt=BF16, gt=BF16, act=2, a=1, b=1, c=1):
        return lib.gdn_linear_bwd_workspace(M, N, K, dyt, gt, act, a, b, c)

    assert size() >= 100 * 104 * 2 and size(gt=F32) >= 3 * 100 * 104 * 2 and size(K=4) == 0 and size(act=9) == 0
    assert size(N=104, act=0, a=1, b=0, c=0) == 0                       # dz is dy, one part: nothing to keep

    def f(M=100, N=100, K=64, dyt=BF16, gt=BF16, act=2, w_=ws, nbytes=None, **at):
        p = list(base)
        if act == 0:
            p[3] = None
        for k, v in at.items():
            p[names.index(k)] = v
        if nbytes is None:
            nbytes = size(M, N, K, dyt, gt, act)
        return lib.gdn_linear_bwd(*[_p(x) for x in p], M, N, K, dyt, gt, act, _p(w_), nbytes, None)

    for k in ("dy", "x", "w"):
        assert f(**{k: None}) == 1
    assert f(dx=None, dw=None, dbias=None) == 1
    assert f(z=None) == 1 and f(act=0, z=base[3]) == 1
    assert f(M=0) == 1 and f(K=12) == 2 and f(dyt=F8) == 2 and f(gt=F8) == 2 and f(act=7) == 2
    for k in ("dy", "x", "w", "z", "dx", "dw"):
        assert f(**{k: base[names.index(k)] + 8}) == 1
    assert f(w_=None) == 3 and f(w_=ws + 16) == 3 and f(nbytes=64) == 3
    assert f(dx=base[0]) == 1 and f(dw=base[4]) == 1 and f(dbias=base[5]) == 1 and f(w_=base[1]) == 1


def test_linear_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_linear(x, w)
    with pytest.raises(ValueError, match="expected shape"):
        gdn.gdn_linear(x, w[:, :8].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gdn_linear(x, torch.zeros(16, 8, dtype=torch.bfloat16).t())
    with pytest.raises(TypeError):
        gdn.gdn_linear(x, w.float())
    with pytest.raises(ValueError, match="act must be"):
        gdn.gdn_linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="belong to"):
        gdn.gdn_linear(x, w, x_scale=torch.ones(4))
    with pytest.raises(ValueError, match="x_scale is required"):
        gdn.gdn_linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn))
    with pytest.raises(TypeError, match="residual"):
        gdn.gdn_linear(x, w, residual=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="multiple of 8"):
        gdn.gdn_linear(x[:, :12].contiguous(), w[:, :12].contiguous())
    with pytest.raises(ValueError, match="needs z"):
        gdn.gdn_linear_bwd(torch.zeros(4, 8), x, w, act="silu")


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_add_rmsnorm(x, w)
    with pytest.raises(TypeError):
        gdn.gdn_add_rmsnorm(x, w.double())
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gdn_add_rmsnorm(torch.zeros(8, 4, dtype=torch.bfloat16).t(), w)
    with pytest.raises(ValueError, match="expected shape"):
        gdn.gdn_add_rmsnorm(x, w, residual=torch.zeros(4, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="residual_out needs residual"):
        gdn.gdn_add_rmsnorm(x, w, residual_out=x)
    with pytest.raises(TypeError):
        gdn.gdn_quantize_rows(x.to(torch.float16))
    with pytest.raises(ValueError, match="at least one axis"):
        gdn.gdn_quantize_rows(torch.zeros(()))


def test_binding_refuses_a_workspace_elsewhere():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    x, w, ws = torch.zeros(4, 8, dtype=bf), torch.ones(8, 8, dtype=bf), torch.empty(1 << 16, device="meta")
    with pytest.raises(ValueError, match="workspace must be"):
        gdn.gdn_linear(x, w, workspace=ws)
    with pytest.raises(ValueError, match="workspace must be"):
        gdn.gdn_linear_bwd(x, x, w, workspace=ws)
    with pytest.raises(ValueError, match="workspace must be"):
        gdn.gdn_add_rmsnorm_bwd(x, x, torch.ones(8), torch.ones(4), workspace=ws)
    with pytest.raises(ValueError, match="workspace must be"):
        gdn.gdn_linear(x, w, workspace=torch.empty(64, 64)[:, :32])
