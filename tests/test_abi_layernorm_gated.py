"""Host checks of the layer norm and gated projection entry points: bad
arguments come back as a status before the GPU is touched (fake,
never-dereferenced addresses; needs no GPU)."""
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
    return [FAKE + (i << 38) for i in range(n)]


def test_layernorm_rejects_bad_arguments():
    lib = gdn.load()
    names = ("x", "residual", "weight", "bias", "y", "r", "mean", "rstd", "y_scale")
    base = dict(zip(names, _ptrs(9)))

    def f(rows=10, D=128, dt=BF16, rdt=BF16, odt=BF16, eps=1e-5, **at):
        p = dict(base, **at)
        if odt != F8 and "y_scale" not in at:
            p["y_scale"] = None
        return lib.gdn_add_layernorm(*[_p(p[n]) for n in names], rows, D, dt, rdt, odt, eps, None)

    assert f(x=None) == 1 and f(weight=None) == 1 and f(y=None) == 1
    assert f(rows=0) == 1 and f(D=0) == 1 and f(eps=0.0) == 1 and f(eps=float("nan")) == 1 and f(D=32769) == 2
    assert f(dt=F32, rdt=BF16, odt=F32) == 2 and f(dt=F8) == 2 and f(odt=F32) == 2 and f(rdt=F8) == 2 and f(odt=9) == 2
    assert f(odt=F8, y_scale=None) == 1 and f(y_scale=base["y_scale"]) == 1 and f(residual=None) == 1
    for n, off in (("x", 8), ("residual", 2), ("y", 8), ("r", 4), ("weight", 2), ("bias", 1), ("mean", 2), ("rstd", 1)):
        assert f(**{n: base[n] + off}) == 1
    assert f(y=base["x"]) == 1 and f(y=base["residual"]) == 1 and f(r=base["residual"] + 16) == 1 and f(r=base["x"]) == 1
    assert f(mean=base["rstd"]) == 1 and f(mean=base["bias"]) == 1 and f(rstd=base["y"]) == 1


def test_layernorm_bwd_rejects_bad_arguments():
    lib = gdn.load()
    names = ("dy", "r", "weight", "mean", "rstd", "dr", "dx", "dweight", "dbias")
    base = dict(zip(names, _ptrs(9)))
    ws = FAKE + (12 << 38)
    need = lib.gdn_add_layernorm_bwd_workspace(10, 128)
    assert need > 0 and need % 256 == 0
    assert lib.gdn_add_layernorm_bwd_workspace(0, 128) == 0 and lib.gdn_add_layernorm_bwd_workspace(10, 32769) == 0

    def f(rows=10, D=128, dt=BF16, rdt=BF16, w=ws, nbytes=need, **at):
        p = dict(base, **at)
        return lib.gdn_add_layernorm_bwd(*[_p(p[n]) for n in names], rows, D, dt, rdt, _p(w), nbytes, None)

    for n in ("dy", "r", "weight", "mean", "rstd", "dx"):
        assert f(**{n: None}) == 1
    assert f(rows=0) == 1 and f(D=-1) == 1 and f(D=40000) == 2 and f(dt=F8) == 2 and f(dt=F32, rdt=BF16) == 2
    assert f(w=None) == 3 and f(w=ws + 64) == 3 and f(nbytes=need - 1) == 3
    assert f(w=None, dweight=None) == 3                 # dbias alone needs it too
    assert f(dx=base["dy"]) == 1 and f(dx=base["r"]) == 1 and f(dx=base["dr"]) == 1 and f(dweight=base["dbias"]) == 1
    assert f(dbias=base["dx"]) == 1 and f(w=base["dx"]) == 1 and f(dweight=base["mean"]) == 1


def test_gated_linear_rejects_bad_arguments():
    lib = gdn.load()
    names = ("x", "w", "x_scale", "w_scale", "bias", "y", "z")
    base = dict(zip(names, _ptrs(7)))
    ws = FAKE + (12 << 38)
    assert lib.gdn_gated_linear_workspace(100, 100, 8192, BF16) > 0
    assert lib.gdn_gated_linear_workspace(100, 100, 8192, BF16) == lib.gdn_linear_workspace(100, 200, 8192, BF16)
    assert lib.gdn_gated_linear_workspace(100, 100, 12, BF16) == 0 and lib.gdn_gated_linear_workspace(0, 100, 64, BF16) == 0

    def f(M=100, N=100, K=8192, dt=BF16, odt=BF16, act=2, w_=ws, nbytes=None, **at):
        p = dict(base)
        if dt != F8:
            p["x_scale"] = p["w_scale"] = None
        p.update(at)
        if nbytes is None:
            nbytes = lib.gdn_gated_linear_workspace(M, N, K, dt)
        return lib.gdn_gated_linear(*[_p(p[n]) for n in names], M, N, K, dt, odt, act, _p(w_), nbytes, None)

    for n in ("x", "w", "y"):
        assert f(**{n: None}) == 1
    assert f(M=0) == 1 and f(N=0) == 1 and f(N=-1) == 1 and f(K=0) == 1
    assert f(K=12) == 2 and f(K=8200, dt=F8) == 2 and f(K=(1 << 22) + 8) == 2 and f(N=(1 << 21) + 1) == 2
    assert f(N=2 ** 31 - 1) == 2 and f(M=2 ** 31 - 1, N=1 << 20) == 2
    assert f(dt=F32) == 2 and f(odt=F8) == 2 and f(act=4) == 2 and f(act=-1) == 2
    assert f(dt=F8, x_scale=None) == 1 and f(dt=F8, w_scale=None) == 1 and f(x_scale=base["x_scale"]) == 1
    for n in ("x", "w", "y", "z"):
        assert f(**{n: base[n] + 8}) == 1
    assert f(bias=base["bias"] + 2) == 1
    assert f(w_=None) == 3 and f(w_=ws + 16) == 3 and f(nbytes=64) == 3
    assert f(y=base["x"]) == 1 and f(z=base["y"]) == 1 and f(w_=base["y"]) == 1
    assert f(z=base["w"] + 2 * 100 * 8192 * 2 - 16) == 1      # the last bytes of the up rows


def test_gated_linear_bwd_rejects_bad_arguments():
    lib = gdn.load()
    names = ("dy", "x", "w", "z", "dx", "dw", "dbias")
    base = dict(zip(names, _ptrs(7)))
    ws = FAKE + (12 << 38)
    need = lib.gdn_gated_linear_bwd_workspace(100, 100, 512, BF16, BF16, 2, 1, 1, 1)
    assert need > 0
    assert lib.gdn_gated_linear_bwd_workspace(100, 100, 512, BF16, F32, 2, 1, 1, 1) > need
    assert lib.gdn_gated_linear_bwd_workspace(100, 100, 12, BF16, BF16, 2, 1, 1, 1) == 0

    def f(M=100, N=100, K=512, dd=BF16, gd=BF16, act=2, w_=ws, nbytes=need, **at):
        p = dict(base, **at)
        return lib.gdn_gated_linear_bwd(*[_p(p[n]) for n in names], M, N, K, dd, gd, act, _p(w_), nbytes, None)

    for n in ("dy", "x", "w", "z"):
        assert f(**{n: None}) == 1
    assert f(dx=None, dw=None, dbias=None) == 1 and f(M=0) == 1 and f(N=0) == 1
    assert f(K=12) == 2 and f(N=(1 << 21) + 1) == 2 and f(dd=F8) == 2 and f(gd=F8) == 2 and f(act=9) == 2
    for n in ("dy", "x", "w", "z", "dx", "dw"):
        assert f(**{n: base[n] + 2}) == 1
    assert f(w_=None) == 3 and f(w_=ws + 8) == 3 and f(nbytes=need - 1) == 3
    assert f(dx=base["dy"]) == 1 and f(dw=base["z"]) == 1 and f(dw=base["dx"]) == 1 and f(w_=base["dw"]) == 1
    assert f(dbias=base["z"] + 100 * 200 * 2 - 4) == 1
