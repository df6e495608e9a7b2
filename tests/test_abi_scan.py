"""Host checks of the convolution and scan entry points: bad arguments come
back as a status before the GPU is touched (fake, never-dereferenced addresses;
needs no GPU)."""
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


@pytest.mark.parametrize("packed", [False, True])
def test_conv_rejects_bad_arguments(packed):
    lib = gdn.load()
    names = ("x", "w", "bias") + (("cu",) if packed else ()) + ("state_in", "y", "state_out")
    base = dict(zip(names, _ptrs(len(names))))
    fn = lib.gdn_causal_conv_varlen if packed else lib.gdn_causal_conv

    def f(B=2, T=100, C=64, W=4, dt=BF16, act=2, **at):
        p = dict(base, **at)
        return fn(*[_p(p[n]) for n in names], B, T, C, W, dt, act, None)

    for n in ("x", "w", "y") + (("cu",) if packed else ()):
        assert f(**{n: None}) == 1
    assert f(B=0) == 1 and f(T=0) == 1 and f(C=0) == 1
    assert f(W=1) == 2 and f(W=5) == 2 and f(dt=F8) == 2 and f(act=1) == 2 and f(act=3) == 2
    assert f(T=1 << 30, C=64) == 2 and f(T=(1 << 30) + 1, C=1) == 2
    assert f(x=base["x"] + 8) == 1 and f(y=base["y"] + 2) == 1 and f(w=base["w"] + 2) == 1
    assert f(y=base["x"]) == 1 and f(y=base["state_in"]) == 1 and f(state_out=base["y"]) == 1
    assert f(state_out=base["state_in"] + 4) == 1 and f(state_out=base["x"]) == 1


@pytest.mark.parametrize("packed", [False, True])
def test_scan_rejects_bad_arguments(packed):
    lib = gdn.load()
    names = ("x", "dt", "A", "B", "C") + (("cu",) if packed else ()) + ("D", "z", "dt_bias", "h0", "y", "ht")
    base = dict(zip(names, _ptrs(len(names))))
    ws = FAKE + (20 << 38)
    fn = lib.gdn_selective_scan_varlen if packed else lib.gdn_selective_scan
    query = lib.gdn_selective_scan_varlen_workspace if packed else lib.gdn_selective_scan_workspace
    need = query(2, 1000, 64, 16)
    assert need > 0 and query(2, 1000, 64, 12) == 0 and query(0, 10, 64, 16) == 0
    assert lib.gdn_selective_scan_workspace(300, 1000, 64, 16) == 0      # enough sequences: in one part each

    def f(n=2, T=1000, ch=64, N=16, dtype=BF16, w_=ws, nbytes=need, **at):
        p = dict(base, **at)
        return fn(*[_p(p[k]) for k in names], n, T, ch, N, dtype, _p(w_), nbytes, None)

    for k in ("x", "dt", "A", "B", "C", "y") + (("cu",) if packed else ()):
        assert f(**{k: None}) == 1
    assert f(n=0) == 1 and f(T=0) == 1 and f(ch=0) == 1 and f(N=0) == 1
    assert f(ch=3) == 2 and f(ch=(1 << 24) + 1) == 2
    assert f(N=12) == 2 and f(N=128) == 2 and f(dtype=F8) == 2 and f(T=(1 << 30) + 1) == 2
    for k in ("x", "dt", "A", "B", "C", "z", "h0", "y", "ht"):
        assert f(**{k: base[k] + 8}) == 1
    assert f(D=base["D"] + 2) == 1 and f(dt_bias=base["dt_bias"] + 1) == 1
    assert f(w_=None) == 3 and f(w_=ws + 16) == 3 and f(nbytes=need - 1) == 3
    assert f(y=base["x"]) == 1 and f(y=base["z"]) == 1 and f(ht=base["y"]) == 1 and f(ht=base["h0"] + 64) == 1
    assert f(w_=base["y"]) == 1 and f(ht=base["A"]) == 1


def test_step_rejects_bad_arguments():
    lib = gdn.load()
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h_in", "h_out", "y")
    base = dict(zip(names, _ptrs(len(names))))

    def f(n=2, ch=64, N=16, dtype=BF16, **at):
        p = dict(base, **at)
        return lib.gdn_selective_step(*[_p(p[k]) for k in names], n, ch, N, dtype, None)

    for k in ("x", "dt", "A", "B", "C", "h_in", "h_out", "y"):
        assert f(**{k: None}) == 1
    assert f(n=0) == 1 and f(ch=0) == 1 and f(N=0) == 1 and f(N=24) == 2 and f(dtype=F8) == 2
    assert f(n=1 << 20, ch=1 << 12) == 2
    for k in ("x", "dt", "A", "B", "C", "z", "h_in", "h_out", "y"):
        assert f(**{k: base[k] + 4}) == 1
    assert f(y=base["x"]) == 1 and f(h_out=base["h_in"] + 64) == 1 and f(h_out=base["y"]) == 1
