"""What gdn_linear_bwd keeps exactly: dz in as many bf16 parts as it needs and
no more, relu's choice between dy and zero, and every part's place in dw."""
import os

import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import block as ob

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(gdn.lib_path), reason="libgdn.so not built")


def _ints(rng, shape, top, dt):
    return torch.from_numpy(rng.integers(-top, top + 1, shape).astype(np.float32)).to(dt).cuda()


def _h(t):
    return t.detach().float().cpu().double().numpy()


@built
def test_dz_of_a_relu_is_one_part():
    """dy or zero, in bf16 as dy is: fp32 gradients need no more workspace than bf16 ones."""
    size = lambda dy, grad, act: gdn.gdn_linear_bwd_workspace(100, 104, 64, dy, grad, act, need_dw=False)  # noqa: E731
    one = 100 * 104 * 2
    assert one <= size(gdn.GDN_BF16, gdn.GDN_F32, "relu") < 2 * one
    assert size(gdn.GDN_BF16, gdn.GDN_F32, "relu") == size(gdn.GDN_BF16, gdn.GDN_BF16, "relu")
    assert size(gdn.GDN_F32, gdn.GDN_F32, "relu") >= 3 * one and size(gdn.GDN_BF16, gdn.GDN_F32, "silu") >= 3 * one


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 3, 8), (70, 130, 136), (600, 515, 264)])
def test_relu_with_bf16_dy_is_exact(M, N, K):
    rng = np.random.default_rng(M)
    x, w, dy, z = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF), _ints(rng, (M, N), 3, BF), _ints(rng, (M, N), 2, BF)
    rx, rw, rb, _ = ob.linear_bwd(_h(dy), _h(x), _h(w), _h(z), "relu")
    dx, dw, db = gdn.gdn_linear_bwd(dy, x, w, z=z, act="relu", bias=True, grad_dtype=F32)
    for got, ref in ((dx, rx), (dw, rw), (db, rb)):
        np.testing.assert_array_equal(_h(got), ref)


@gpu
def test_an_infinite_weight_meets_no_parts_of_zero():
    """An infinity in w makes an infinity of the gradients it enters, not zero times infinity."""
    rng = np.random.default_rng(5)
    M, N, K = 150, 140, 72
    x, w = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF)
    w[100, 7] = float("inf")
    dy, z = torch.ones(M, N, dtype=BF, device="cuda"), torch.ones(M, N, dtype=BF, device="cuda")
    dx, dw, _ = gdn.gdn_linear_bwd(dy, x, w, z=z, act="relu", grad_dtype=F32)
    assert (dx[:, 7] == float("inf")).all()
    rest = [c for c in range(K) if c != 7]
    np.testing.assert_array_equal(_h(dx[:, rest]), np.broadcast_to(_h(w[:, rest]).sum(0), (M, K - 1)))
    np.testing.assert_array_equal(_h(dw), np.broadcast_to(_h(x).sum(0), (N, K)))


@gpu
@pytest.mark.parametrize("dyt,grad", [(BF, BF), (BF, F32), (F32, F32)])
def test_relu_hides_what_it_masks(dyt, grad):
    """Where z <= 0 nothing of dy comes through, an infinity or NaN neither."""
    rng = np.random.default_rng(6)
    M, N, K = 70, 136, 64
    x, w, dy, z = _ints(rng, (M, K), 3, BF), _ints(rng, (N, K), 3, BF), _ints(rng, (M, N), 3, dyt), _ints(rng, (M, N), 2, BF)
    z[5, 9], z[6, 130], z[69, 0] = 0.0, -1.0, -2.0
    want = gdn.gdn_linear_bwd(dy, x, w, z=z, act="relu", bias=True, grad_dtype=grad)
    dy[5, 9], dy[6, 130], dy[69, 0] = float("nan"), float("inf"), -float("inf")
    got = gdn.gdn_linear_bwd(dy, x, w, z=z, act="relu", bias=True, grad_dtype=grad)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
