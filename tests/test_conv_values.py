"""The short convolution on packed batches in every type and width, with its
activation, and on infinities and NaN.  Bars as in test_parity_scan.py."""
import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import scan as sc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 0.0}


def _t(rng, shape, dt, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _h(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("C,W", [(7, 2), (16, 3), (135, 4), (264, 2), (1031, 3)])
@pytest.mark.parametrize("lens", [[1, 1, 1], [0, 3, 0, 0, 1, 40, 0], [100, 2, 17, 0, 300], [16, 16, 4, 12]])
def test_packed(lens, C, W, dt):
    rng = np.random.default_rng(sum(lens) + C)
    T, k = sum(lens), len(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x, w, b = _t(rng, (T + 5, C), dt), _t(rng, (C, W), F32), _t(rng, (C,), F32)
    for state in (None, _t(rng, (k, W - 1, C), F32)):
        out = torch.full_like(x, 7.0)
        y, new = gdn.gdn_causal_conv_varlen(x, w, cu, bias=b, conv_state=state, out=out)
        assert (y[T:] == 7).all()
        at = 0
        for i, n in enumerate(lens):
            s = None if state is None else _h(state[i:i + 1])
            parts = _h(x[at:at + n])[None], _h(w), _h(b), s
            ref, rs = sc.causal_conv(*parts)
            v, _ = sc.causal_conv(*parts, "none")
            mag, _ = sc.causal_conv(*(None if q is None else np.abs(q) for q in parts), "none")
            bar = 1.1 * (W + 1) * 2.0 ** -24 * mag + (2.0 ** -22 * np.abs(v) + 2.0 ** -20) * np.abs(ref)
            bad = np.abs(_h(y[None, at:at + n]) - ref) - bar - HALF[dt] * (np.abs(ref) + bar)
            assert n == 0 or bad.max() <= 0
            np.testing.assert_array_equal(_h(new[i]), rs[0])
            at += n
        if state is not None:
            held = state.clone()
            y2, new2 = gdn.gdn_causal_conv_varlen(x, w, cu, bias=b, conv_state=held, update_conv_state=True)
            assert new2 is held and torch.equal(held, new) and torch.equal(y2[:T], y[:T])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("C", [64, 129])
def test_special_values_stay_in_their_window(C, act, dt):
    """An input that is no number reaches the W outputs from its own token on, in its channel and its sequence, as the
    definition has it (silu of minus infinity is no number), and the state where it is among the last inputs."""
    rng = np.random.default_rng(C)
    W, T = 4, 50
    x, w, b = _t(rng, (2, T, C), dt), _t(rng, (C, W), F32), _t(rng, (C,), F32)
    st = _t(rng, (2, W - 1, C), F32)
    plain, state = gdn.gdn_causal_conv(x, w, bias=b, act=act, conv_state=st)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x2, s2 = x.clone(), st.clone()
        hits = [(0, 17, 3), (0, T - 2, C - 1), (1, 31, C - 9)]
        for at in hits:
            x2[at] = bad
        s2[1, 1, 5] = bad       # the last but one before the first token: tokens 0 and 1
        with np.errstate(all="ignore"):
            ref, rs = sc.causal_conv(_h(x2), _h(w), _h(b), _h(s2), act)
        y, new = gdn.gdn_causal_conv(x2, w, bias=b, act=act, conv_state=s2)
        odd = ~np.isfinite(ref)
        assert odd.sum() == 4 + 2 + 4 + 2 or (act == "silu" and odd.any())
        np.testing.assert_array_equal(_h(y)[odd], ref[odd])
        touched = np.zeros(ref.shape, bool)
        for n, t, c in hits:
            touched[n, t:t + W, c] = True
        touched[1, :2, 5] = True
        np.testing.assert_array_equal(_h(y)[~touched], _h(plain)[~touched])
        np.testing.assert_array_equal(_h(new), rs)
        held = s2.clone()
        y2, _ = gdn.gdn_causal_conv(x2, w, bias=b, act=act, conv_state=held, update_conv_state=True)
        np.testing.assert_array_equal(_h(y2), _h(y))
        np.testing.assert_array_equal(_h(held), rs)
