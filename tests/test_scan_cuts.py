"""Every form of the scan's kernel -- states, scanning waves, dense and packed,
in one part and cut along the tokens -- against the fp64 definition; special
values that pass from part to part; the accuracy of small steps; and states of
one to three channels.

The bars are those of test_parity_scan.py.  CPU tests hold the lists of sizes to
what they are there for: the workspace says whether a call is cut, and into how
many parts at least."""
import os

import numpy as np
import pytest

import gated_delta_rule_34_amd as gdn
from oracle import scan as sc

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu
built = pytest.mark.skipif(not os.path.exists(gdn.lib_path), reason="libgdn.so not built")
HALF = {BF: 2.0 ** -8, F32: 0.0}
STATES = [8, 16, 32, 64]
CARD = 256  # workgroups, up to which 32 and 64 states take eight scanning waves

# (sequences, tokens, channels): one part, few workgroups; one part, more than 256; in parts, few; in parts, more than
# 256 (from 32 states on); in parts that end with the sequence (of 64 tokens, from 32 states on of 32)
DENSE = [(2, 40, 72), (130, 20, 130), (3, 700, 70), (1, 1100, 520), (1, 512, 64), (2, 384, 64)]
# sequences' lengths, and tokens behind the last one, channels
PACKED = [([0, 3, 0, 0, 1, 40, 0], 5, 72), ([100, 2, 17, 0, 300, 64, 256], 3, 70), ([700, 1, 0, 399], 2, 520),
          ([3] * 150, 1, 24), ([5, 0, 6], 0, 16500)]


def _up(n):
    return (n + 255) // 256 * 256


def _parts(nbytes, seqs, ch, N):
    """Parts of all sequences together, from what is kept between them: (N + 1) numbers a part and channel, N a
    sequence and channel, in three pieces of whole 256 bytes."""
    return (nbytes - _up(seqs * ch * N * 4)) // (ch * (N + 1) * 4) if nbytes else 0


def _groups(ch):
    return (ch + 63) // 64


@built
@pytest.mark.parametrize("N", STATES)
def test_the_sizes_reach_every_form(N):
    seen = set()
    for n, T, ch in DENSE:
        parts = _parts(gdn.gdn_selective_scan_workspace(n, T, ch, N), n, ch, N)
        seen.add((parts > 0, (parts or n) * _groups(ch) > CARD))
    every = {(False, False), (False, True), (True, False)} | ({(True, True)} if N >= 32 else set())
    assert seen == every
    step = 64 if N < 32 else 32
    for n, T, ch in DENSE[-2:]:
        assert T % step == 0 and _parts(gdn.gdn_selective_scan_workspace(n, T, ch, N), n, ch, N) == n * T // step
    seen = set()
    for lens, extra, ch in PACKED:
        parts = _parts(gdn.gdn_selective_scan_varlen_workspace(len(lens), sum(lens) + extra, ch, N), len(lens), ch, N)
        seen.add((parts > 0, (parts or 1) * _groups(ch) > CARD))
    assert seen == every


def _t(rng, shape, dt, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _h(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def _inputs(rng, lead, ch, N, dt, z=True, h0=0):
    p = {"x": _t(rng, lead + (ch,), dt), "dt": _t(rng, lead + (ch,), dt), "B": _t(rng, lead + (N,), dt),
         "C": _t(rng, lead + (N,), dt), "A": -torch.exp(_t(rng, (ch, N), F32)), "D": _t(rng, (ch,), F32),
         "dt_bias": _t(rng, (ch,), F32) - 3.0, "z": _t(rng, lead + (ch,), dt, 2.0) if z else None}
    p["h0"] = _t(rng, (h0, ch, N), F32) if h0 else None
    return p


def _check(y, h, p, T, dt, what=""):
    keys = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")
    ry, rh, by, bh = sc.selective_scan(*(_h(p[k]) for k in keys), per_step=T * 2.0 ** -24)
    for got, ref, bar, name in ((_h(y), ry, by + HALF[dt] * (np.abs(ry) + by), "y"), (_h(h), rh, bh, "h")):
        bad = np.abs(got - ref) - bar
        assert np.isfinite(got).all() and bad.max() <= 0, f"{what}{name}: worst excess {bad.max():.3e}"


@gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("n,T,ch", DENSE)
def test_dense(n, T, ch, N, dt):
    rng = np.random.default_rng(n + T + N)
    p = _inputs(rng, (n, T), ch, N, dt, h0=n)
    y, h = gdn.gdn_selective_scan(**p)
    _check(y, h, p, T, dt)
    again = gdn.gdn_selective_scan(**p)
    assert torch.equal(again[0], y) and torch.equal(again[1], h)
    held = dict(p, h0=p["h0"].clone())
    y2, h2 = gdn.gdn_selective_scan(**held, final_state=held["h0"])
    assert h2 is held["h0"] and torch.equal(h2, h) and torch.equal(y2, y)


@gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("lens,extra,ch", PACKED)
def test_packed(lens, extra, ch, N, dt):
    rng = np.random.default_rng(sum(lens) + N)
    T, k = sum(lens), len(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    for h0 in (0, k):
        p = _inputs(rng, (T + extra,), ch, N, dt, z=h0 > 0, h0=h0)
        out = torch.full_like(p["x"], 7.0)
        y, h = gdn.gdn_selective_scan_varlen(**p, cu_seqlens=cu, out=out)
        assert (y[T:] == 7).all()
        at = 0
        for i, n in enumerate(lens):
            if n == 0:
                assert (h[i] == (p["h0"][i] if h0 else 0)).all()
                continue
            q = dict(p, **{s: p[s][None, at:at + n] for s in ("x", "dt", "B", "C") + (("z",) if h0 else ())})
            q["h0"] = p["h0"][i:i + 1] if h0 else None
            _check(y[None, at:at + n], h[i:i + 1], q, n, dt, f"sequence {i} ")
            at += n
        if h0:
            held = dict(p, h0=p["h0"].clone())
            y2, h2 = gdn.gdn_selective_scan_varlen(**held, cu_seqlens=cu, final_state=held["h0"])
            assert torch.equal(h2, h) and torch.equal(y2[:T], y[:T])


@gpu
@pytest.mark.parametrize("N", [16, 64])
def test_extreme_steps_and_decays_in_parts(N):
    """softplus from far below zero to far above; decays that underflow; A of zero: through a sequence of many parts."""
    rng = np.random.default_rng(4)
    T = 600
    assert gdn.gdn_selective_scan_workspace(1, T, 64, N) > 0
    p = _inputs(rng, (1, T), 64, N, F32, h0=1)
    p["dt"] = torch.linspace(-60, 60, T, device="cuda")[None, :, None].expand(1, T, 64).contiguous()
    p["dt_bias"] = torch.zeros(64, device="cuda")
    p["A"][:, 3] = 0.0
    p["A"][:, 4] = -1e30
    y, h = gdn.gdn_selective_scan(**p)
    _check(y, h, p, T, F32)
    p["dt"] = p["dt"].flip(1).contiguous()
    y, h = gdn.gdn_selective_scan(**p)
    _check(y, h, p, T, F32)


@gpu
@pytest.mark.parametrize("N", [16, 64])
@pytest.mark.parametrize("where", ["x", "dt"])
def test_nan_stays_in_its_channel_and_sequence_in_parts(where, N):
    rng = np.random.default_rng(5)
    p = _inputs(rng, (2, 600), 130, N, F32)
    assert gdn.gdn_selective_scan_workspace(2, 600, 130, N) > 0
    want, hw = gdn.gdn_selective_scan(**p)
    p[where][1, 40, 70] = float("nan")
    y, h = gdn.gdn_selective_scan(**p)
    assert torch.isnan(y[1, 40:, 70]).all() and torch.isnan(h[1, 70]).all()
    y[1, 40:, 70], h[1, 70] = want[1, 40:, 70], hw[1, 70]
    assert torch.equal(y, want) and torch.equal(h, hw)
    cu = torch.tensor([0, 600, 1200], dtype=torch.int32, device="cuda")
    flat = {k: v.reshape(1200, -1) if k in ("x", "dt", "B", "C", "z") else v for k, v in p.items()}
    y, h = gdn.gdn_selective_scan_varlen(**flat, cu_seqlens=cu)
    assert torch.isnan(y[640:, 70]).all() and torch.isnan(h[1, 70]).all()
    y[640:, 70], h[1, 70] = 0, 0
    assert torch.isfinite(y).all() and torch.isfinite(h).all()


@gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_small_steps_keep_their_relative_accuracy(dt):
    """One token, x = B = 1 and no state before it: h is d = softplus(dt), within 2^-20 of itself down to where it
    leaves fp32's normal range; and what the limits give."""
    ch = 2048
    v = torch.linspace(-86, 30, ch).to(dt)
    v[-4:] = torch.tensor([float("inf"), -float("inf"), 3e38, -3e38]).to(dt)
    one = lambda *shape, d=dt: torch.ones(shape, dtype=d, device="cuda")  # noqa: E731
    A, h0 = -one(ch, 8, d=F32), torch.zeros(1, ch, 8, device="cuda")
    _, h = gdn.gdn_selective_scan(one(1, 1, ch), v.cuda()[None, None], A, one(1, 1, 8), one(1, 1, 8))
    _, s = gdn.gdn_selective_step(one(1, ch), v.cuda()[None], A, one(1, 8), one(1, 8), h0)
    want = sc.softplus(v.double().numpy())[:-4]
    for got in (h, s):
        got = _h(got)[0]
        assert (got == got[:, :1]).all()
        assert (np.abs(got[:-4, 0] - want) <= 2.0 ** -20 * want).all()
        assert got[-4, 0] == np.inf and got[-3, 0] == 0 and got[-2, 0] == float(v[-2]) and got[-1, 0] == 0


@gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", [8, 64])
@pytest.mark.parametrize("n,T,ch", [(2, 40, 1), (3, 700, 2), (1, 1, 3), (5, 333, 3)])
def test_few_channels(n, T, ch, N, dt):
    """One to three channels, dense and packed, with and without what is optional, and the step that goes on from them."""
    rng = np.random.default_rng(n + T + N)
    p = _inputs(rng, (n, T), ch, N, dt, h0=n)
    y, h = gdn.gdn_selective_scan(**p)
    assert y.shape == (n, T, ch) and h.shape == (n, ch, N) and y.is_contiguous() and h.is_contiguous()
    _check(y, h, p, T, dt)
    held, out = dict(p, h0=p["h0"].clone()), torch.empty_like(y)
    ws = torch.empty(gdn.gdn_selective_scan_workspace(n, T, ch, N) + 256, dtype=torch.uint8, device="cuda")
    y2, h2 = gdn.gdn_selective_scan(**held, final_state=held["h0"], out=out, workspace=ws)
    assert y2 is out and h2 is held["h0"] and torch.equal(y2, y) and torch.equal(h2, h)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") * T
    flat = {k: v.reshape(n * T, -1) if k in ("x", "dt", "B", "C", "z") else v for k, v in p.items()}
    y3, h3 = gdn.gdn_selective_scan_varlen(**flat, cu_seqlens=cu)
    _check(y3.view(n, T, ch), h3, p, T, dt)
    tail = torch.full((n * T + 2, ch), 7.0, dtype=dt, device="cuda")
    more = {k: torch.cat([v, v[:1], v[:1]]) if k in ("x", "dt", "B", "C", "z") else v for k, v in flat.items()}
    y4, _ = gdn.gdn_selective_scan_varlen(**more, cu_seqlens=cu, out=tail)
    assert y4 is tail and (tail[n * T:] == 7).all()
    q = dict(p, D=None, z=None, dt_bias=None, h0=None, dt=p["dt"] - 3)
    y5, h5 = gdn.gdn_selective_scan(**q)
    _check(y5, h5, q, T, dt)
    y6, none = gdn.gdn_selective_scan(**q, output_final_state=False)
    assert none is None and torch.equal(y6, y5)
    last = {k: p[k][:, -1].contiguous() for k in ("x", "dt", "B", "C", "z")}
    ys, hs = gdn.gdn_selective_step(**last, A=p["A"], D=p["D"], dt_bias=p["dt_bias"], state=h.clone())
    go = dict(p, h0=h, **{k: v[:, None].contiguous() for k, v in last.items()})
    _check(ys[:, None], hs, go, 1, dt)
    yg, hg = gdn.gdn_selective_scan(**go)
    _check(yg, hg, go, 1, dt)
    with pytest.raises(RuntimeError):
        gdn.gdn_selective_scan(**p, out=p["x"])
    with pytest.raises(RuntimeError):
        gdn.gdn_selective_scan(**p, out=p["z"])
    if dt == F32 and T >= N:        # out over what becomes the state
        with pytest.raises(RuntimeError):
            gdn.gdn_selective_scan(**p, out=y, final_state=y.view(-1)[:n * ch * N].view(n, ch, N))


@gpu
def test_few_channels_captured():
    rng = np.random.default_rng(3)
    p = _inputs(rng, (1, 300), 3, 16, BF, h0=1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        gdn.gdn_selective_scan(**p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = gdn.gdn_selective_scan(**p)
    for _ in range(3):
        p["x"].copy_(_t(rng, (1, 300, 3), BF))
        graph.replay()
        torch.cuda.synchronize()
        ey, eh = gdn.gdn_selective_scan(**p)
        assert torch.equal(y, ey) and torch.equal(h, eh)
        torch.cuda.synchronize()
