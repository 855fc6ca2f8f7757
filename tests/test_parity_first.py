"""Prefill with a sliding window and pinned first tokens against the float64 oracle.

Bounds: the rotated dims of Q and K are carried in f16 (half a step 2^-11 each, on the products of
64 dims), the weights in bf16 (2^-8), the output in bf16."""

import numpy as np
import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib, workloads as wl
from oracle import serve
from serve_util import BF16, F16, check, score_error

SCALE = 192 ** -0.5


def _inputs(B, n, off, hq, hkv, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"q": (r(B, n, hq, 192) * scale).bfloat16(), "k": r(B, off + n, hkv, 192).bfloat16(),
            "v": r(B, off + n, hkv, 128).bfloat16(), "sink": r(hq)}


def _delta(inp, rot):
    """Score error: that of the fp32 sums, and of rounding the rotated dims to f16, 2 * 2^-11 of the
    magnitudes |q_r| |k_r| (Cauchy) of the rotated part."""
    q, k = wl.to_f64(inp["q"]), wl.to_f64(inp["k"])
    norm = lambda x: np.linalg.norm(x[..., :rot], axis=-1).max() if rot else 0.0  # noqa: E731
    return score_error(q, k, SCALE) + 2.0 * F16 * SCALE * norm(q) * norm(k)


def _check(inp, dev, window, first, off=0, rotated=False, theta=1e4, rot=64, sink=True, what=""):
    d = {k: v.to(dev) for k, v in inp.items()}
    out, lse = _lib.prefill_first(d["q"], d["k"], d["v"], d["sink"] if sink else None, window=window, n_first=first,
                                  pos_offset=off, k_prefix_rotated=rotated, rope_theta=theta, rot_dims=rot)
    torch.cuda.synchronize()
    assert _lib.last_device_error() == 0
    o, l, mass = serve.prefill_first(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]), wl.to_f64(inp["v"]), off, rotated,
                                     wl.to_f64(inp["sink"]) if sink else None, window, first, theta, rot)
    check(out, lse, o, l, mass, BF16, _delta(inp, rot), what)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (16, 2), (4, 1), (4, 2), (2, 2)])
@pytest.mark.parametrize("window,first", [(128, 4), (129, 16), (128, 17), (16, 1), (1, 3), (200, 64), (64, 150)])
def test_heads_windows(cuda_device, hq, hkv, window, first):
    _check(_inputs(1, 403, 0, hq, hkv, hq + window + first), cuda_device, window, first, what=f"{hq}/{hkv} {window} {first}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 145, 300])
def test_lengths(cuda_device, n):
    _check(_inputs(2, n, 0, 16, 2, 50 + n), cuda_device, 128, 4, what=f"n={n}")
    _check(_inputs(1, n, 0, 8, 1, 51 + n), cuda_device, 32, 20, sink=False, what=f"n={n}")


@pytest.mark.gpu
@pytest.mark.parametrize("off,rotated", [(16, True), (160, False), (160, True), (333, True), (333, False), (2000, True)])
@pytest.mark.parametrize("window,first", [(128, 4), (100, 16), (300, 5), (129, 140)])
def test_chunks(cuda_device, off, rotated, window, first):
    for hq, hkv in ((8, 1), (16, 1)):
        _check(_inputs(1, 75, off, hq, hkv, off + window), cuda_device, window, first, off, rotated,
               what=f"{hq}/{hkv} off {off} W {window} F {first}")


@pytest.mark.gpu
@pytest.mark.parametrize("rot,theta", [(0, 1e4), (16, 1e4), (64, 1e7), (128, 1e4), (192, 5e5)])
def test_rotations(cuda_device, rot, theta):
    for window, first in ((128, 4), (150, 40)):
        _check(_inputs(1, 310, 0, 8, 1, rot), cuda_device, window, first, theta=theta, rot=rot, what=f"rot {rot}")


@pytest.mark.gpu
def test_many_blocks(cuda_device):
    """Runs that cross sequences and heads, so that first tokens change hands inside a CTA."""
    _check(_inputs(3, 700, 0, 16, 2, 60), cuda_device, 128, 4, what="3 x 700")
    _check(_inputs(2, 520, 0, 32, 2, 61), cuda_device, 192, 130, what="2 x 520, G=16")


@pytest.mark.gpu
def test_peaked_and_dominant_sink(cuda_device):
    inp = _inputs(1, 300, 0, 8, 1, 62, scale=8.0)
    for window, first in ((128, 4), (160, 9)):
        _check(inp, cuda_device, window, first, what="peaked")
    inp["sink"] += 60
    for window, first in ((128, 4), (160, 9)):
        _check(inp, cuda_device, window, first, what="dominant sink")


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,window,first", [(16, 2, 128, 4), (16, 1, 256, 32), (8, 2, 64, 64)])
def test_long_sampled(cuda_device, hq, hkv, window, first):
    """Every CTA holds several blocks; the oracle runs on the last 40 rows as a chunk."""
    n = 9001
    inp = _inputs(1, n, 0, hq, hkv, 63)
    d = {k: v.to(cuda_device) for k, v in inp.items()}
    out, lse = _lib.prefill_first(d["q"], d["k"], d["v"], d["sink"], window=window, n_first=first)
    torch.cuda.synchronize()
    assert _lib.last_device_error() == 0
    for at in (0, 4321, n - 40):
        end = at + 40
        o, l, mass = serve.prefill_first(wl.to_f64(inp["q"][:, at:end]), wl.to_f64(inp["k"][:, :end]),
                                         wl.to_f64(inp["v"][:, :end]), at, False, wl.to_f64(inp["sink"]), window, first,
                                         1e4, 64)
        check(out[:, at:end], lse[:, :, at:end], o, l, mass, BF16, _delta(inp, 64), f"rows {at}")


@pytest.mark.gpu
def test_chunks_are_the_whole(cuda_device):
    """Chunk by chunk over raw keys gives the rows of one call (the same tiles up to their borders:
    both within their bounds of the same numbers)."""
    inp = {k: v.to(cuda_device) for k, v in _inputs(1, 512, 0, 8, 1, 64).items()}
    want, _ = _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=128, n_first=4)
    for lo, hi in ((0, 100), (100, 256), (256, 512)):
        got, _ = _lib.prefill_first(inp["q"][:, lo:hi].contiguous(), inp["k"][:, :hi].contiguous(),
                                    inp["v"][:, :hi].contiguous(), inp["sink"], window=128, n_first=4, pos_offset=lo,
                                    k_prefix_rotated=False)
        torch.cuda.synchronize()
        tol = 4 * BF16 * want[:, lo:hi].float().abs() + 0.02
        assert ((got.float() - want[:, lo:hi].float()).abs() <= tol).all()


@pytest.mark.gpu
def test_without_first_tokens_is_the_chunk_call(cuda_device):
    inp = {k: v.to(cuda_device) for k, v in _inputs(1, 300, 0, 8, 1, 65).items()}
    for window, first in ((128, 0), (0, 9), (300, 9), (5000, 9)):
        a = _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=window, n_first=first)
        b = _lib.prefill_chunk(inp["q"], inp["k"], inp["v"], inp["sink"], pos_offset=0, window=window)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_repeats_streams_graph(cuda_device):
    inp = {k: v.to(cuda_device) for k, v in _inputs(1, 500, 0, 8, 1, 66).items()}
    for window, first in ((128, 4), (200, 40)):
        call = lambda **kw: _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=window,  # noqa: E731
                                               n_first=first, **kw)
        want = call()
        side = torch.cuda.Stream(cuda_device)
        side.wait_stream(torch.cuda.current_stream())
        other = call(stream=side)
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out=out, lse=lse)
        graph.replay()
        torch.cuda.synchronize()
        for got in (other, (out, lse), call()):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,window,first", [(8, 1, 128, 4), (8, 1, 200, 40), (16, 1, 64, 130), (4, 2, 128, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_where_they_are_seen(cuda_device, hq, hkv, window, first, bad):
    """A V row of NaN or infinity: queries that mask its key are as if it were 0 (a weight of 0 must
    not multiply it), queries that see a NaN are NaN (the column, or the whole row). Also K rows that are not finite behind a
    sequence's end, as the padding of a batch may hold them."""
    n = 400
    inp = _inputs(1, n, 0, hq, hkv, 70)
    clean = {k: v.clone() for k, v in inp.items()}
    at = [2, 150, 333]
    for t in at:
        inp["v"][0, t, 0, t % 128] = bad
        clean["v"][0, t, 0] = 0
    inp["k"][0, 385:] = bad
    inp["v"][0, 385:] = bad
    d = {k: v.to(cuda_device) for k, v in inp.items()}
    out, lse = _lib.prefill_first(d["q"], d["k"], d["v"], d["sink"], window=window, n_first=first)
    torch.cuda.synchronize()
    assert _lib.last_device_error() == 0
    o, l, mass = serve.prefill_first(*(wl.to_f64(clean[x]) for x in "qkv"), 0, False, wl.to_f64(inp["sink"]), window,
                                     first, 1e4, 64)
    seen = np.array([[any(t <= i and (t > i - window or t < first) for t in at) for i in range(n)]])
    seen = np.repeat(seen[..., None], hq, -1)
    seen[:, :, hq // hkv:] = False                       # the other KV heads are clean
    seen[:, 385:] = True
    fine = ~seen
    got = wl.to_f64(out)
    tol = np.abs(o) * BF16 + mass * (BF16 + 2 * _delta(clean, 64))
    assert (np.abs(got - o)[fine] <= tol[fine]).all()
    if bad != bad:                                       # the definition's NaN: that column of the rows that see it
        for t in at:
            sees = [i for i in range(t, 385) if t > i - window or t < first]
            assert np.isnan(got[0, sees, :hq // hkv, t % 128]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,window,first", [(8, 1, 128, 4), (8, 1, 200, 40), (4, 2, 128, 4)])
def test_a_nan_score_shows(cuda_device, hq, hkv, window, first):
    inp = _inputs(1, 300, 0, hq, hkv, 71)
    inp["k"][0, 20, 0, 100] = float("nan")
    d = {k: v.to(cuda_device) for k, v in inp.items()}
    out, lse = _lib.prefill_first(d["q"], d["k"], d["v"], d["sink"], window=window, n_first=first)
    torch.cuda.synchronize()
    sees = torch.tensor([20 <= i < 20 + window or (i >= 20 and 20 < first) for i in range(300)])
    G = hq // hkv
    assert torch.isnan(out[0, sees, :G]).all() and torch.isnan(lse[0, :G, sees]).all()
    assert torch.isfinite(out[0, ~sees]).all() and torch.isfinite(lse[0][:, ~sees]).all()


@pytest.mark.gpu
def test_scores_that_rise_along_the_window(cuda_device):
    """Keys whose scores climb by far more than 2^8 from slot to slot, so that references move."""
    inp = _inputs(1, 420, 0, 8, 1, 72)
    ramp = torch.linspace(0, 30, 420)[None, :, None]
    for sign in (1, -1):
        inp["k"][..., 64] = (ramp * sign).bfloat16()
        inp["q"][..., 64] = 20.0
        for window, first in ((128, 4), (160, 30)):
            _check(inp, cuda_device, window, first, rot=64, what=f"ramp {sign}")


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [0, 32, 64])
@pytest.mark.parametrize("n,off", [(12, 0), (20, 0), (40, 32), (60, 0)])
def test_runs_over_many_short_sequences(cuda_device, n, off, rot):
    """More row blocks than SMs, one to four per (sequence, KV head): a CTA's run starts anew at its
    second block, at its third, and in between."""
    _check(_inputs(40, n, off, 64, 8, n + rot), cuda_device, 9, 4, off=off, rotated=off > 0, rot=rot, what=f"{n} {off} {rot}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [20, 36, 60])
def test_run_starts_repeat_bit_for_bit(cuda_device, n):
    """Several run starts per CTA (two to four row blocks per (sequence, KV head)), each followed by a
    block that writes the table which held the start's turns: the same bits every time."""
    inp = {k: v.to(cuda_device) for k, v in _inputs(60, n, 0, 64, 8, 90 + n).items()}
    want = _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=11, n_first=4)
    for _ in range(60):
        got = _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=11, n_first=4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,rot", [(8, 1, 64), (16, 1, 64), (4, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("n,off", [(100, 0), (75, 16), (300, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_padding_of_a_batch_shorter_than_its_window(cuda_device, hq, hkv, rot, n, off, bad):
    """Rows behind a sequence's end that are not finite, where the window holds every key (n below the
    default window among them): the queries before them mask them and stay what they are."""
    end = n - 20
    window = max(128, off + n)
    inp = _inputs(2, n, off, hq, hkv, 95 + n)
    clean = {k: v.clone() for k, v in inp.items()}
    inp["k"][1, off + end:] = bad
    inp["v"][1, off + end:] = bad
    clean["v"][1, off + end:] = 0
    clean["k"][1, off + end:] = 0
    d = {k: v.to(cuda_device) for k, v in inp.items()}
    out, lse = _lib.prefill_first(d["q"], d["k"], d["v"], d["sink"], window=window, n_first=4, pos_offset=off,
                                  k_prefix_rotated=False, rot_dims=rot)
    torch.cuda.synchronize()
    o, l, mass = serve.prefill_first(*(wl.to_f64(clean[x]) for x in "qkv"), off, False, wl.to_f64(inp["sink"]), window, 4,
                                     1e4, rot)
    check(out[:, :end].contiguous(), lse[:, :, :end], o[:, :end], l[:, :, :end], mass[:, :end], BF16, _delta(clean, rot),
          f"{hq}/{hkv} n {n}")
    check(out[:1], lse[:1], o[:1], l[:1], mass[:1], BF16, _delta(clean, rot), "the sequence without padding")


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,window,first", [(8, 1, 128, 4), (8, 1, 200, 40), (16, 1, 64, 130), (4, 2, 128, 4),
                                                 (4, 2, 400, 4), (2, 2, 300, 140), (8, 1, 400, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_show_where_they_are_seen(cuda_device, hq, hkv, window, first, bad):
    """A query that sees a V row with a NaN or an infinity is not finite in that column, in every kernel."""
    n, at = 400, [2, 150, 333]
    inp = _inputs(1, n, 0, hq, hkv, 73)
    for t in at:
        inp["v"][0, t, 0, t % 128] = bad
    d = {k: v.to(cuda_device) for k, v in inp.items()}
    out, _ = _lib.prefill_first(d["q"], d["k"], d["v"], d["sink"], window=window, n_first=first)
    torch.cuda.synchronize()
    for t in at:
        sees = [i for i in range(t, n) if t > i - window or t < first]
        assert not torch.isfinite(out[0, sees, :hq // hkv, t % 128]).any(), t
        hides = [i for i in range(n) if not any(u <= i and (u > i - window or u < first) for u in at)]
        assert torch.isfinite(out[0, hides]).all()
    assert torch.isfinite(out[0, :, hq // hkv:]).all()
