"""Paged decode and paged cache writes against the float64 oracle.

Bounds (serve_util.check): P has 16 significant bits on bf16 pages (two bf16 terms: 2^-16 with the
remainder's own rounding) and 11 on FP8 pages (f16 half step 2^-11)."""

import numpy as np
import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib, workloads as wl
from oracle import ref, serve
from serve_util import F16, BF16, check, paged_inputs, score_error, to_dev

SCALE = 192 ** -0.5


def _oracle(inp, window, first, sink=True, k=None, v=None, scale=None):
    return serve.decode_paged(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]) if k is None else k,
                              wl.to_f64(inp["v"]) if v is None else v, inp["table"].numpy(),
                              inp["lengths"].tolist(), window, first, wl.to_f64(inp["sink"]) if sink else None, scale)


def _run(inp, dev, window=0, first=0, sink=True, **kw):
    d = to_dev(inp, dev)
    out, lse = _lib.decode_paged(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["sink"] if sink else None,
                                 window=window, n_first=first, **kw)
    torch.cuda.synchronize()
    assert _lib.last_device_error() == 0
    return out, lse


def _check(inp, dev, window=0, first=0, sink=True, what="", **kw):
    out, lse = _run(inp, dev, window, first, sink, **kw)
    o, l, mass, _ = _oracle(inp, window, first, sink)
    check(out, lse, o, l, mass, 2.0 ** -16, score_error(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]), SCALE), what)


LENGTHS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 129, 500, 777]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(64, 8), (64, 4), (8, 8), (16, 8), (8, 2)])
@pytest.mark.parametrize("page", [1, 16, 24, 100])
def test_heads_and_pages(cuda_device, hq, hkv, page):
    _check(paged_inputs(LENGTHS, hq, hkv, page, seed=hq + hkv + page), cuda_device, what=f"{hq}/{hkv} page {page}")


@pytest.mark.gpu
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (16, 4), (128, 0), (128, 4), (128, 200), (129, 33), (5000, 7)])
def test_window_and_first(cuda_device, window, first):
    inp = paged_inputs(LENGTHS + [1500], 16, 2, 16, seed=window + first)
    _check(inp, cuda_device, window, first, what=f"W={window} F={first}")
    _check(inp, cuda_device, window, first, sink=False, what=f"W={window} F={first}, no sink")


@pytest.mark.gpu
def test_window_never_reads_given_up_pages(cuda_device):
    """Entries between the first tokens and the window are -1, their rows are NaN."""
    inp = paged_inputs([1000, 700], 64, 8, 16, seed=5)
    want = _oracle(inp, 64, 4)
    for b, L in enumerate((1000, 700)):
        for pg in range(1, (L - 64) // 16):
            inp["k"][inp["table"][b, pg].item()] = float("nan")
            inp["v"][inp["table"][b, pg].item()] = float("nan")
            inp["table"][b, pg] = -1
    out, lse = _run(inp, cuda_device, 64, 4)
    check(out, lse, *want[:3], 2.0 ** -16, score_error(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]), SCALE), "given up")


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3.0e38])
def test_rows_outside_the_sequences(cuda_device, fill):
    """Rows behind a sequence's end, spare pages and the gaps between pages never reach a result."""
    inp = paged_inputs([1, 17, 40, 333], 64, 4, 24, seed=6, fill=fill, page_gap=8, max_pages=20)
    _check(inp, cuda_device, what=f"fill {fill}")


@pytest.mark.gpu
def test_entries_that_name_no_page(cuda_device):
    inp = paged_inputs([200, 90, 64, 300], 8, 1, 16, seed=7)
    inp["table"][0, 3] = -1
    inp["table"][0, 4] = inp["k"].shape[0]            # behind the pool
    inp["table"][1, :] = -1                           # every key is gone: an empty key set
    inp["table"][2, 0] = 2 ** 31 - 1
    inp["table"][3, 18] = -2 ** 31
    _check(inp, cuda_device, what="bad entries")
    _check(inp, cuda_device, sink=False, what="bad entries, no sink")


@pytest.mark.gpu
def test_lengths_are_clamped(cuda_device):
    inp = paged_inputs([48, 48, 0], 8, 1, 16, seed=8, max_pages=3)
    want = _oracle(inp, 0, 0)
    inp["lengths"] = torch.tensor([48, 2 ** 31 - 1, -5], dtype=torch.int32)
    out, lse = _run(inp, cuda_device)
    check(out, lse, *want[:3], 2.0 ** -16, score_error(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]), SCALE), "clamped")


@pytest.mark.gpu
def test_many_units(cuda_device):
    """More (sequence, KV head) units than CTAs: most are whole inside a run, some are cut."""
    g = torch.Generator().manual_seed(9)
    lengths = torch.randint(0, 90, (150,), generator=g).tolist()
    _check(paged_inputs(lengths, 16, 4, 16, seed=9), cuda_device, what="600 units")


@pytest.mark.gpu
def test_long_split(cuda_device):
    _check(paged_inputs([20011], 8, 1, 64, seed=10), cuda_device, what="one unit over all CTAs")
    _check(paged_inputs([9000, 3], 16, 1, 128, seed=11), cuda_device, what="long and short")


@pytest.mark.gpu
def test_shared_pages_and_large_scores(cuda_device):
    inp = paged_inputs([100, 100, 70], 8, 1, 16, seed=12)
    inp["table"][1] = inp["table"][0]                 # a shared prefix
    inp["q"] *= 30                                    # peaked weights
    _check(inp, cuda_device, what="shared, peaked")
    inp["sink"] += 500                                # the sink takes nearly everything
    _check(inp, cuda_device, what="dominant sink")


@pytest.mark.gpu
def test_nan_in_a_valid_key_shows(cuda_device):
    inp = paged_inputs([40, 40], 8, 1, 16, seed=13)
    inp["k"][inp["table"][0, 1].item(), 3] = float("nan")
    out, lse = _run(inp, cuda_device)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[1]).all()


@pytest.mark.gpu
def test_agrees_with_the_linear_cache(cuda_device):
    lengths = [3000, 1, 1234]
    lin = wl.decode_inputs(3, 64, 4, 3000, lengths, seed=14)
    page = 64
    pages = [torch.arange(b * 47, b * 47 + 47, dtype=torch.int32) for b in range(3)]
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 47 * 64 - 3000)).reshape(3 * 47, page, 4, -1)  # noqa: E731
    d = {k: v.to(cuda_device) for k, v in lin.items()}
    a = _lib.decode(d["q"], d["k_cache"], d["v_cache"], d["lengths"], d["sink"], kind="linear")
    b = _lib.decode_paged(d["q"], pad(d["k_cache"]), pad(d["v_cache"]), torch.stack(pages).to(cuda_device),
                          d["lengths"], d["sink"])
    torch.cuda.synchronize()
    # one bf16 rounding on each side, and P's bf16 rounding (2^-8 of the weights' mass) on the linear side
    assert (a[0].float() - b[0].float()).abs().max() <= 2 * BF16 * 4 + BF16 * 4
    assert (a[1] - b[1]).abs().max() <= 1e-4


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda_device):
    """The last pages of a pool of more than 2^31 elements per tensor."""
    page, hkv = 128, 8
    N = (2 ** 31 // (page * hkv * 128)) + 40
    k = torch.empty(N, page, hkv, 192, dtype=torch.bfloat16, device=cuda_device)
    v = torch.empty(N, page, hkv, 128, dtype=torch.bfloat16, device=cuda_device)
    inp = paged_inputs([300], 64, hkv, page, seed=15)
    ids = [N - 1, 0, N - 30]
    table = torch.tensor([ids], dtype=torch.int32, device=cuda_device)
    kn = torch.randn(1, 300, hkv, 192).bfloat16()
    vn = torch.randn(1, 300, hkv, 128).bfloat16()
    _lib.cache_append_paged(kn.to(cuda_device), vn.to(cuda_device), k, v, table,
                            torch.zeros(1, dtype=torch.int32, device=cuda_device), rot_dims=0)
    out, lse = _lib.decode_paged(inp["q"].to(cuda_device), k, v, table, inp["lengths"].to(cuda_device))
    torch.cuda.synchronize()
    pool = torch.zeros(3, page, hkv, 192).bfloat16(), torch.zeros(3, page, hkv, 128).bfloat16()
    for p, n in zip(pool, (kn, vn)):
        p.view(-1, *p.shape[2:])[:300] = n[0]
    o, l, mass, _ = serve.decode_paged(wl.to_f64(inp["q"]), wl.to_f64(pool[0]), wl.to_f64(pool[1]),
                                       np.array([[0, 1, 2]]), [300], 0, 0, None)
    check(out, lse, o, l, mass, 2.0 ** -16, score_error(wl.to_f64(inp["q"]), wl.to_f64(kn), SCALE), "far pages")


@pytest.mark.gpu
def test_agrees_with_the_linear_cache_within_the_roundings(cuda_device):
    """Both outputs per element: a bf16 rounding each, and P's rounding on the sum of weights times |v|
    (half a step of bf16 on the linear cache, 2^-16 here), with the score errors of both."""
    lengths = [3000, 1, 1234]
    lin = wl.decode_inputs(3, 64, 4, 3000, lengths, seed=14)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 47 * 64 - 3000)).reshape(3 * 47, 64, 4, -1)  # noqa: E731
    table = torch.arange(3 * 47, dtype=torch.int32).view(3, 47)
    d = {k: v.to(cuda_device) for k, v in lin.items()}
    a = _lib.decode(d["q"], d["k_cache"], d["v_cache"], d["lengths"], d["sink"], kind="linear")
    b = _lib.decode_paged(d["q"], pad(d["k_cache"]), pad(d["v_cache"]), table.to(cuda_device), d["lengths"], d["sink"])
    torch.cuda.synchronize()
    o, _, mass, _ = serve.decode_paged(wl.to_f64(lin["q"]), wl.to_f64(pad(lin["k_cache"])), wl.to_f64(pad(lin["v_cache"])),
                                       table.numpy(), lengths, 0, 0, wl.to_f64(lin["sink"]))
    delta = score_error(wl.to_f64(lin["q"]), wl.to_f64(lin["k_cache"]), SCALE)
    # off from the definition before its rounding (2^-18: sums and exponentials, as serve_util.check), each side
    off = mass * (BF16 + 2 * delta + 2.0 ** -18) + mass * (2.0 ** -16 + 2 * delta + 2.0 ** -18)
    tol = 2 * np.abs(o) * BF16 + off * (1 + BF16)
    assert (np.abs(wl.to_f64(a[0]) - wl.to_f64(b[0])) <= tol).all()


# ------------------------------------------------------------------ FP8 pages
def _fp8(inp, spread=0.0, seed=0):
    k8, ks = wl.fp8_cache(inp["k"])
    v8, vs = wl.fp8_cache(inp["v"])
    if spread:
        g = torch.Generator().manual_seed(seed)
        vs = vs * torch.exp(spread * torch.randn(vs.shape, generator=g))
    return dict(inp, k=k8, v=v8, ks=ks, vs=vs)


def _check_fp8(inp, dev, window=0, first=0, sink=True, what=""):
    k = ref.dequant_fp8(inp["k"].numpy(), inp["ks"].numpy())
    v = ref.dequant_fp8(inp["v"].numpy(), inp["vs"].numpy())
    d = to_dev(inp, dev)
    out, lse = _lib.decode_paged_fp8(d["q"], d["k"], d["v"], d["ks"], d["vs"], d["table"], d["lengths"],
                                     d["sink"] if sink else None, window=window, n_first=first)
    torch.cuda.synchronize()
    assert _lib.last_device_error() == 0
    o, l, mass, top = _oracle(inp, window, first, sink, k, v)
    # f16 weights: half a step, and per key half of f16's smallest step (2^-25) of the row's largest
    # weight times |v| of its scale (448 / |v|max of a row is at most about 448)
    n = max(1, int(inp["lengths"].max()))
    extra = (n * 2.0 ** -25 * top * 2)[..., None]
    check(out, lse, o, l, mass, F16 + 2.0 ** -18, 2 * score_error(wl.to_f64(inp["q"]), k, SCALE), what, extra)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,page", [(64, 8, 16), (64, 4, 128), (8, 8, 24), (8, 2, 1), (16, 8, 100)])
def test_fp8(cuda_device, hq, hkv, page):
    _check_fp8(_fp8(paged_inputs(LENGTHS, hq, hkv, page, seed=20 + hq)), cuda_device, what=f"fp8 {hq}/{hkv} {page}")


@pytest.mark.gpu
@pytest.mark.parametrize("window,first", [(16, 4), (128, 0), (129, 70)])
def test_fp8_window(cuda_device, window, first):
    inp = _fp8(paged_inputs([1500, 3, 200], 64, 8, 32, seed=21))
    _check_fp8(inp, cuda_device, window, first, what="fp8 window")


@pytest.mark.gpu
def test_fp8_scales_over_many_orders(cuda_device):
    inp = _fp8(paged_inputs([700, 65, 1], 16, 2, 16, seed=22), spread=5.0, seed=3)
    _check_fp8(inp, cuda_device, what="spread scales")
    inp["vs"][::2] = 0.0                              # half of the pages' values vanish
    _check_fp8(inp, cuda_device, what="zero scales")
    inp["vs"][:] = 0.0
    _check_fp8(inp, cuda_device, what="all zero")


@pytest.mark.gpu
def test_fp8_strided_and_split(cuda_device):
    inp = paged_inputs([6000, 77], 16, 1, 24, seed=23, fill=0.0, page_gap=8)
    f = _fp8(inp)
    wide = lambda t: torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, 8))[:, :24]  # noqa: E731
    for name in ("k", "v", "ks", "vs"):
        f[name] = wide(f[name])
    for name in ("k", "v", "ks", "vs"):
        assert f[name].stride(0) // (f[name][0, 0].numel()) == 32
    _check_fp8(f, cuda_device, what="fp8 strided")


@pytest.mark.gpu
@pytest.mark.parametrize("small", [2.0 ** -6, 2.0 ** -12, 2.0 ** -16])
def test_fp8_small_queries_and_large_key_scales(cuda_device, small):
    """Q becomes f16: exact while 2^-17 <= |q| <= 65504, off by at most 2^-25 an element below (half of
    f16's smallest step), which large K scales bring back into the scores."""
    inp = _fp8(paged_inputs([333, 40], 16, 2, 16, seed=24))
    inp["q"] = (inp["q"].float() * small).bfloat16()
    inp["ks"] = inp["ks"] / small
    k = ref.dequant_fp8(inp["k"].numpy(), inp["ks"].numpy())
    v = ref.dequant_fp8(inp["v"].numpy(), inp["vs"].numpy())
    d = to_dev(inp, cuda_device)
    out, lse = _lib.decode_paged_fp8(d["q"], d["k"], d["v"], d["ks"], d["vs"], d["table"], d["lengths"], d["sink"])
    torch.cuda.synchronize()
    o, l, mass, top = _oracle(inp, 0, 0, True, k, v)
    # a score is off by 2^-25 for each of the 192 dims times |k| of that dim, besides the sum's own error;
    # two scores off by delta move a weight by a factor of at most e^(2 delta)
    conv = SCALE * 2.0 ** -25 * np.abs(k).sum(-1).max()
    delta = 2 * score_error(wl.to_f64(inp["q"]), k, SCALE) + conv
    check(out, lse, o, l, mass, F16 + 2.0 ** -18 + (np.expm1(2 * delta) - 2 * delta), delta, f"small {small}",
          (333 * 2.0 ** -25 * top * 2)[..., None])


# ------------------------------------------------------------------ cache writes
def _append_case(hkv, page, n, positions, seed, n_new=None, fp8=False):
    g = torch.Generator().manual_seed(seed)
    B = len(positions)
    width = max(1, -(-(max(positions) + n) // page))
    N = B * width + 2
    table = torch.randperm(N, generator=g)[: B * width].view(B, width).int()
    kn = torch.randn(B, n, hkv, 192, generator=g).bfloat16()
    vn = torch.randn(B, n, hkv, 128, generator=g).bfloat16()
    if fp8:
        k = torch.randint(0, 120, (N, page, hkv, 192), generator=g, dtype=torch.uint8)
        v = torch.randint(0, 120, (N, page, hkv, 128), generator=g, dtype=torch.uint8)
    else:
        k = torch.randn(N, page, hkv, 192, generator=g).bfloat16()
        v = torch.randn(N, page, hkv, 128, generator=g).bfloat16()
    ks, vs = torch.rand(N, page, hkv, generator=g), torch.rand(N, page, hkv, generator=g)
    return dict(kn=kn, vn=vn, k=k, v=v, ks=ks, vs=vs, table=table,
                pos=torch.tensor(positions, dtype=torch.int32),
                n_new=None if n_new is None else torch.tensor(n_new, dtype=torch.int32))


def _check_append(c, dev, theta=1e4, rot=64, fp8=False):
    d = {k: None if v is None else v.to(dev) for k, v in c.items()}
    if fp8:
        _lib.cache_append_paged_fp8(d["kn"], d["vn"], d["k"], d["v"], d["ks"], d["vs"], d["table"], d["pos"],
                                    n_new=d["n_new"], rope_theta=theta, rot_dims=rot)
    else:
        _lib.cache_append_paged(d["kn"], d["vn"], d["k"], d["v"], d["table"], d["pos"], n_new=d["n_new"],
                                rope_theta=theta, rot_dims=rot)
    torch.cuda.synchronize()
    B, n = c["kn"].shape[:2]
    N, page = c["k"].shape[:2]
    where, kr = serve.append_paged(wl.to_f64(c["kn"]), c["pos"].numpy().astype(np.int64),
                                   [n] * B if c["n_new"] is None else c["n_new"].tolist(), c["table"].numpy(), page, N,
                                   c["table"].shape[1] * page, theta, rot)
    vr = wl.to_f64(c["vn"])
    touched = torch.zeros(N, page, dtype=torch.bool)
    for _, _, r, o in where:
        touched[r, o] = True
    for name in ("k", "v") + (("ks", "vs") if fp8 else ()):
        assert torch.equal(d[name].cpu()[~touched], c[name][~touched]), f"{name}: other rows changed"
    if not where:
        return
    b, i, r, o = (np.array(x) for x in zip(*where))
    # the angle is reduced in double and its sine and cosine are good to 2 fp32 steps, three products
    # and a sum: 2^-21 of the two dims' magnitudes
    near = 2.0 ** -21 * 2 * np.abs(wl.to_f64(c["kn"])).max()
    if not fp8:
        got = wl.to_f64(d["k"])[r, o]
        want = kr[b, i]
        assert (np.abs(got - want) <= np.abs(want) * BF16 + near).all()
        assert np.array_equal(got[..., rot:], want[..., rot:])
        assert np.array_equal(wl.to_f64(d["v"])[r, o], vr[b, i])
        return
    for got8, gots, want in ((d["k"], d["ks"], kr[b, i]), (d["v"], d["vs"], vr[b, i])):
        x, scale = serve.quantize_row(want)
        gs = wl.to_f64(gots)[r, o]
        assert (np.abs(gs - scale) <= scale * 2.0 ** -22 + near / 448).all()
        got = ref.e4m3_to_float(got8.cpu().numpy())[r, o]
        # half a step of e4m3 (2^-4 relative, 2^-10 among the subnormals), and the value's own error
        tol = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10) + near / scale[..., None] + np.abs(x) * 2.0 ** -20
        assert (np.abs(got - x) <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,page,n,positions", [
    (8, 16, 1, [0, 5, 15, 16, 1000]), (4, 24, 7, [3, 40]), (1, 1, 3, [0, 2]), (1, 100, 150, [77]), (3, 64, 65, [0, 64]),
])
def test_append(cuda_device, hkv, page, n, positions, fp8):
    c = _append_case(hkv, page, n, positions, 30 + n, fp8=fp8)
    _check_append(c, cuda_device, fp8=fp8)


@pytest.mark.gpu
@pytest.mark.parametrize("rot,theta", [(0, 0.0), (16, 1e4), (64, 1e7), (128, 5e5), (192, 1e4)])
def test_append_rotations(cuda_device, rot, theta):
    for fp8 in (False, True):
        c = _append_case(2, 16, 5, [20000, 3], 31, fp8=fp8)
        _check_append(c, cuda_device, theta, rot, fp8)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_append_ragged_and_outside(cuda_device, fp8):
    """n_new per sequence (a padded batch), positions before 0 and behind the table, bad entries."""
    c = _append_case(2, 16, 9, [0, 10, 20, 30, 5, 12], 32, n_new=[9, 0, 4, -3, 100, 9], fp8=fp8)
    c["pos"] = torch.tensor([-4, 10, c["table"].shape[1] * 16 - 2, 30, 2 ** 31 - 3, 12], dtype=torch.int32)
    c["table"][5, 1] = -1
    c["table"][2, -1] = c["k"].shape[0]
    _check_append(c, cuda_device, fp8=fp8)


@pytest.mark.gpu
def test_append_fp8_special_rows(cuda_device):
    c = _append_case(2, 16, 4, [0], 33, fp8=True)
    c["kn"][0, 0] = 0                                  # a row of zeros: scale 1
    c["vn"][0, 0] = 0
    c["kn"][0, 1] *= 1e-30
    c["vn"][0, 2] *= 1e30
    _check_append(c, cuda_device, fp8=True)
    d = {k: None if v is None else v.to(cuda_device) for k, v in c.items()}
    d["vn"][0, 3, 1, 127] = float("nan")
    d["kn"][0, 3, 0, 0] = float("nan")
    _lib.cache_append_paged_fp8(d["kn"], d["vn"], d["k"], d["v"], d["ks"], d["vs"], d["table"], d["pos"])
    r = int(c["table"][0, 0])
    assert torch.isnan(d["ks"][r, 3]).tolist() == [True, False]
    assert torch.isnan(d["vs"][r, 3]).tolist() == [False, True]
    assert d["ks"][r, 0].tolist() == [1.0, 1.0]


# ------------------------------------------------------------------ how it is called
@pytest.mark.gpu
def test_repeats_streams_graphs_and_buffers(cuda_device):
    inp = to_dev(paged_inputs([3000, 1, 700, 64], 64, 4, 32, seed=40), cuda_device)
    args = [inp[x] for x in ("q", "k", "v", "table", "lengths", "sink")]
    want = _lib.decode_paged(*args)
    again = _lib.decode_paged(*args)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _lib.decode_paged(*args)
    third = _lib.decode_paged(*args, stream=side)      # a stream that is not current, its own scratch
    torch.cuda.synchronize()
    for got in (other, third):
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    size = _lib.decode_paged_workspace_size(4, 64, 4, max_pages=inp["table"].shape[1], page_size=32)
    ws = torch.empty(size, dtype=torch.uint8, device=cuda_device)
    out = torch.empty(4, 64, 128, dtype=torch.bfloat16, device=cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.decode_paged(*args, out=out, want_lse=False, workspace=ws)
    for lengths in ([3000, 1, 700, 64], [5, 0, 31, 1], [3000, 3000, 0, 0]):
        inp["table"][1] = inp["table"][0]
        inp["lengths"].copy_(torch.tensor(lengths))
        ws.fill_(255)
        graph.replay()                                  # the split follows the lengths on the device
        eager = _lib.decode_paged(*args)
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0])


@pytest.mark.gpu
def test_append_then_decode_in_a_graph(cuda_device):
    """One captured decode step (append, attend), replayed for several tokens with advancing lengths."""
    inp = paged_inputs([40, 100], 64, 8, 16, seed=41, max_pages=10)
    for b in range(2):
        free = [x for x in range(inp["k"].shape[0]) if x not in inp["table"].flatten().tolist()]
        inp["table"][b, (40, 100)[b] // 16 + 1] = free[0]
    d = to_dev(inp, cuda_device)
    pos = d["lengths"].clone()
    kn = torch.zeros(2, 1, 8, 192, dtype=torch.bfloat16, device=cuda_device)
    vn = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty(2, 64, 128, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty(2, 64, device=cuda_device)

    def step():
        _lib.cache_append_paged(kn, vn, d["k"], d["v"], d["table"], pos)
        d["lengths"].copy_(pos + 1)
        _lib.decode_paged(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["sink"], out=out, lse=lse)
        pos.add_(1)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(2)
    for t in range(5):
        k1, v1 = torch.randn(2, 1, 8, 192, generator=g).bfloat16(), torch.randn(2, 1, 8, 128, generator=g).bfloat16()
        kn.copy_(k1)
        vn.copy_(v1)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            at = (40, 100)[b] + t
            row = int(inp["table"][b, at // 16]), at % 16
            inp["k"][row] = d["k"][row].cpu()          # what the append wrote (held to the oracle above)
            inp["v"][row] = v1[b, 0]
        inp["lengths"] = torch.tensor([41 + t, 101 + t], dtype=torch.int32)
        o, l, mass, _ = _oracle(inp, 0, 0)
        check(out, lse, o, l, mass, 2.0 ** -16, score_error(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]), SCALE), f"step {t}")


@pytest.mark.gpu
def test_the_two_marshallings_agree(cuda_device):
    """The C++ marshalling is in place, and what it passes on (given outputs, another stream, refused
    sizes) goes through Python with the same results."""
    from hybrid_sliding_window_sink_b200 import _lib as lib
    assert lib._usual(), "_call.so has not been built"
    inp = to_dev(paged_inputs([300, 5, 0], 16, 2, 24, seed=42, page_gap=8), cuda_device)
    args = [inp[x] for x in ("q", "k", "v", "table", "lengths", "sink")]
    fast = lib._usual().decode_paged(args[0], args[1], args[2], None, None, *args[3:], 64, 3, 0.0, True)
    out, lse = torch.empty_like(fast[0]), torch.empty_like(fast[1])
    slow = _lib.decode_paged(*args, window=64, n_first=3, out=out, lse=lse)
    torch.cuda.synchronize()
    assert slow[0] is out and torch.equal(fast[0], out) and torch.equal(fast[1], lse)
    none = lib._usual().decode_paged(args[0], args[1], args[2], None, None, *args[3:], 64, 3, 0.0, False)
    assert none[1] is None
    bad = [(0, args[0].float()), (0, args[0].cpu()), (1, args[1].transpose(1, 2)), (2, args[2][:, :10]), (3, args[3].long()),
           (3, args[3][:2]), (4, args[4][:2]), (5, args[5].double()), (4, None), (1, None)]
    for i, x in bad:
        a = list(args)
        a[i] = x
        assert lib._usual().decode_paged(a[0], a[1], a[2], None, None, *a[3:], 64, 3, 0.0, True) is None, i
        with pytest.raises((TypeError, ValueError)):
            _lib.decode_paged(*a, window=64, n_first=3)
    with pytest.raises(_lib.MimoError, match="SHAPE"):
        _lib.decode_paged(*args, n_first=-1)
    with pytest.raises((TypeError, ValueError)):
        _lib.decode_paged(*args, window="no")
    wide = _lib.decode_paged(*args, window=np.int64(64), n_first=np.int32(3), softmax_scale=0)
    torch.cuda.synchronize()
    assert torch.equal(wide[0], out)
    with pytest.raises(TypeError):
        lib._usual().decode_paged(1)


@pytest.mark.gpu
def test_bad_calls_of_the_other_operators(cuda_device):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=cuda_device)  # noqa: E731
    i32 = torch.int32
    k, v, t, p = z(3, 16, 2, 192), z(3, 16, 2, 128), z(1, 3, dtype=i32), z(1, dtype=i32)
    kn, vn = z(1, 2, 2, 192), z(1, 2, 2, 128)
    good = dict(k_new=kn, v_new=vn, k_pages=k, v_pages=v, block_table=t, positions=p)
    for name, x in (("k_new", kn.float()), ("v_new", vn[:, :1]), ("k_pages", k[:, :, :1]), ("v_pages", v.cpu()),
                    ("block_table", t.long()), ("positions", z(2, dtype=i32)), ("v_pages", v[:2])):
        with pytest.raises((TypeError, ValueError)):
            _lib.cache_append_paged(**{**good, name: x})
    with pytest.raises(_lib.MimoError, match="UNSUPPORTED"):
        _lib.cache_append_paged(**good, rot_dims=24)
    with pytest.raises((TypeError, ValueError)):
        _lib.cache_append_paged_fp8(kn, vn, k, v, z(3, 16, 2), z(3, 16, 2), t, p)
    pr, d, u = z(2, 3, 50, dtype=torch.float32), z(2, 2, dtype=i32), z(2, 3, dtype=torch.float32)
    for bad in ((pr.double(), d, u), (pr[0], d, u), (pr, d.long(), u), (pr, d, u[:, :2]), (pr, d, u.half()), (pr, d.cpu(), u)):
        with pytest.raises((TypeError, ValueError)):
            _lib.verify_drafts(*bad)
    with pytest.raises((TypeError, ValueError)):
        _lib.verify_drafts(pr, d, u, z(2, 2, 50))          # bf16 drafts beside fp32 targets
    q, kk, vv = z(1, 5, 8, 192), z(1, 5, 1, 192), z(1, 5, 1, 128)
    for bad in ((q, kk[:, :4], vv), (q, kk, vv.float()), (q.transpose(1, 2), kk, vv), (q, kk, vv, z(8))):
        with pytest.raises((TypeError, ValueError)):
            _lib.prefill_first(*bad, window=2, n_first=1)
    with pytest.raises(_lib.MimoError, match="SHAPE"):
        _lib.prefill_first(q, kk, vv, window=2, n_first=-1)
    with pytest.raises(ValueError, match="stream"):
        class Other:
            device_index = 5
        _lib.prefill_first(q, kk, vv, window=2, n_first=1, stream=Other())
