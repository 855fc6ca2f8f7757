"""Calls at the edges of what the paged calls document: large batches, the largest windows and counts
of first tokens, other scales, given buffers, and the Python marshalling of every call."""

import numpy as np
import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib, workloads as wl
from oracle import serve
from serve_util import BF16, check, paged_inputs, score_error, to_dev

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
BIG = 2 ** 31 - 1


def _paged_check(inp, dev, window=0, first=0, scale=0.0, rows=None, what=""):
    d = to_dev(inp, dev)
    out, lse = _lib.decode_paged(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["sink"], window=window,
                                 n_first=first, softmax_scale=scale)
    torch.cuda.synchronize()
    rows = list(range(len(inp["lengths"]))) if rows is None else rows
    s = scale if scale > 0 else SCALE
    o, l, mass, _ = serve.decode_paged(wl.to_f64(inp["q"])[rows], wl.to_f64(inp["k"]), wl.to_f64(inp["v"]),
                                       inp["table"].numpy()[rows], inp["lengths"].numpy()[rows], window, first,
                                       wl.to_f64(inp["sink"]), s)
    check(out[rows], lse[rows], o, l, mass, 2.0 ** -16, score_error(wl.to_f64(inp["q"]), wl.to_f64(inp["k"]), s), what)


def test_a_large_batch(cuda_device):
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 40, (5003,), generator=g).tolist()
    lengths[4000] = 900                                  # one unit cut over several CTAs among many whole ones
    inp = paged_inputs(lengths, 2, 2, 16, seed=1)
    _paged_check(inp, cuda_device, rows=[0, 1, 2, 700, 2500, 3999, 4000, 4001, 5002], what="5003 sequences")


def test_largest_window_and_first(cuda_device):
    inp = paged_inputs([100, 333, 1], 8, 1, 16, seed=2)
    for window, first in ((BIG, 0), (BIG, BIG), (1, BIG), (50, BIG), (-5, 7)):
        _paged_check(inp, cuda_device, window, first, what=f"W={window} F={first}")


def test_scales_and_large_pages(cuda_device):
    inp = paged_inputs([100, 333, 4097], 16, 1, 5000, seed=3)
    for scale in (0.01, 1.0):
        _paged_check(inp, cuda_device, scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (4, 1)])
def test_prefill_first_scales_and_everything_first(cuda_device, hq, hkv):
    inp = {k: v.to(cuda_device) for k, v in wl.prefill_inputs(1, 290, hq, hkv, seed=4).items()}
    # all earlier tokens pinned: the causal prefix
    a = _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=20, n_first=BIG)
    b = _lib.prefill(inp["q"], inp["k"], inp["v"], inp["sink"], window=0)
    torch.cuda.synchronize()
    assert ((a[0].float() - b[0].float()).abs() <= 4 * BF16 * b[0].float().abs() + 0.02).all()
    assert (a[1] - b[1]).abs().max() <= 1e-3
    x = {k: wl.to_f64(v) for k, v in inp.items()}
    for window, first in ((128, 4), (150, 40)):
        out, lse = _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=window, n_first=first,
                                      softmax_scale=0.02)
        torch.cuda.synchronize()
        o, l, mass = serve.prefill_first(x["q"], x["k"], x["v"], 0, False, x["sink"], window, first, 1e4, 64, 0.02)
        delta = score_error(x["q"], x["k"], 0.02) + 2.0 * 2.0 ** -11 * 0.02 * np.linalg.norm(
            x["q"][..., :64], axis=-1).max() * np.linalg.norm(x["k"][..., :64], axis=-1).max()
        check(out, lse, o, l, mass, BF16, delta, f"scale 0.02, {hq}/{hkv}")


def test_given_buffers(cuda_device):
    d = to_dev(paged_inputs([300, 20], 16, 2, 16, seed=5), cuda_device)
    args = [d[x] for x in ("q", "k", "v", "table", "lengths", "sink")]
    size = _lib.decode_paged_workspace_size(2, 16, 2, max_pages=d["table"].shape[1], page_size=16)
    with pytest.raises(ValueError, match="too small"):
        _lib.decode_paged(*args, workspace=torch.empty(size - 1, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(ValueError, match="workspace"):
        _lib.decode_paged(*args, workspace=torch.empty(size, dtype=torch.uint8))
    with pytest.raises((ValueError, TypeError)):
        _lib.decode_paged(*args, out=torch.empty(2, 16, 128, device=cuda_device))
    with pytest.raises(ValueError):
        _lib.decode_paged(*args, lse=torch.empty(2, 8, device=cuda_device))
    with pytest.raises(_lib.MimoError, match="ALIGN"):
        _lib.decode_paged(*args, workspace=torch.empty(size + 8, dtype=torch.uint8, device=cuda_device)[4:])


def test_python_marshalling_of_every_call(cuda_device, monkeypatch):
    """The same calls with and without the C++ marshalling, bit for bit."""
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    d = to_dev(paged_inputs([300, 20], 16, 2, 16, seed=6), dev)
    k8, ks = wl.fp8_cache(d["k"])
    v8, vs = wl.fp8_cache(d["v"])
    kn = torch.randn(2, 3, 2, 192, generator=g).bfloat16().to(dev)
    vn = torch.randn(2, 3, 2, 128, generator=g).bfloat16().to(dev)
    pos = torch.tensor([5, 17], dtype=torch.int32, device=dev)
    count = torch.tensor([3, 2], dtype=torch.int32, device=dev)
    p = torch.softmax(torch.randn(3, 4, 999, generator=g), -1).to(dev)
    dq = torch.softmax(torch.randn(3, 3, 999, generator=g), -1).to(dev)
    draft, u = torch.randint(0, 999, (3, 3), generator=g).int().to(dev), torch.rand(3, 4, generator=g).to(dev)
    nv = torch.tensor([3, 1, 0], dtype=torch.int32, device=dev)
    x = {k: v.to(dev) for k, v in wl.prefill_inputs(1, 70, 8, 1, seed=7).items()}

    def everything():
        out = [*_lib.decode_paged(d["q"], d["k"], d["v"], d["table"], d["lengths"], d["sink"], window=40, n_first=2),
               *_lib.decode_paged_fp8(d["q"], k8, v8, ks, vs, d["table"], d["lengths"], window=40, n_first=2),
               *_lib.verify_drafts(p, draft, u, dq, n_valid=nv), *_lib.verify_drafts(p.bfloat16(), draft, u),
               *_lib.prefill_first(x["q"], x["k"], x["v"], x["sink"], window=30, n_first=5)]
        pools = [t.clone() for t in (d["k"], d["v"], k8, v8, ks, vs)]
        _lib.cache_append_paged(kn, vn, pools[0], pools[1], d["table"], pos, n_new=count, rope_theta=1e6, rot_dims=32)
        _lib.cache_append_paged_fp8(kn, vn, *pools[2:], d["table"], pos)
        torch.cuda.synchronize()
        return out + pools

    fast = everything()
    monkeypatch.setattr(_lib, "_usual", lambda: False)
    slow = everything()
    assert len(fast) == len(slow) and all(torch.equal(a, b) for a, b in zip(fast, slow))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 7, 8, 9, 255, 257, 2049, 4099, 20005])
@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_rows_at_any_alignment(cuda_device, V, shift, dtype):
    """Rows of p and q that start anywhere between two 16-byte borders, inside larger buffers whose
    neighbours would win if they were read as part of a row."""
    B, T = 5, 3
    g = torch.Generator().manual_seed(V + 31 * shift)
    n_p, n_q = B * (T + 1) * V, B * T * V
    base_p, base_q = (torch.full((n + 32,), 1e30, dtype=dtype, device=cuda_device) for n in (n_p, n_q))
    p = base_p[shift:shift + n_p].view(B, T + 1, V)
    q = base_q[2 * shift + 1:2 * shift + 1 + n_q].view(B, T, V)
    p.copy_(torch.softmax(torch.randn(B, T + 1, V, generator=g), -1))
    q.copy_(torch.softmax(torch.randn(B, T, V, generator=g), -1))
    draft = torch.randint(0, V, (B, T), generator=g).int()
    u = torch.rand(B, T + 1, generator=g)
    for given in (q, None):
        acc, tok = _lib.verify_drafts(p, draft.to(cuda_device), u.to(cuda_device), given)
        want = serve.verify_drafts(wl.to_f64(p.cpu()), None if given is None else wl.to_f64(q.cpu()),
                                   draft.numpy(), wl.to_f64(u))
        assert acc.tolist() == want[0].tolist() and tok.tolist() == want[1].tolist()


def test_want_lse_goes_by_its_truth_value(cuda_device, monkeypatch):
    """Both marshallings, with everything that is not a bool itself."""
    d = to_dev(paged_inputs([40, 20], 8, 1, 16, seed=8), cuda_device)
    x = {k: v.to(cuda_device) for k, v in wl.prefill_inputs(1, 40, 8, 1, seed=9).items()}
    calls = [lambda w: _lib.decode_paged(d["q"], d["k"], d["v"], d["table"], d["lengths"], want_lse=w),
             lambda w: _lib.prefill_first(x["q"], x["k"], x["v"], window=30, n_first=5, want_lse=w)]
    for usual in (_lib._usual, lambda: False):
        monkeypatch.setattr(_lib, "_usual", usual)
        for call in calls:
            want = call(True)[1]
            for yes in (1, np.bool_(True), "yes", [0]):
                assert torch.equal(call(yes)[1], want), yes
            for no in (False, 0, np.bool_(False), None, ""):
                assert call(no)[1] is None, no


@pytest.mark.parametrize("usual", [True, False])
def test_numbers_beyond_32_bits_are_refused(cuda_device, monkeypatch, usual):
    """The C ABI counts in 32 bits: a window of 2^32 + 5 is not one of 5."""
    if not usual:
        monkeypatch.setattr(_lib, "_usual", lambda: False)
    d = to_dev(paged_inputs([40, 20], 8, 1, 16, seed=8), cuda_device)
    args = [d[x] for x in ("q", "k", "v", "table", "lengths")]
    x = {k: v.to(cuda_device) for k, v in wl.prefill_inputs(1, 40, 8, 1, seed=9).items()}
    qkv = [x[k] for k in "qkv"]
    kn, vn = (torch.zeros(2, 1, 1, w, dtype=torch.bfloat16, device=cuda_device) for w in (192, 128))
    for big in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 70):
        for kw in (dict(window=big), dict(window=5, n_first=big)):
            with pytest.raises(ValueError, match="32 bits"):
                _lib.decode_paged(*args, **kw)
            with pytest.raises(ValueError, match="32 bits"):
                _lib.prefill_first(*qkv, **{"n_first": 1, **kw})
            with pytest.raises(ValueError, match="32 bits"):
                _lib.decode_paged_workspace_size(2, 8, 1, max_pages=3, page_size=16, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            _lib.prefill_first(*qkv, window=5, n_first=1, rot_dims=big)
        with pytest.raises(ValueError):
            _lib.prefill_first(*qkv, window=5, n_first=1, pos_offset=big)
        with pytest.raises(ValueError, match="32 bits"):
            _lib.cache_append_paged(kn, vn, d["k"], d["v"], d["table"], d["lengths"], rot_dims=big)
        with pytest.raises(ValueError, match="32 bits"):
            _lib.decode_paged_workspace_size(2, 8, 1, max_pages=big, page_size=16)
    V = 2 ** 32 + 3                                      # 8 GB a row, never touched
    p = torch.empty(1, 1, V, dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError, match="32 bits"):
        _lib.verify_drafts(p, torch.empty(1, 0, dtype=torch.int32, device=cuda_device), torch.zeros(1, 1, device=cuda_device))
