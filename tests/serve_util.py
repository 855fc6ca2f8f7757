"""Inputs and error bounds of the tests of the calls around a paged KV cache."""

import numpy as np
import torch

from hybrid_sliding_window_sink_b200 import workloads as wl

BF16, F16 = 2.0 ** -8, 2.0 ** -11      # half a step, relative


def paged_inputs(lengths, hq, hkv, page, *, seed, spare=2, max_pages=None, fill=None, page_gap=0):
    """CPU tensors: q, pools, a random block table, lengths, sink. Unused entries of the table are
    -1; ``fill`` is written into every pool row that no sequence holds; pages lie page_gap tokens apart."""
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    need = [-(-max(L, 0) // page) for L in lengths]
    width = max(max(need), 1) if max_pages is None else max_pages
    N = sum(need) + spare
    order = torch.randperm(N, generator=g)[: sum(need)].tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    q = torch.randn(B, hq, 192, generator=g).bfloat16()
    kbuf = torch.randn(N, page + page_gap, hkv, 192, generator=g).bfloat16()
    vbuf = torch.randn(N, page + page_gap, hkv, 128, generator=g).bfloat16()
    if fill is not None:
        held = torch.zeros(N, page + page_gap, dtype=torch.bool)
        for b, L in enumerate(lengths):
            for t in range(max(L, 0)):
                held[int(table[b, t // page]), t % page] = True
        kbuf[~held] = fill
        vbuf[~held] = fill
    return {"q": q, "k": kbuf[:, :page], "v": vbuf[:, :page], "table": table,
            "lengths": torch.tensor(lengths, dtype=torch.int32), "sink": torch.randn(hq, generator=g)}


def to_dev(inp, dev):
    """Copies to the device, strides of the pools kept."""
    out = {}
    for name, t in inp.items():
        d = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=dev)
        out[name] = d.copy_(t)
    return out


def score_error(q, k, scale):
    """Bound on an fp32 tensor-core dot product of exact products, after the softmax scale: 12 MMAs
    accumulate 16 products each, and each of those sums is off by at most 2^-22 of the sum of the
    magnitudes (it may cut rather than round), which is at most |q| |k|. One more for the last sum."""
    k = np.where(np.isfinite(k), k, 0.0)
    return 13 * 2.0 ** -22 * scale * np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max()


def check(out, lse, o_ref, l_ref, mass, weight, delta, what, extra=0.0):
    """Output within its bf16 rounding (half a step), plus the weights' relative error ``weight``
    and twice the score error ``delta`` (numerator and denominator) on the sum of weights times |v|;
    lse within the score error, the 2^-22 of an exp2 and 16 fp32 roundings. A weight below fp32's
    smallest normal number counts as 0 (ex2 flushes): at most 2^15 keys, each off by 2^-126 |v| with
    |v| < 8, so 2^-108 in all, which matters only where a dominant sink leaves nothing else."""
    o, l = wl.to_f64(out), wl.to_f64(lse)
    tol = np.abs(o_ref) * BF16 + mass * (weight + 2 * delta + 2.0 ** -18) + extra + 2.0 ** -110 * 4
    bad = ~(np.abs(o - o_ref) <= tol)
    assert not bad.any(), (what, "out", np.abs(o - o_ref)[bad].max(), int(bad.sum()), np.argwhere(bad)[:4].tolist())
    inf = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(l), inf), (what, "lse -inf")
    err = np.abs(np.where(inf, 0, l) - np.where(inf, 0, l_ref))
    ltol = delta + 2.0 ** -18 + np.where(inf, 0, np.abs(l_ref)) * 2.0 ** -20
    assert (err <= ltol).all(), (what, "lse", err.max())
