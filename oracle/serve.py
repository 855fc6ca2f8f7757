"""Float64 CPU oracle of the calls around a paged KV cache. TEST INFRASTRUCTURE, NOT PRODUCT CODE.

Like oracle/ref.py (whose rope, sink_softmax and FP8 definitions it uses): the plain definitions
in float64 NumPy, sharing nothing with the CUDA package. Readings where the sources are silent:

* Paged cache: token t of sequence b is row table[b][t // page], t % page of the pool; an entry
  outside [0, num_pages) names no page: its tokens are no keys, and are not written.
* Window with pinned first tokens: the query at position p sees [max(0, p - W + 1), p] and
  [0, F); W <= 0 is the causal prefix.
* Draft verification: speculative sampling with given uniform numbers; see verify_drafts.
"""

from __future__ import annotations

import numpy as np

from oracle import ref

__all__ = ["first_keys", "paged_rows", "decode_paged", "append_paged", "quantize_row", "prefill_first",
           "verify_drafts"]


def first_keys(p: int, window: int, first: int) -> np.ndarray:
    """Keys of the query at position p: its window, and the first tokens."""
    if window <= 0:
        return np.arange(p + 1)
    lo = max(0, p - window + 1)
    return np.concatenate([np.arange(min(first, lo)), np.arange(lo, p + 1)])


def paged_rows(table_row, tokens, page: int, num_pages: int) -> np.ndarray:
    """Pool rows (page id, offset) of tokens; tokens whose entry names no page are left out."""
    ids = np.asarray(table_row)[tokens // page]
    ok = (ids >= 0) & (ids < num_pages)
    return np.stack([ids[ok], (tokens % page)[ok]], 1)


def decode_paged(q, k_pages, v_pages, table, lengths, window, first, sink, scale=None):
    """q [B,Hq,d]; pools [N,page,Hkv,·] in float64 (FP8 pools dequantized). Returns out, lse, the
    sum of weights times |v| (for error bounds), and the largest weight times |v| per row."""
    B, hq, d = q.shape
    N, page, hkv, _ = k_pages.shape
    group = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((B, hq, v_pages.shape[-1]))
    lse, mass, top = np.zeros((B, hq)), np.zeros_like(out), np.zeros((B, hq))
    for b in range(B):
        L = min(max(int(lengths[b]), 0), table.shape[1] * page)
        keys = first_keys(L - 1, window, first) if L > 0 else np.arange(0)
        rows = paged_rows(table[b], keys, page, N)
        for h in range(hq):
            K = k_pages[rows[:, 0], rows[:, 1], h // group]
            V = v_pages[rows[:, 0], rows[:, 1], h // group]
            w, lse[b, h] = ref.sink_softmax(K @ q[b, h] * scale, None if sink is None else sink[h])
            out[b, h] = w @ V
            mass[b, h] = w @ np.abs(V)
            top[b, h] = (w * np.abs(V).max(-1)).max() if len(w) else 0.0
    return out, lse, mass, top


def quantize_row(x):
    """Scale amax / 448 (1 for zeros) of rows x [..., D], and the values x / scale before rounding."""
    amax = np.abs(x).max(-1)
    scale = np.where(amax > 0, amax / 448.0, 1.0)
    return x / scale[..., None], scale


def append_paged(k_new, positions, n_new, table, page, num_pages, max_tokens, theta, rot):
    """[(b, i, page id, offset)] of the tokens that are written, and the rotated K [B,n,Hkv,d]."""
    B, n = k_new.shape[:2]
    where, rotated = [], np.zeros_like(k_new)
    for b in range(B):
        pos = positions[b] + np.arange(n)
        rotated[b] = ref.rope(k_new[b], pos, theta, rot)
        for i in range(min(n, int(n_new[b]))):
            if 0 <= pos[i] < max_tokens:
                row = paged_rows(table[b], pos[i:i + 1], page, num_pages)
                where += [(b, i, int(r), int(o)) for r, o in row]
    return where, rotated


def prefill_first(q, k, v, pos_offset, prefix_rotated, sink, window, first, theta, rot, scale=None):
    """q [B,n,Hq,d], k / v [B,off+n,Hkv,·]. Returns out [B,n,Hq,dv], lse [B,Hq,n], mass as above."""
    B, n, hq, d = q.shape
    nk, hkv = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    out, lse, mass = np.zeros((B, n, hq, v.shape[-1])), np.zeros((B, hq, n)), np.zeros((B, n, hq, v.shape[-1]))
    for b in range(B):
        K = ref.rope(k[b], np.arange(nk), theta, rot)
        if prefix_rotated:
            K[:pos_offset] = k[b, :pos_offset]
        Q = ref.rope(q[b], pos_offset + np.arange(n), theta, rot)
        for h in range(hq):
            g = h // (hq // hkv)
            for i in range(n):
                keys = first_keys(pos_offset + i, window, first)
                w, lse[b, h, i] = ref.sink_softmax(K[keys, g] @ Q[i, h] * scale, None if sink is None else sink[h])
                out[b, i, h] = w @ v[b, keys, g]
                mass[b, i, h] = w @ np.abs(v[b, keys, g])
    return out, lse, mass


def verify_drafts(p, q, draft, u, n_valid=None):
    """p [B,T+1,V], q [B,T,V] or None (one-hot), draft [B,T], u [B,T+1]: (accepted [B], tokens [B,T+1]).
    Draft t is accepted while u_t q_t(x) < p_t(x); the next token is the first whose running sum of
    max(p - q, 0) (p after a full acceptance, or when nothing is left) exceeds u_T times the total."""
    B, T = draft.shape
    V = p.shape[2]
    acc, tok = np.zeros(B, np.int64), np.full((B, T + 1), -1, np.int64)

    def mass(x):
        return np.where(np.isfinite(x) & (x > 0), x, 0.0)

    with np.errstate(invalid="ignore"):
        for b in range(B):
            n = T if n_valid is None else min(max(int(n_valid[b]), 0), T)
            t = 0
            while t < n:
                x = draft[b, t]
                inside = 0 <= x < V
                px = p[b, t, x] if inside else 0.0
                qx = 1.0 if q is None else (q[b, t, x] if inside else 0.0)
                if not u[b, t] * qx < px:
                    break
                t += 1
            w = p[b, t].copy()
            if t < n:
                if q is not None:
                    w = w - q[b, t]
                elif 0 <= draft[b, t] < V:
                    w[draft[b, t]] -= 1.0
            w = mass(w)
            if not w.sum() > 0:
                w = mass(p[b, t])
            acc[b] = t
            tok[b, :t] = draft[b, :t]
            if w.sum() > 0:
                run = np.cumsum(w)
                above = np.nonzero((run > u[b, T] * run[-1]) & (w > 0))[0]
                tok[b, t] = above[0] if len(above) else np.nonzero(w)[0][-1]
    return acc, tok
