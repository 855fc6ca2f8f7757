"""Runs one kernel of the library on a named, profiler-sized case.

Each case is small enough for a full profiler capture (a few GB on the device at
most) but larger than the 126 MB L2, so DRAM counters stay meaningful. Usage:

    python -m hybrid_sliding_window_sink_b200.profile_cases <case> [--reps N]

Cases:
  swa_prefill_n8192     SWA layer prefill, n=8192, 64 Q / 8 KV heads, W=128, RoPE 64 (theta 1e4)
  ga_prefill_n8192      GA layer prefill, n=8192 causal, 64 Q / 4 KV heads, RoPE 64 (theta 1e7)
  decode_ring_b256      SWA decode, B=256, ring of 128 slots, 64 Q / 8 KV heads
  decode_linear_b64_l16k GA decode, B=64, linear cache of 16384 tokens (all full), 64 Q / 4 KV heads
  sparse_b8_l65536      token-level sparse decode, B=8, L=65536, recent 128 + 1024 selected
  mtp_linear_b64_l16k   multi-query (1 + 3 draft tokens) GA decode, B=64, linear cache of 16384
                        tokens (all full), 64 Q / 4 KV heads
  fp8_linear_b64_l16k   GA decode over an FP8 (E4M3 + per-row scale) linear cache, B=64, 16384
                        tokens (all full), 64 Q / 4 KV heads
  chunk_ga_c8192_p8192  GA chunked prefill: 8192-token chunk after an 8192-token rotated prefix,
                        64 Q / 4 KV heads (row-block pair kernel)
  chunk_swa_c8192_p8192 SWA chunked prefill: 8192-token chunk after an 8192-token rotated prefix,
                        64 Q / 8 KV heads, W=128 (K/V-ring kernel)
  paged_b64_ragged      paged decode, B=64, 1024-16384 tokens in pages of 64, 64 Q / 4 KV heads
  paged_fp8_b2_long     paged decode over FP8 pages of 128, B=2, 100k-131k tokens, 64 Q / 4 KV heads
  append_fp8_n4096      page writes, B=2, 4096 tokens, 4 KV heads, FP8 pages of 64
  first_swa_n8192       window prefill with 4 pinned first tokens, n=8192, 64 Q / 8 KV heads, W=128
                        (K/V-ring kernel)
  first_wide_n8192      window prefill with 64 pinned first tokens, n=8192, 64 Q / 4 KV heads, W=2048
                        (row-block pair kernel)
  verify_b64_v131072    draft verification, B=64, 3 drafts, 131072 tokens, fp32
  select_b8_l65536      token selection, B=8, L=65536, 64 Q / 4 KV heads, the 1024 best
                        outside the recent 128
Prints the mean time per call over --reps calls (after two warm-up calls).
"""

from __future__ import annotations

import argparse
import ctypes
import sys

import torch

from . import _lib
from . import workloads as wl


def _paged(lengths, hkv, page, fp8, dev):
    """Pools, a random block table, lengths, q and sink of a paged decode case."""
    g = wl._gen(13, dev)
    B, width = len(lengths), -(-max(lengths) // page)
    table = torch.randperm(B * width, generator=g, device=dev).view(B, width).int()
    if fp8:
        k, v, ks, vs = wl.random_fp8_cache(B * width, page, hkv, seed=14, device=dev)
        pools = (k, v, ks, vs)
    else:
        pools = tuple(wl._randn_bf16((B * width, page, hkv, d), g, dev) for d in (wl.DQK, wl.DV))
    q = wl._randn_bf16((B, 64, wl.DQK), g, dev)
    return q, pools, table, torch.tensor(lengths, dtype=torch.int32, device=dev), torch.randn(64, generator=g, device=dev)


def _case(name, dev):
    if name == "paged_b64_ragged":
        L = wl.lengths_uniform(64, 1024, 16384, seed=13).tolist()
        q, pools, table, lengths, sink = _paged(L, 4, 64, False, dev)
        return lambda: _lib.decode_paged(q, *pools, table, lengths, sink)
    if name == "paged_fp8_b2_long":
        q, pools, table, lengths, sink = _paged([131072, 100001], 4, 128, True, dev)
        return lambda: _lib.decode_paged_fp8(q, *pools, table, lengths, sink)
    if name == "append_fp8_n4096":
        _, pools, table, _, _ = _paged([4096, 4096], 4, 64, True, dev)
        g = wl._gen(15, dev)
        kn, vn = (wl._randn_bf16((2, 4096, 4, d), g, dev) for d in (wl.DQK, wl.DV))
        pos = torch.zeros(2, dtype=torch.int32, device=dev)
        return lambda: _lib.cache_append_paged_fp8(kn, vn, *pools, table, pos)
    if name in ("first_swa_n8192", "first_wide_n8192"):
        hkv, W, F, theta = (8, 128, 4, 1e4) if name == "first_swa_n8192" else (4, 2048, 64, 1e7)
        inp = wl.prefill_inputs(1, 8192, 64, hkv, seed=1, device=dev)
        return lambda: _lib.prefill_first(inp["q"], inp["k"], inp["v"], inp["sink"], window=W, n_first=F, rope_theta=theta)
    if name == "verify_b64_v131072":
        g = wl._gen(16, dev)
        p = torch.softmax(torch.randn(64, 4, 131072, generator=g, device=dev) * 3, -1)
        qd = torch.softmax(torch.randn(64, 3, 131072, generator=g, device=dev) * 3, -1)
        draft = torch.randint(0, 131072, (64, 3), generator=g, device=dev).int()
        u = torch.rand(64, 4, generator=g, device=dev)
        return lambda: _lib.verify_drafts(p, draft, u, qd)
    if name == "swa_prefill_n8192":
        inp = wl.prefill_inputs(1, 8192, 64, 8, seed=1, device=dev)
        return lambda: _lib.prefill(inp["q"], inp["k"], inp["v"], inp["sink"], window=128,
                                    rope_theta=1e4, rot_dims=64)
    if name == "ga_prefill_n8192":
        inp = wl.prefill_inputs(1, 8192, 64, 4, seed=1, device=dev, k_scale=0.5)
        return lambda: _lib.prefill(inp["q"], inp["k"], inp["v"], inp["sink"], window=0,
                                    rope_theta=1e7, rot_dims=64)
    if name == "decode_ring_b256":
        L = wl.lengths_uniform(256, 4096, 131072, seed=7)
        d = wl.decode_inputs(256, 64, 8, 128, L, seed=7, device=dev)
        return lambda: _lib.decode(d["q"], d["k_cache"], d["v_cache"], d["lengths"], d["sink"],
                                   kind="ring")
    if name == "decode_linear_b64_l16k":
        d = wl.decode_inputs(64, 64, 4, 16384, [16384] * 64, seed=8, device=dev)
        ws = torch.empty(_lib.workspace_size(64, 64, 4, op=_lib.MIMO_OP_DECODE,
                                             kind=_lib.MIMO_CACHE_LINEAR, capacity=16384),
                         dtype=torch.uint8, device=dev)
        return lambda: _lib.decode(d["q"], d["k_cache"], d["v_cache"], d["lengths"], d["sink"],
                                   kind="linear", workspace=ws)
    if name == "sparse_b8_l65536":
        L = 65536
        d = wl.decode_inputs(8, 64, 4, L, [L] * 8, seed=9, device=dev)
        sel = wl.sorted_unique_indices(8, 4, 1024, [L - 128] * 8, seed=9).to(dev)
        return lambda: _lib.sparse(d["q"], d["k_cache"], d["v_cache"], d["lengths"], sel, d["sink"],
                                   recent=128)
    if name == "mtp_linear_b64_l16k":
        d = wl.decode_mq_inputs(64, 4, 64, 4, 16384, [16384] * 64, seed=10, device=dev)
        shape = _lib.make_shape(64, 1, 64, 4)
        nws = int(_lib.lib().mimo_attn_decode_mq_workspace_size(ctypes.byref(shape),
                                                               _lib.MIMO_CACHE_LINEAR, 16384, 4, 0))
        ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
        return lambda: _lib.decode_mq(d["q_mq"], d["k_cache"], d["v_cache"], d["lengths"], d["sink"],
                                      kind="linear", window=0, workspace=ws)
    if name == "fp8_linear_b64_l16k":
        d = wl.decode_fp8_inputs(64, 64, 4, 16384, [16384] * 64, seed=11, device=dev)
        del d["k_cache"], d["v_cache"]
        ws = torch.empty(_lib.workspace_size(64, 64, 4, op=_lib.MIMO_OP_DECODE,
                                             kind=_lib.MIMO_CACHE_LINEAR, capacity=16384),
                         dtype=torch.uint8, device=dev)
        return lambda: _lib.decode_fp8(d["q"], d["k8"], d["v8"], d["k_scale"], d["v_scale"],
                                       d["lengths"], d["sink"], kind="linear", workspace=ws)
    if name == "chunk_ga_c8192_p8192":
        inp = wl.prefill_inputs(1, 16384, 64, 4, seed=12, device=dev, k_scale=0.5)
        q = inp["q"][:, 8192:].contiguous()
        return lambda: _lib.prefill_chunk(q, inp["k"], inp["v"], inp["sink"], pos_offset=8192,
                                          k_prefix_rotated=True, window=0, rope_theta=1e7, rot_dims=64)
    if name == "chunk_swa_c8192_p8192":
        inp = wl.prefill_inputs(1, 16384, 64, 8, seed=13, device=dev)
        q = inp["q"][:, 8192:].contiguous()
        return lambda: _lib.prefill_chunk(q, inp["k"], inp["v"], inp["sink"], pos_offset=8192,
                                          k_prefix_rotated=True, window=128, rope_theta=1e4, rot_dims=64)
    if name == "select_b8_l65536":
        L = 65536
        d = wl.decode_inputs(8, 64, 4, L, [L] * 8, seed=14, device=dev)
        del d["v_cache"]
        out = torch.empty(8, 4, 1024, dtype=torch.int32, device=dev)
        shape = _lib.make_shape(8, 1, 64, 4)
        ws = torch.empty(int(_lib.lib().mimo_attn_select_workspace_size(ctypes.byref(shape), L)),
                         dtype=torch.uint8, device=dev)
        return lambda: _lib.select_tokens(d["q"], d["k_cache"], d["lengths"], recent=128, n_sel=1024,
                                          out=out, workspace=ws)
    raise SystemExit(f"unknown case {name}")


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("case")
    ap.add_argument("--reps", type=int, default=3)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    fn = _case(a.case, dev)
    fn()
    fn()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(a.reps):
        fn()
    e1.record()
    torch.cuda.synchronize()
    err = _lib.last_device_error()
    print(f"{a.case}: {e0.elapsed_time(e1) / a.reps:.4f} ms per call, device error {err}")
    return 0 if err == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
