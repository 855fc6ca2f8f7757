"""The calls around a paged KV cache together, as a serving loop makes them: prompt pass with a window
and pinned first tokens, its K and V into pages, decode steps over the pages, verification of drafted
tokens, rollback and the next step - on bf16 pages and on FP8 pages, eager and as captured steps."""

import numpy as np
import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib, workloads as wl
from oracle import ref, serve
from serve_util import BF16, F16, check, score_error

pytestmark = pytest.mark.gpu

HQ, HKV, W, F, THETA, PAGE, V = 16, 2, 128, 4, 1.0e4, 16, 600
SCALE = 192 ** -0.5


def _rotate(x, pos):
    """x [B, H, 192] bf16 at positions pos [B], as the prefill rotates it, rounded to bf16."""
    r = np.stack([ref.rope(wl.to_f64(x[b:b + 1]), np.array([int(pos[b])]), THETA, 64)[0] for b in range(len(pos))])
    return torch.from_numpy(r).to(torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_generation(cuda_device, fp8):
    dev, B, n, extra = cuda_device, 2, 333, 12
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q = r(B, n + extra, HQ, 192).bfloat16()              # the token stream's projections, raw
    k = r(B, n + extra, HKV, 192).bfloat16()
    v = r(B, n + extra, HKV, 128).bfloat16()
    sink, unembed = r(HQ), r(HQ * 128, V) * 0.02
    width = -(-(n + extra) // PAGE)
    table = torch.randperm(B * width, generator=g).view(B, width).int().to(dev)
    dt = torch.uint8 if fp8 else torch.bfloat16
    pools = [torch.zeros(B * width, PAGE, HKV, d, dtype=dt, device=dev) for d in (192, 128)]
    scales = [torch.ones(B * width, PAGE, HKV, device=dev) for _ in range(2)]
    qd, kd, vd, sd = (t.to(dev) for t in (q, k, v, sink))

    def append(lo, hi, pos):
        a = (kd[:, lo:hi].contiguous(), vd[:, lo:hi].contiguous(), *pools)
        if fp8:
            _lib.cache_append_paged_fp8(*a, *scales, table, pos, rope_theta=THETA)
        else:
            _lib.cache_append_paged(*a, table, pos, rope_theta=THETA)

    def decode(qt, lengths):
        if fp8:
            return _lib.decode_paged_fp8(qt, *pools, *scales, table, lengths, sd, window=W, n_first=F)
        return _lib.decode_paged(qt, *pools, table, lengths, sd, window=W, n_first=F)

    # the prompt: chunks of 200 and 133, the second over the raw prefix
    o1, l1 = _lib.prefill_first(qd[:, :200].contiguous(), kd[:, :200].contiguous(), vd[:, :200].contiguous(), sd,
                                window=W, n_first=F, rope_theta=THETA)
    o2, l2 = _lib.prefill_first(qd[:, 200:n].contiguous(), kd[:, :n].contiguous(), vd[:, :n].contiguous(), sd, window=W,
                                n_first=F, pos_offset=200, k_prefix_rotated=False, rope_theta=THETA)
    at = torch.zeros(B, dtype=torch.int32, device=dev)
    append(0, 200, at)
    append(200, n, at + 200)
    delta = score_error(wl.to_f64(q), wl.to_f64(k), SCALE)
    rot = 2.0 * F16 * SCALE * np.linalg.norm(wl.to_f64(q)[..., :64], axis=-1).max() * np.linalg.norm(
        wl.to_f64(k)[..., :64], axis=-1).max()
    o, l, mass = serve.prefill_first(wl.to_f64(q[:, 190:n]), wl.to_f64(k[:, :n]), wl.to_f64(v[:, :n]), 190, False,
                                     wl.to_f64(sink), W, F, THETA, 64)
    torch.cuda.synchronize()
    got, gl = torch.cat([o1[:, 190:], o2], 1), torch.cat([l1[:, :, 190:], l2], 2)
    check(got, gl, o, l, mass, BF16, delta + rot, "prompt")

    def cache64():
        if fp8:
            return [ref.dequant_fp8(p.cpu().numpy(), s.cpu().numpy()) for p, s in zip(pools, scales)]
        return [wl.to_f64(p) for p in pools]

    lengths = torch.full((B,), n, dtype=torch.int32, device=dev)
    stream = list(range(n))                              # positions whose projections the sequence holds
    for step in range(3):
        # one step: the newest token, then three drafts, each attended over the pages
        outs = []
        for t in range(4):
            tok = len(stream) + t
            append(tok, tok + 1, lengths)
            lengths = lengths + 1
            qt = _rotate(q[:, tok], [tok] * B).to(dev)
            out, lse = decode(qt, lengths)
            torch.cuda.synchronize()
            kk, vv = cache64()
            o, l, mass, top = serve.decode_paged(wl.to_f64(qt), kk, vv, table.cpu().numpy(), lengths.tolist(), W, F,
                                                 wl.to_f64(sink))
            check(out, lse, o, l, mass, F16 + 2.0 ** -18 if fp8 else 2.0 ** -16, 2 * delta, f"step {step} token {t}",
                  extra=((W + F) * 2.0 ** -24 * top)[..., None] if fp8 else 0.0)
            outs.append(out.float().view(B, -1) @ unembed.to(dev))
        p = torch.softmax(torch.stack(outs, 1), -1)      # [B, 4, V]: rows for three drafts and the next token
        dq = torch.softmax(torch.stack(outs[:3], 1) + 0.5 * r(B, 3, V).to(dev), -1)
        draft = torch.multinomial(dq.view(-1, V).cpu(), 1, generator=g).view(B, 3).int().to(dev)
        u = torch.rand(B, 4, generator=g).to(dev)
        acc, tok = _lib.verify_drafts(p, draft, u, dq)
        torch.cuda.synchronize()
        a, want = serve.verify_drafts(wl.to_f64(p), wl.to_f64(dq), draft.cpu().numpy(), wl.to_f64(u))
        assert acc.tolist() == a.tolist() and tok.tolist() == want.tolist()
        # rollback: both sequences keep the fewest accepted, so that one stream serves them
        keep = 1 + int(acc.min())
        stream += list(range(len(stream), len(stream) + keep))
        lengths = torch.full((B,), len(stream), dtype=torch.int32, device=dev)
    assert _lib.last_device_error() == 0


def test_captured_steps_share_a_pool_and_a_workspace(cuda_device):
    """Two captured decode graphs over one pool, one workspace and one stream, replayed in turn with
    changing lengths: each as if it were alone."""
    dev, B = cuda_device, 3
    g = torch.Generator().manual_seed(6)
    pools = [torch.randn(40, PAGE, HKV, d, generator=g).bfloat16().to(dev) for d in (192, 128)]
    table = torch.randperm(40, generator=g)[:36].view(B, 12).int().to(dev)
    ws = torch.empty(_lib.decode_paged_workspace_size(B, HQ, HKV, max_pages=12, page_size=PAGE), dtype=torch.uint8,
                     device=dev)
    q = [torch.randn(B, HQ, 192, generator=g).bfloat16().to(dev) for _ in range(2)]
    L = [torch.tensor(x, dtype=torch.int32, device=dev) for x in ([100, 5, 192], [1, 64, 33])]
    out = [torch.empty(B, HQ, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            _lib.decode_paged(q[i], *pools, table, L[i], out=out[i], want_lse=False, workspace=ws, window=50 * i, n_first=2)
    for k in range(6):
        L[0].copy_(torch.tensor([10 * k, 5 + k, 192 - k]))
        L[1].copy_(torch.tensor([1, 64 + 3 * k, 33 * (k % 2)]))
        for i in (k % 2, 1 - k % 2):
            graphs[i].replay()
        want = [_lib.decode_paged(q[i], *pools, table, L[i], window=50 * i, n_first=2)[0] for i in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_streams_at_once(cuda_device):
    """The same call on two streams at the same time, each with its own scratch."""
    dev, B = cuda_device, 4
    g = torch.Generator().manual_seed(7)
    pools = [torch.randn(300, 64, 4, d, generator=g).bfloat16().to(dev) for d in (192, 128)]
    table = torch.randperm(300, generator=g)[:240].view(B, 60).int().to(dev)
    L = torch.tensor([3840, 100, 2000, 3000], dtype=torch.int32, device=dev)
    q = [torch.randn(B, 64, 192, generator=g).bfloat16().to(dev) for _ in range(2)]
    want = [_lib.decode_paged(x, *pools, table, L) for x in q]
    p = torch.softmax(torch.randn(8, 4, 5000, generator=g), -1).to(dev)
    draft, u = torch.randint(0, 5000, (8, 3), generator=g).int().to(dev), torch.rand(8, 4, generator=g).to(dev)
    tokens = _lib.verify_drafts(p, draft, u)[1]
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    torch.cuda.synchronize()
    got, tok = [[], []], []
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_lib.decode_paged(q[i], *pools, table, L))
                tok.append(_lib.verify_drafts(p, draft, u)[1])
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
    assert all(torch.equal(t, tokens) for t in tok)
