"""Draft verification against the float64 oracle: whole numbers, which have to be equal."""

import numpy as np
import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib, workloads as wl
from oracle import serve


def _case(B, T, V, seed, dtype=torch.float32, greedy=False, sharp=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, T + 1, V, generator=g) * sharp
    p = torch.softmax(logits, -1).to(dtype)
    near = logits[:, :T] + 0.7 * torch.randn(B, T, V, generator=g)
    q = torch.softmax(near, -1)
    draft = q.argmax(-1) if greedy or T == 0 else torch.multinomial(q.reshape(-1, V), 1, generator=g).view(B, T)
    return dict(p=p, q=None if greedy else q.to(dtype), draft=draft.int(), u=torch.rand(B, T + 1, generator=g))


def _check(c, dev, n_valid=None):
    d = {k: None if v is None else v.to(dev) for k, v in c.items()}
    nv = None if n_valid is None else torch.tensor(n_valid, dtype=torch.int32)
    acc, tok = _lib.verify_drafts(d["p"], d["draft"], d["u"], d["q"], n_valid=None if nv is None else nv.to(dev))
    torch.cuda.synchronize()
    f = lambda t: None if t is None else wl.to_f64(t)  # noqa: E731
    a, t = serve.verify_drafts(f(c["p"]), f(c["q"]), c["draft"].numpy(), f(c["u"]), n_valid)
    assert np.array_equal(acc.cpu().numpy(), a), (acc.tolist(), a.tolist())
    assert np.array_equal(tok.cpu().numpy(), t), (tok.tolist(), t.tolist())
    return a, t


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,T,V", [(1, 3, 32000), (5, 0, 700), (64, 3, 1000), (3, 8, 50021), (40, 1, 1), (16, 2, 33),
                                   (7, 40, 129), (2, 3, 131072), (9, 3, 2047)])
def test_against_the_oracle(cuda_device, B, T, V, dtype, greedy):
    _check(_case(B, T, V, B + T + V, dtype, greedy), cuda_device)


@pytest.mark.gpu
def test_counts_vary(cuda_device):
    a, _ = _check(_case(64, 4, 500, 3), cuda_device)
    assert set(a.tolist()) == {0, 1, 2, 3, 4}          # every way to leave the loop is taken


@pytest.mark.gpu
def test_ragged_drafts(cuda_device):
    _check(_case(8, 4, 300, 4), cuda_device, n_valid=[0, 1, 2, 3, 4, -2, 9, 2])
    _check(_case(8, 4, 300, 5, greedy=True), cuda_device, n_valid=[0, 1, 2, 3, 4, -2, 9, 2])


@pytest.mark.gpu
def test_borders(cuda_device):
    """u at 0, next to a border of the running sum and next to 1; p = q; p below q everywhere."""
    V = 1024
    p = torch.full((6, 2, V), 1.0 / V)
    q = torch.full((6, 1, V), 1.0 / V)
    draft = torch.arange(6, dtype=torch.int32).view(6, 1)
    u = torch.zeros(6, 2)
    below = np.nextafter(np.float32(1), np.float32(0))
    u[:, 1] = torch.tensor([0.0, 0.5, np.nextafter(np.float32(0.5), np.float32(0)), below, 3 / V, 1.0])
    u[:, 0] = torch.tensor([0.0, below, 0.25, 0.5, 1.0, 0.0])
    c = dict(p=p, q=q, draft=draft, u=u)
    a, t = _check(c, cuda_device)
    assert a.tolist() == [1, 1, 1, 1, 0, 1]            # u q < p: u = 1 rejects p = q, and all of p is sampled
    assert t[:, 1].tolist() == [0, 512, 511, 1023, -1, 1023] and t[4, 0] == 3
    c["q"] = q * 2                                     # nothing is left of p - q
    c["u"] = torch.rand(6, 2, generator=torch.Generator().manual_seed(1)) * 0.4 + 0.55
    a, _ = _check(c, cuda_device)
    assert a.tolist() == [0] * 6


@pytest.mark.gpu
def test_rows_without_mass_and_bad_values(cuda_device):
    c = _case(6, 2, 777, 6)
    c["p"][0] = 0                                      # no mass at all: the token is -1
    c["p"][1, 0, :] = float("nan")
    c["p"][2, 0, 5:9] = float("inf")
    c["q"][2, 0] = 0.5
    c["p"][3, 0, ::2] = -1.0
    c["draft"][4, 0] = 777                             # outside the vocabulary
    c["draft"][5, 0] = -1
    a, t = _check(c, cuda_device)
    assert t[0].tolist() == [-1, -1, -1] and a[0] == 0
    c["u"][:, 1] = float("nan")
    _check(c, cuda_device)


@pytest.mark.gpu
def test_single_token_mass_and_sharp_rows(cuda_device):
    _check(_case(32, 3, 5000, 7, sharp=30.0), cuda_device)
    c = _case(4, 1, 4097, 8)
    c["p"].zero_()
    for b, v in enumerate((0, 4096, 2048, 127)):
        c["p"][b, :, v] = 1e-40                        # a subnormal weight is mass too
    c["u"].fill_(0.999)
    _, t = _check(c, cuda_device)
    assert [r[0] for r in t.tolist()] == [0, 4096, 2048, 127]


@pytest.mark.gpu
def test_distribution(cuda_device):
    """Over many uniforms the emitted first token follows the target's distribution (the point of the
    rule): counts within 5 standard deviations."""
    V, N = 16, 40000
    g = torch.Generator().manual_seed(9)
    p1, q1 = torch.softmax(torch.randn(V, generator=g) * 1.5, -1), torch.softmax(torch.randn(V, generator=g) * 1.5, -1)
    draft = torch.multinomial(q1, N, replacement=True, generator=g).int().view(N, 1)
    acc, tok = _lib.verify_drafts(p1.expand(N, 2, V).contiguous().to(cuda_device), draft.to(cuda_device),
                                  torch.rand(N, 2, generator=g).to(cuda_device),
                                  q1.expand(N, 1, V).contiguous().to(cuda_device))
    got = np.bincount(tok[:, 0].cpu().numpy(), minlength=V)
    want = wl.to_f64(p1) * N
    assert (np.abs(got - want) <= 5 * np.sqrt(want) + 1).all()


@pytest.mark.gpu
def test_streams_graph_and_buffers(cuda_device):
    c = {k: v.to(cuda_device) for k, v in _case(4, 3, 9000, 10).items()}
    want = _lib.verify_drafts(c["p"], c["draft"], c["u"], c["q"])
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    got = _lib.verify_drafts(c["p"], c["draft"], c["u"], c["q"], stream=side)
    acc = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    tok = torch.zeros(4, 4, dtype=torch.int32, device=cuda_device)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.verify_drafts(c["p"], c["draft"], c["u"], c["q"], n_accepted=acc, tokens=tok)
    for s in range(3):
        c["u"].copy_(torch.rand(4, 4, generator=torch.Generator().manual_seed(s)))
        graph.replay()
        want = _lib.verify_drafts(c["p"], c["draft"], c["u"], c["q"])
        torch.cuda.synchronize()
        assert torch.equal(acc, want[0]) and torch.equal(tok, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,V", [(torch.float32, 2 ** 27), (torch.float32, 2 ** 27 - 3), (torch.bfloat16, 2 ** 27),
                                     (torch.bfloat16, 2 ** 27 - 3)])
def test_long_rows(cuda_device, dtype, V):
    """Equal weights, 2^15 of them to a lane's sum: with V (24-bit) weights every running sum is a whole
    multiple of one, exact in 64 bits, so that the token is floor(u V), whatever the weight. A sum that
    carried its errors in 32 bits over the whole piece drifts by tens of tokens here."""
    u = torch.tensor([0.25, 0.7311, 0.99999])
    for weight in (1.37 / V, 1.0 / V, 0.73 / V):
        p = torch.full((1, 1, V), weight, dtype=dtype, device=cuda_device)
        for x in u:
            acc, tok = _lib.verify_drafts(p, torch.empty(1, 0, dtype=torch.int32, device=cuda_device), x.view(1, 1).to(cuda_device))
            assert acc.tolist() == [0]
            assert tok.item() == int(np.floor(float(x) * V)), (weight, float(x))
        del p
