"""Refusals of the calls around a paged KV cache, before any launch (no GPU work), and the oracle's
own definitions against each other."""

import ctypes

import numpy as np
import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib
from hybrid_sliding_window_sink_b200.build import build
from oracle import ref, serve

P = ctypes.c_void_p
GOOD, ODD = P(0x10000), P(0x10002)     # never dereferenced: every case below fails validation first


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


def _shape(batch=2, seqlen=3, hq=8, hkv=1, dqk=192, dv=128, scale=0.0):
    return _lib.make_shape(batch, seqlen, hq, hkv, dqk, dv, scale)


def _pages(table=0x10000, max_pages=4, num_pages=9, page=16, stride=16):
    return _lib.MimoPages(table, max_pages, num_pages, page, stride)


BAD_PAGES = [(_pages(table=None), 1), (_pages(max_pages=0), 2), (_pages(num_pages=0), 2), (_pages(page=0), 2),
             (_pages(page=-1), 2), (_pages(stride=15), 2), (_pages(max_pages=2 ** 20, page=2048, stride=2048), 3),
             (_pages(table=0x10002), 4)]


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_paged_rejects(L, fp8):
    def call(shape=None, q=GOOD, k=GOOD, v=GOOD, ks=GOOD, vs=GOOD, pages=None, lengths=GOOD, first=0, sink=None,
             out=GOOD, lse=None, ws=None, nbytes=0):
        shape, pages = _shape() if shape is None else shape, _pages() if pages is None else pages
        if fp8:
            return L.mimo_attn_decode_paged_fp8(shape, q, k, v, ks, vs, pages, lengths, 0, first, sink, out, lse, ws,
                                                nbytes, None)
        return L.mimo_attn_decode_paged(shape, q, k, v, pages, lengths, 0, first, sink, out, lse, ws, nbytes, None)

    for name in ("q", "k", "v", "lengths", "out") + (("ks", "vs") if fp8 else ()):
        assert call(**{name: None}) == 1, name
        assert call(**{name: ODD}) == 4, name
    for bad, code in BAD_PAGES:
        assert call(pages=bad) == code
    for bad, code in ((_shape(batch=0), 2), (_shape(hq=6, hkv=4), 2), (_shape(hq=3), 3), (_shape(hq=32), 3),
                      (_shape(dqk=128), 3), (_shape(dv=64), 3), (_shape(batch=70000), 3),
                      (_shape(scale=float("nan")), 2), (_shape(batch=65535, hq=65535, hkv=65535), 3)):
        assert call(shape=bad) == code
    assert call(first=-1) == 2
    assert call(sink=ODD) == 4 and call(lse=ODD) == 4
    assert call() in (5, 6)                # no workspace (a GPU is there), or no GPU


def test_workspace_size(L):
    def size(shape=None, pages=None, window=0, first=0):
        return L.mimo_attn_decode_paged_workspace_size(_shape() if shape is None else shape,
                                                       _pages() if pages is None else pages, window, first)
    assert size() > 0
    assert size(pages=_pages(max_pages=2)) == 0            # 32 tokens: one tile, nothing to join
    assert size(window=20, first=12) == 0 and size(window=20, first=13) > 0
    assert size(shape=_shape(hq=3)) == 0 and size(pages=_pages(page=0)) == 0 and size(first=-1) == 0
    # bounded by the CTAs, not by the batch or the length
    assert size(shape=_shape(batch=60000), pages=_pages(max_pages=100000)) < 8 << 20


@pytest.mark.parametrize("fp8", [False, True])
def test_append_rejects(L, fp8):
    def call(shape=None, kn=GOOD, vn=GOOD, pos=GOOD, n_new=None, theta=1e4, rot=64, pages=None, k=GOOD, v=GOOD,
             ks=GOOD, vs=GOOD):
        shape, pages = _shape(hq=1) if shape is None else shape, _pages() if pages is None else pages
        if fp8:
            return L.mimo_attn_cache_append_paged_fp8(shape, kn, vn, pos, n_new, theta, rot, pages, k, v, ks, vs, None)
        return L.mimo_attn_cache_append_paged(shape, kn, vn, pos, n_new, theta, rot, pages, k, v, None)

    for name in ("kn", "vn", "pos", "k", "v") + (("ks", "vs") if fp8 else ()):
        assert call(**{name: None}) == 1, name
        assert call(**{name: ODD}) == 4, name
    assert call(n_new=ODD) == 4
    for bad, code in BAD_PAGES:
        assert call(pages=bad) == code
    assert call(shape=_shape(hq=1, seqlen=0)) == 2 and call(shape=_shape(hq=1, dqk=64)) == 3
    assert call(rot=-16) == 2 and call(rot=208) == 2 and call(rot=24) == 3
    assert call(theta=0.0) == 2 and call(theta=float("inf")) == 2 and call(theta=float("nan")) == 2
    assert call(shape=_shape(batch=65535, seqlen=2 ** 31 - 1, hq=1)) == 3


def test_verify_rejects(L):
    def call(B=2, T=3, V=100, kind=0, p=GOOD, q=GOOD, draft=GOOD, u=GOOD, nv=None, acc=GOOD, tok=GOOD):
        return L.mimo_attn_verify_drafts(B, T, V, kind, p, q, draft, u, nv, acc, tok, None)

    for name in ("p", "draft", "u", "acc", "tok"):
        assert call(**{name: None}) == 1, name
    for name in ("p", "q", "draft", "u", "nv", "acc", "tok"):
        assert call(**{name: ODD}) == 4, name
    assert call(kind=1, p=P(0x10001)) == 4 and call(kind=1, q=P(0x10001)) == 4
    assert call(B=0) == 2 and call(T=-1) == 2 and call(V=0) == 2 and call(kind=2) == 2
    assert call(B=65536) == 3 and call(V=2 ** 30 + 1) == 3


def test_python_side_rejects_cpu_tensors():
    z = torch.zeros
    q, k, v = z(1, 8, 192).bfloat16(), z(2, 16, 1, 192).bfloat16(), z(2, 16, 1, 128).bfloat16()
    t, n = z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        _lib.decode_paged(q, k, v, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        _lib.cache_append_paged(k, v, k, v, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        _lib.verify_drafts(z(1, 2, 9), z(1, 1, dtype=torch.int32), z(1, 2))
    with pytest.raises(TypeError):
        _lib.decode_paged(None, k, v, t, n)


def test_pool_geometry():
    k, v = torch.zeros(4, 16, 2, 192), torch.zeros(4, 16, 2, 128)
    t = torch.zeros(1, 3, dtype=torch.int32)
    p = _lib._pages(k, v, t)
    assert (p.max_pages, p.num_pages, p.page_size, p.page_stride_tokens) == (3, 4, 16, 16)
    assert _lib._pages(k[:, :10], v[:, :10], t).page_stride_tokens == 16
    both = torch.zeros(4, 2, 16, 2, 192)                  # K and V pages interleaved: K's stride is 32 tokens
    wide = torch.zeros(4, 32, 2, 128)[:, :16]
    assert _lib._pages(both[:, 0], wide, t).page_stride_tokens == 32
    with pytest.raises(ValueError, match="same distance"):
        _lib._pages(both[:, 0], v, t)
    with pytest.raises(ValueError, match="contiguous within"):
        _lib._pages(k.transpose(1, 2).contiguous().transpose(1, 2), v, t)
    with pytest.raises(ValueError, match="whole tokens"):
        _lib._pages(torch.zeros(40000).as_strided((4, 16, 2, 192), (16 * 384 + 192, 384, 192, 1)), v, t)
    with pytest.raises(ValueError, match="overlap"):
        _lib._pages(torch.zeros(40000).as_strided((4, 16, 2, 192), (384, 384, 192, 1)), v, t)
    with pytest.raises(ValueError, match="no page"):
        _lib._pages(k[:0], v[:0], t)


# ------------------------------------------------------------------ the oracle's definitions
def test_oracle_paged_is_the_linear_decode():
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(2, 4, 8)), g.normal(size=(2, 12, 2, 8)), g.normal(size=(2, 12, 2, 4))
    table = np.array([[3, 0, 5], [4, 1, 2]])
    at = table.reshape(-1).argsort()                      # page i holds block at[i] of the flattened sequences
    pool = lambda x: x.reshape(6, 4, 2, -1)[at]  # noqa: E731
    sink = g.normal(size=4)
    o, l, mass, _ = serve.decode_paged(q, pool(k), pool(v), table, [11, 5], 0, 0, sink)
    want = ref.decode(q, k, v, "linear", [11, 5], sink)
    assert np.allclose(o, want[0], atol=1e-13) and np.allclose(l, want[1], atol=1e-13)
    assert (mass >= np.abs(o) - 1e-15).all()
    # a window is the ring of that many slots
    o, _, _, _ = serve.decode_paged(q, pool(k), pool(v), table, [11, 5], 4, 0, sink)
    ring = np.stack([[k[b][[t for t in range(L - 4, L) if t % 4 == s][0]] for s in range(4)] for b, L in enumerate((11, 5))])
    ringv = np.stack([[v[b][[t for t in range(L - 4, L) if t % 4 == s][0]] for s in range(4)] for b, L in enumerate((11, 5))])
    assert np.allclose(o, ref.decode(q, ring, ringv, "ring", [11, 5], sink)[0], atol=1e-13)


def test_oracle_first_keys():
    assert serve.first_keys(9, 4, 0).tolist() == [6, 7, 8, 9]
    assert serve.first_keys(9, 4, 2).tolist() == [0, 1, 6, 7, 8, 9]
    assert serve.first_keys(9, 4, 8).tolist() == list(range(10))
    assert serve.first_keys(2, 4, 3).tolist() == [0, 1, 2]
    assert serve.first_keys(9, 0, 3).tolist() == list(range(10))
    assert serve.first_keys(0, 1, 5).tolist() == [0]


def test_oracle_verify_by_hand():
    p = np.array([[[0.5, 0.5, 0.0], [0.25, 0.25, 0.5]]])
    q = np.array([[[0.25, 0.75, 0.0]]])
    run = lambda d, u: tuple(x.tolist() for x in serve.verify_drafts(p, q, np.array([[d]]), np.array([u])))  # noqa: E731
    assert run(1, [0.5, 0.3]) == ([1], [[1, 1]])          # 0.5 * 0.75 < 0.5; 0.25 is not > 0.3
    assert run(1, [0.7, 0.9]) == ([0], [[0, -1]])         # rejected: only token 0 has p > q
    assert run(2, [0.0, 0.0]) == ([0], [[0, -1]])         # 0 < 0 does not hold
    assert run(0, [0.99, 0.999]) == ([1], [[0, 2]])
    one = tuple(x.tolist() for x in serve.verify_drafts(p, None, np.array([[0]]), np.array([[0.6, 0.0]])))
    assert one == ([0], [[1, -1]])                        # argmax drafts: accepted with p(x), x leaves the rest


def test_prefill_first_rejects(L):
    def call(shape=None, q=GOOD, k=GOOD, v=GOOD, off=0, sink=None, window=128, first=4, theta=1e4, rot=64, out=GOOD,
             lse=None):
        return L.mimo_attn_prefill_first(_shape() if shape is None else shape, q, k, v, off, 0, sink, window, first,
                                         theta, rot, out, lse, None)
    for name in ("q", "k", "v", "out"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: ODD}) == 4, name
    assert call(sink=ODD) == 4 and call(lse=ODD) == 4
    assert call(first=-1) == 2 and call(off=-1) == 2 and call(shape=_shape(seqlen=0)) == 2
    assert call(off=2 ** 31 - 2) == 3 and call(shape=_shape(hq=3)) == 3 and call(rot=8) == 3
    assert call(rot=-16) == 2 and call(rot=208) == 2 and call(theta=0.0) == 2
    with pytest.raises(ValueError, match="CUDA"):
        _lib.prefill_first(torch.zeros(1, 2, 8, 192).bfloat16(), None, None, window=1, n_first=1)
