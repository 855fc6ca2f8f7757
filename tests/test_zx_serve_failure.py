"""Failure detection of the window prefill kernels and the paged decode, without faulting or hanging
the GPU: the test builds of test_zy_failure_detection.py (waits that give up after 1 ns; debug checks),
then the product build on the same context."""

import contextlib
import ctypes

import pytest
import torch

from hybrid_sliding_window_sink_b200 import _lib, build, workloads as wl

pytestmark = pytest.mark.gpu

MIMO_OK, MIMO_ERR_DEVICE = 0, 7
WAIT_TIMEOUT, DRAIN_TIMEOUT, BAD_LENGTH, F16_RANGE = 1, 2, 4, 16


@contextlib.contextmanager
def _library(name):
    lib = _lib.load(build.build(variant=name))
    saved = _lib._LIB
    _lib._LIB = lib
    try:
        yield lib
    finally:
        _lib._LIB = saved


def _status(lib):
    word = ctypes.c_uint(0)
    return lib.mimo_attn_device_status(ctypes.byref(word)), word.value


CASES = [(640, 64, 8, 128, 4), (640, 64, 4, 200, 40), (300, 16, 4, 64, 9), (16, 8, 1, 128, 4),
         (16, 16, 1, 8, 4)]   # ring, pair, generic kernel, and a single block of the first two


def _run(x, dev, window, first):
    return _lib.prefill_first(*(x[k].to(dev) for k in ("q", "k", "v", "sink")), window=window, n_first=first)


def test_window_kernels_give_up_and_the_context_stays_usable(cuda_device):
    inputs = [wl.prefill_inputs(1, n, hq, hkv, seed=80 + n) for n, hq, hkv, _, _ in CASES]
    want = [_run(x, cuda_device, c[3], c[4]) for x, c in zip(inputs, CASES)]
    torch.cuda.synchronize()
    with _library("shortwait") as lib:
        assert _status(lib) == (MIMO_OK, 0)
        for i, (x, c) in enumerate(zip(inputs, CASES)):
            _run(x, cuda_device, c[3], c[4])
            st, word = _status(lib)
            assert st == (MIMO_ERR_DEVICE if word else MIMO_OK) and not word & DRAIN_TIMEOUT, (c, word)
            if i < 2:
                assert word == WAIT_TIMEOUT, (c, word)
    for x, c, w in zip(inputs, CASES, want):
        got = _run(x, cuda_device, c[3], c[4])
        torch.cuda.synchronize()
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1]), c
    assert _status(_lib.lib()) == (MIMO_OK, 0)


def test_debug_build(cuda_device):
    """Valid calls leave the error word clear and give the product build's results; lengths outside the
    table and operands beyond f16 are recorded."""
    dev = cuda_device
    inputs = [wl.prefill_inputs(1, n, hq, hkv, seed=80 + n) for n, hq, hkv, _, _ in CASES]
    want = [_run(x, dev, c[3], c[4]) for x, c in zip(inputs, CASES)]
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(8, 16, 2, 192, generator=g).bfloat16().to(dev), torch.randn(8, 16, 2, 128, generator=g).bfloat16().to(dev)
    k8, ks = wl.fp8_cache(k)
    v8, vs = wl.fp8_cache(v)
    q = torch.randn(2, 16, 192, generator=g).bfloat16().to(dev)
    table = torch.arange(8, dtype=torch.int32, device=dev).view(2, 4)
    L = torch.tensor([64, 30], dtype=torch.int32, device=dev)
    calls = [lambda n=L: _lib.decode_paged(q, k, v, table, n), lambda n=L: _lib.decode_paged_fp8(q, k8, v8, ks, vs, table, n)]
    good = [c() for c in calls]
    torch.cuda.synchronize()
    with _library("debug") as lib:
        for x, c, w in zip(inputs, CASES, want):
            got = _run(x, dev, c[3], c[4])
            assert _status(lib) == (MIMO_OK, 0), c
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1]), c
            bad = dict(x, k=x["k"].clone())
            bad["k"][0, c[0] // 2, 0, 5] = 1e5            # a rotated dim, carried in f16
            _run(bad, dev, c[3], c[4])
            assert _status(lib) == (MIMO_ERR_DEVICE, F16_RANGE), c
        for call, w in zip(calls, good):
            got = call()
            assert _status(lib) == (MIMO_OK, 0)
            assert torch.equal(got[0], w[0])
            for lengths in ([65, 30], [64, -1]):
                call(torch.tensor(lengths, dtype=torch.int32, device=dev))
                assert _status(lib) == (MIMO_ERR_DEVICE, BAD_LENGTH)
        q[0, 0, 7] = 1e5
        calls[1]()
        assert _status(lib) == (MIMO_ERR_DEVICE, F16_RANGE)
