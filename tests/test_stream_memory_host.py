"""Calls with ``stream=``: memory that a call makes, clears or drops belongs to
the stream its kernels run on.  Without a GPU: tensors that only say they are on
one, a library that only notes its stream, and torch's stream calls replaced by
ones that keep the current stream's name."""
from __future__ import annotations

import contextlib

import pytest
import torch

from ssd_chunked_forward_b200 import ssd

BF, F32 = torch.bfloat16, torch.float32


class OnGPU(torch.Tensor):
    """A CUDA tensor without memory."""

    used_by = ()

    @staticmethod
    def __new__(cls, size, dtype):
        stride, n = [], 1
        for d in reversed(size):
            stride.insert(0, n)
            n *= d
        return torch.Tensor._make_wrapper_subclass(cls, size, strides=stride, dtype=dtype, device="cuda:0")

    __torch_function__ = torch._C._disabled_torch_function_impl

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} of a tensor without memory")

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.used_by = self.used_by + (stream,)


class Stream:
    device = torch.device("cuda:0")

    def __init__(self, handle):
        self.cuda_stream = handle


MAIN, SIDE = Stream(5000), Stream(6000)


@pytest.fixture
def world(monkeypatch):
    """A record of (what, stream): allocations, clearings and the library's calls."""
    seen, current = [], [MAIN]

    @contextlib.contextmanager
    def entered(s):
        current.append(s)
        yield
        current.pop()

    class Cuda:
        def __getattr__(self, name):
            return getattr(torch.cuda, name)

        Stream, stream = Stream, staticmethod(entered)
        current_device = staticmethod(lambda: 0)
        current_stream = staticmethod(lambda device=None: current[-1])
        default_stream = staticmethod(lambda device=None: MAIN)
        ExternalStream = staticmethod(lambda handle, device=None: {5000: MAIN, 6000: SIDE}[handle])

    class C:
        _cuda_getCurrentRawStream = staticmethod(lambda index: current[-1].cuda_stream)

    class Torch:
        cuda, _C = Cuda(), C()

        def __getattr__(self, name):
            return getattr(torch, name)

        @staticmethod
        def _make(what, size, dtype):
            seen.append((what, current[-1].cuda_stream))
            return OnGPU((size,) if isinstance(size, int) else tuple(size), dtype)

        def empty(self, size, dtype=F32, device=None):
            return self._make("empty", size, dtype)

        def zeros(self, size, dtype=F32, device=None):
            return self._make("zeros", size, dtype)

        def empty_like(self, t):
            return self._make("empty", t.shape, t.dtype)

    class Lib:
        def __getattr__(self, name):
            if name.endswith("size"):
                return lambda *a: 4096
            return lambda *a: seen.append((name, next(x for x in a if x in (5000, 6000)))) or 0

    monkeypatch.setattr(ssd, "torch", Torch())
    monkeypatch.setattr(ssd, "load", Lib)
    monkeypatch.setattr(ssd, "_plans", {})
    return seen


def t(*size, dtype=BF):
    return OnGPU(size, dtype)


CU = t(3, dtype=torch.int32)
Q, K, V, DECAY = t(20, 4, 64), t(20, 2, 64), t(20, 2, 128), t(4, dtype=F32)
X, W, STATS = t(6, 64), t(64, dtype=F32), t(6, 2, 2, dtype=F32)
CALLS = {
    "linear": lambda s: ssd.linear_attention(Q, K, V, DECAY, cu_seqlens=CU, stream=s),
    "linear_backward": lambda s: ssd.linear_attention_backward(Q, K, V, DECAY, t(20, 4, 128), cu_seqlens=CU, stream=s),
    "linear_step": lambda s: ssd.linear_attention_step(Q, K, V, DECAY, t(20, 4, 64, 128, dtype=F32), stream=s),
    "norm": lambda s: ssd.layer_norm(X, W, W, groups=2, stream=s),
    "norm_backward": lambda s: ssd.layer_norm_backward(X, W, W, X, STATS, groups=2, stream=s),
}

XS, A, BM, D = t(2, 8, 4, 16), t(2, 8, 4, dtype=F32), t(2, 8, 1, 32), t(4, dtype=F32)
STATE, SHAPE = t(2, 4, 32, 16, dtype=F32), ssd.make_shape(2, 8, 4, 16, 1, 32, 8)
CALLS |= {
    "forward": lambda s: ssd.forward(XS, A, BM, BM, D, 8, stream=s),
    "forward_init": lambda s: ssd.forward(XS, A, BM, BM, D, 8, initial_state=STATE, stream=s),
    "forward_noalloc": lambda s: ssd.forward_noalloc(XS, A, BM, BM, D, 8, stream=s),
    "forward_discretized": lambda s: ssd.forward_discretized(XS, A, D, D, BM, BM, D, 8, stream=s),
    "backward": lambda s: ssd.backward(XS, A, BM, BM, D, XS, 8, stream=s),
    "decode_step": lambda s: ssd.decode_step(t(2, 4, 16), t(2, 4, dtype=F32), t(2, 1, 32), t(2, 1, 32), D, STATE, stream=s),
    "discretize": lambda s: ssd.discretize(A, D, D, XS, stream=s),
    "decay_total": lambda s: ssd.decay_total(A, stream=s),
    "segment_state": lambda s: ssd.segment_state(XS, A, BM, 8, stream=s),
    "state_combine": lambda s: ssd.state_combine(t(3, 2, 4, 32, 16, dtype=F32), t(3, 2, 4, dtype=F32), stream=s),
    "chunk_cumsum": lambda s: ssd.chunk_cumsum(SHAPE, A, None, s),
    "chunk_state": lambda s: ssd.chunk_state(SHAPE, XS, BM, A, stream=s),
    "chunk_scan": lambda s: ssd.chunk_scan(SHAPE, XS, BM, BM, A, STATE, stream=s),
}


def results(out):
    return [r for r in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,))
            if r is not None]


@pytest.mark.parametrize("given", [SIDE, 6000], ids=["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_everything_happens_on_the_given_stream(world, name, given):
    out = CALLS[name](given)
    assert any(what == "empty" for what, _ in world) and any(what.startswith("ssd_") for what, _ in world)
    assert all(s == 6000 for _, s in world), world
    assert all(r.used_by == (MAIN,) for r in results(out))  # the caller's stream may read them and drop them


@pytest.mark.parametrize("given", [None, MAIN, 5000], ids=["none", "stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_otherwise(world, name, given):
    out = CALLS[name](given)
    assert all(s == 5000 for _, s in world), world
    assert all(r.used_by == () for r in results(out))


def test_what_the_caller_gave_stays_the_callers(world):
    y = t(20, 4, 128)
    out, final = ssd.linear_attention(Q, K, V, DECAY, cu_seqlens=CU, y=y, stream=SIDE)
    assert out is y and y.used_by == () and final.used_by == (MAIN,)


def test_addresses_instead_of_tensors(world):
    assert ssd.chunk_cumsum(SHAPE, 1 << 20, 1 << 21, stream=SIDE) == 1 << 21
    assert world == [("ssd_chunk_cumsum", 6000)]


def test_a_stream_of_another_device_is_refused(world):
    other = Stream(6000)
    other.device = torch.device("cuda:1")
    with pytest.raises(ValueError, match="stream"):
        ssd.layer_norm(X, W, W, stream=other)
