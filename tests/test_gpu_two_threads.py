"""Calls of different sizes from several host threads at once: every launch is
taken, and the results are those of one thread.  The threads repeat the C calls
themselves, so that as little as possible of their time is spent under Python's
lock."""
from __future__ import annotations

import threading

import pytest
import torch

from ssd_chunked_forward_b200 import ssd
from tests.linear_cases import slopes

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def scan(dtype, K, V):
    """Kernels on CUDA cores, whose shared memory goes by K."""
    g = torch.Generator(device="cuda").manual_seed(K)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v, decay = rnd(1, 4, 1, K), rnd(1, 4, 1, K), rnd(1, 4, 1, V), slopes(1)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    return lambda: ssd.linear_attention(q, k, v, decay, workspace=ws)


def norm(dtype, width, backward):
    """Blocks and rows ahead that go by the width."""
    g = torch.Generator(device="cuda").manual_seed(width)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, z, dy = rnd(2, width), rnd(2, width), rnd(2, width)
    stats = ssd.layer_norm(x, gate=z)[1]
    if not backward:
        return lambda: ssd.layer_norm(x, gate=z)

    def call():
        g = ssd.layer_norm_backward(x, None, None, dy, stats, gate=z, want_dweight=False, want_dbias=False)
        return g["dx"], g["dgate"]

    return call


def chunked(dtype, P, N, backward, per_state=False):
    """Kernels on CUDA cores, whose shared memory goes by the state's sizes."""
    g = torch.Generator(device="cuda").manual_seed(N)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, Bm, Cm = rnd(1, 8, 1, P), rnd(1, 8, 1, N), rnd(1, 8, 1, N)
    a = -torch.rand((1, 8, 1, N) if per_state else (1, 8, 1), generator=g, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    if not backward:
        return lambda: ssd.forward(x, a, Bm, Cm, None, 8, path=ssd.PATH_SIMT, workspace=ws)

    def call():
        g = ssd.backward(x, a, Bm, Cm, None, x, 8, want_dD=False, workspace=ws)
        return g["dx"], g["da"], g["dBm"], g["dCm"], g["dinit"]

    return call


PAIRS = {"scan": (lambda: scan(F32, 256, 16), lambda: scan(F32, 20, 16)),
         "scan bf16": (lambda: scan(BF, 250, 30), lambda: scan(BF, 36, 30)),
         # (blocks of 512 threads, and of 384 and 320)
         "norm": (lambda: norm(BF, 8192, False), lambda: norm(BF, 6000, False)),
         "norm gradients": (lambda: norm(F32, 4096, True), lambda: norm(F32, 2400, True)),
         "chunked": (lambda: chunked(F32, 16, 256, False), lambda: chunked(F32, 16, 20, False)),
         "per state": (lambda: chunked(F32, 16, 256, False, True), lambda: chunked(F32, 16, 20, False, True)),
         "chunked gradients": (lambda: chunked(F32, 64, 128, True), lambda: chunked(F32, 64, 64, True)),
         "per state gradients": (lambda: chunked(F32, 64, 128, True, True), lambda: chunked(F32, 64, 64, True, True))}


class Recorder:
    """The library, and every call that is made of it."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if name.endswith("size"):
            return fn

        def call(*args):
            self.calls.append((fn, args))
            return fn(*args)

        return call


@pytest.mark.parametrize("pair", PAIRS)
def test_threads_side_by_side(pair, monkeypatch):
    calls = [make() for make in PAIRS[pair]]  # (hold the inputs while the threads run)
    lib = Recorder(ssd.load())
    monkeypatch.setattr(ssd, "load", lambda: lib)
    out = [c() for c in calls]
    (one, a), (other, b) = lib.calls
    want = [[t.clone() for t in o] for o in out]
    torch.cuda.synchronize()
    start, codes = threading.Barrier(4), [set() for _ in range(4)]

    def run(i):
        fn, args = (one, a) if i % 2 else (other, b)
        start.wait()
        for _ in range(10000):
            codes[i].add(fn(*args))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{ssd.SSD_OK}] * 4
    assert all(torch.equal(a, b) for o, w in zip(out, want) for a, b in zip(o, w))
