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


PAIRS = {"scan": (lambda: scan(F32, 256, 16), lambda: scan(F32, 20, 16)),
         "scan bf16": (lambda: scan(BF, 250, 30), lambda: scan(BF, 36, 30)),
         # (blocks of 512 threads, and of 384 and 320)
         "norm": (lambda: norm(BF, 8192, False), lambda: norm(BF, 6000, False)),
         "norm gradients": (lambda: norm(F32, 4096, True), lambda: norm(F32, 2400, True))}


@pytest.mark.parametrize("pair", PAIRS)
def test_threads_side_by_side(pair, monkeypatch):
    calls = [make() for make in PAIRS[pair]]  # (hold the inputs while the threads run)
    queued, call = [], ssd._call
    monkeypatch.setattr(ssd, "_call", lambda where, dev, fn, *a: (queued.append((fn, a)), call(where, dev, fn, *a)))
    out = [c() for c in calls]
    want = [[t.clone() for t in o] for o in out]
    torch.cuda.synchronize()
    start, codes = threading.Barrier(4), [set() for _ in range(4)]

    def run(i):
        fn, args = queued[i % 2]
        stream = streams[i].cuda_stream
        start.wait()
        for _ in range(10000):
            codes[i].add(fn(*args, stream))

    # the two of a size write the same results
    streams = [torch.cuda.Stream() for _ in range(4)]
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{ssd.SSD_OK}] * 4
    assert all(torch.equal(a, b) for o, w in zip(out, want) for a, b in zip(o, w))
