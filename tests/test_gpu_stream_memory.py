"""Calls with ``stream=`` while the caller's own stream is busy: nothing that is
queued there before or after, and no memory that is allocated there, touches what
the call makes or uses."""
from __future__ import annotations

import pytest
import torch

from ssd_chunked_forward_b200 import ssd
from tests.linear_cases import slopes

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def linear(dtype, K, V):
    cuts, total, H, G = [5, 140, 140, 2400], 2460, 4, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    q, k, v, dy, decay = rnd(total, H, K), rnd(total, G, K), rnd(total, G, V), rnd(total, H, V), slopes(H)
    init = rnd(3, H, K, V, dt=F32)

    def call(stream):
        y, final = ssd.linear_attention(q, k, v, decay, initial_state=init, cu_seqlens=cu, stream=stream)
        grads = ssd.linear_attention_backward(q, k, v, decay, dy, initial_state=init, dfinal=init, cu_seqlens=cu,
                                              stream=stream)
        return {"y": y[5:2400], "final": final, **grads}

    return call


def norm(dtype, K, V):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, z, dy, w, b = rnd(4000, K), rnd(4000, K), rnd(4000, K), rnd(K, dt=F32), rnd(K, dt=F32)

    def call(stream):
        y, stats = ssd.layer_norm(x, w, b, groups=K // V, gate=z, stream=stream)
        return {"y": y, **ssd.layer_norm_backward(x, w, b, dy, stats, groups=K // V, gate=z, stream=stream)}

    return call


def chunked(dtype, K, V):
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, Bm, Cm, dy, D = rnd(2, 512, 4, V), rnd(2, 512, 1, K), rnd(2, 512, 1, K), rnd(2, 512, 4, V), rnd(4, dt=F32)
    a = -torch.rand(2, 512, 4, generator=g, device="cuda")

    def call(stream):
        y, final = ssd.forward(x, a, Bm, Cm, D, 128, stream=stream)
        return {"y": y, "final": final, **ssd.backward(x, a, Bm, Cm, D, dy, 128, dfinal=final, stream=stream)}

    return call


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("make,dtype,K,V", [(linear, BF, 128, 64), (linear, BF, 64, 64), (linear, F32, 24, 20),
                                            (norm, BF, 1536, 64), (norm, F32, 700, 700), (chunked, BF, 128, 64),
                                            (chunked, F32, 24, 20)])
def test_the_callers_stream_is_busy(make, dtype, K, V, handle):
    call = make(dtype, K, V)
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(40_000_000)  # some 20 ms, in which the side stream gets done
        got = call(side.cuda_stream if handle else side)
        # memory of many sizes, filled on the caller's stream
        junk = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device="cuda") for n in range(9, 26)]
        ends = torch.cuda.Event()
        ends.record(side)
        ends.synchronize()
        side_first = {n: t.clone() for n, t in got.items()}  # (queued behind the sleep)
        torch.cuda.synchronize()
        del junk
        for n, t in want.items():
            assert torch.equal(t, got[n]) and torch.equal(t, side_first[n]), n


def test_results_dropped_while_the_callers_stream_reads_them():
    """A result that the caller's stream still reads when its last name goes is not handed
    out again to the side stream."""
    call = norm(BF, 1536, 64)
    want = call(None)["y"].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    copies = []
    for _ in range(8):
        y = call(side)["y"]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(4_000_000)
        copies.append(y.clone())
        del y
        with torch.cuda.stream(side):
            torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in copies)


@pytest.mark.parametrize("make,dtype,K,V", [(linear, BF, 128, 64), (norm, BF, 1536, 64)])
def test_captured_on_a_branch(make, dtype, K, V):
    """A call on a side stream that has joined a capture: its memory is the graph's, and
    replays give the results again."""
    call = make(dtype, K, V)
    want = call(None)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        held = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in held.values():
            t.fill_(7.0)
        graph.replay()
        junk = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device="cuda") for n in range(9, 26)]
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(held[n], want[n]) for n in want)
