"""Linear attention over long sequences: no wait of a call gives up, and the state
that outlives the call keeps its bits."""
from __future__ import annotations

import pytest
import torch

from ssd_chunked_forward_b200 import ssd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("K,V", [(8, 8), (128, 128)])
def test_no_wait_gives_up(K, V, packed):
    """One head and a long sequence: the blocks of the last launch start while the
    states' passes still run, and wait for them; the final state (the sums of the last
    tokens, since the decay leaves no more) says that they did."""
    T = (1 << 26) // (K + V)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(T, 1, d, generator=g, device="cuda", dtype=BF) for d in (K, K, V))
    decay = torch.tensor([-0.25], device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    e = (lambda t: t) if packed else (lambda t: t[None])
    shape = ssd.LinearShape(1, T, 1, 1, K, V, ssd.SSD_DTYPE_BF16, int(packed))
    for name, size in (("forward", ssd.linear_workspace_size), ("backward", ssd.linear_backward_workspace_size)):
        ws = torch.full((size(shape),), 0xFF, dtype=torch.uint8, device="cuda")
        if name == "forward":
            _, state = ssd.linear_attention(e(q), e(k), e(v), decay, cu_seqlens=cu, workspace=ws)
        else:
            state = ssd.linear_attention_backward(e(k), e(q), e(v), decay, e(v), scale=1.0, cu_seqlens=cu,
                                                  workspace=ws)["dinit"]
        assert ssd.device_status(ws) == ssd.SSD_OK, name
        n = 400  # exp(-100) is nothing
        w = torch.exp(-0.25 * torch.arange(n, device="cuda", dtype=torch.float64))
        kn, vn = (k[-n:, 0].flip(0), v[-n:, 0].flip(0)) if name == "forward" else (k[:n, 0], v[:n, 0])
        if name == "backward":
            w = w * torch.exp(torch.tensor(-0.25, dtype=torch.float64))
        kn, vn = kn.double() * w[:, None], vn.double()
        size_of = kn.abs().T @ vn.abs()
        # a few factors, the products of a chunk, the chunks that the state remembers
        assert bool(((state[0, 0].double() - kn.T @ vn).abs() <= 160 * 2 ** -24 * size_of).all()), name
