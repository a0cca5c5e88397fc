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


def one_token(dtype, K, V, H, T):
    """Sequences that hold one token, each head's somewhere in the last chunks: the state is
    one product, and what the kernels round of it cannot hide behind other terms."""
    g = torch.Generator(device="cuda").manual_seed(K + V)
    rnd = lambda d: torch.randn(H, d, generator=g, device="cuda").to(dtype)  # noqa: E731
    a, b, decay = rnd(K), rnd(V), -torch.linspace(0.01, 0.05, H, device="cuda")
    at = torch.randint(0, T - 1, (H,), generator=g, device="cuda")  # (not the last token, whose weight is 1)
    ka, vb = torch.zeros(1, T, H, K, device="cuda", dtype=dtype), torch.zeros(1, T, H, V, device="cuda", dtype=dtype)
    heads = torch.arange(H, device="cuda")
    ka[0, at, heads], vb[0, at, heads] = a, b
    return a.double(), b.double(), decay, at, ka, vb


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (64, 128), (128, 128), (40, 72)])
@pytest.mark.parametrize("H", [2, 148], ids=["cut", "whole"])
def test_states_keep_fp32(dtype, K, V, H):
    """final_state and dinit of one token.  Roundings on the way: the weight, its product with
    the token, the sums of that product's three pieces (two, a step of a truncating
    adder each), and for three chunks and three items a factor and a sum each.  A
    piece less in the tensor cores' products leaves 2^-16 (typically 2^-18)."""
    T = 300
    a, b, decay, at, ka, vb = one_token(dtype, K, V, H, T)
    rounds = 2 + 2 * 2 + 2 * 3 + 2 * 3
    outer = a[:, :, None] * b[:, None, :]
    _, final = ssd.linear_attention(ka, ka, vb, decay)
    want = torch.exp(decay.double() * (T - 1 - at))[:, None, None] * outer
    assert bool(((final[0].double() - want).abs() <= rounds * 2 ** -24 * want.abs()).all())
    # (scale enters dinit at the end, the decay of the first token's step before it)
    g = ssd.linear_attention_backward(ka, ka, vb, decay, vb, scale=0.3)
    want = 0.3 * torch.exp(decay.double() * (at + 1))[:, None, None] * outer
    assert bool(((g["dinit"][0].double() - want).abs() <= (rounds + 4) * 2 ** -24 * want.abs()).all())


@pytest.mark.parametrize("K,V", [(128, 64), (128, 128)])
def test_states_of_long_sequences(K, V):
    """65536 random tokens, memories up to thousands of them: the final state against
    the sum in 64 bits.  A term is rounded in its weight and product, in the sums of its chunk (8
    parts of three pieces, a step each), and then once for every chunk that the state
    remembers; the last only in proportion to the state itself."""
    T, H = 65536, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(1, T, H, d, generator=g, device="cuda", dtype=BF) for d in (K, V))
    decay = -torch.exp2(-torch.tensor([1.0, 5.0, 9.0, 12.0], device="cuda"))
    _, final = ssd.linear_attention(k, k, v, decay)
    for h in range(H):
        w = torch.exp(decay[h].double() * torch.arange(T - 1, -1, -1, device="cuda"))[:, None]
        kh, vh = k[0, :, h].double() * w, v[0, :, h].double()
        want, size = kh.T @ vh, kh.abs().T @ vh.abs()
        carried = 1 / (1 - torch.exp(128 * decay[h].double()))
        bound = (2 + 2 * 24) * 2 ** -24 * size + 2 * carried * 2 ** -24 * want.abs().max()
        assert bool(((final[0, h].double() - want).abs() <= bound).all())
