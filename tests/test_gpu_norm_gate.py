"""The gate of the layer norm over the whole range of its sigmoid: y = silu(gate)
and dgate = silu'(gate) on their own (weight 0, bias 1)."""
from __future__ import annotations

import pytest
import torch

from ssd_chunked_forward_b200 import ssd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gate_from_end_to_end(dtype):
    z = torch.cat([torch.linspace(-110, 110, 8000), torch.linspace(-4, 4, 190), torch.zeros(2)]).to(dtype).cuda()
    z = z.view(32, 256)
    x = torch.randn(z.shape, device="cuda").to(dtype)
    w, b = torch.zeros(256, device="cuda"), torch.ones(256, device="cuda")
    y, stats = ssd.layer_norm(x, w, b, gate=z)
    g = ssd.layer_norm_backward(x, w, b, torch.ones_like(x), stats, gate=z)
    d = z.double()
    s = torch.sigmoid(d)
    own = 2 ** -8 if dtype == BF else 2 ** -24
    # the sigmoid's error (fp32: its exponential's two ulp at most, sum and quotient), two products
    rel = ((1.25 * d.neg().clamp(min=0) + 9) if dtype == BF else 6.0) * 2 ** -24 + 3 * 2 ** -24
    # gone below 2^-119 (bf16), or where exp(-z) leaves fp32; the smallest numbers round by half a step
    least = 2.0 ** -119 if dtype == BF else 2.0 ** -120
    want = d * s
    assert bool(((y.double() - want).abs() <= want.abs() * (rel + own * (1 + rel)) + least).all())
    # s + z s (1 - s): in its two terms, the second's factor 1 - s by a step of 1
    size = s + want.abs() * (1 - s) + want.abs() * 2 ** -23
    want = s + want * (1 - s)
    assert bool(((g["dgate"].double() - want).abs() <= size * (3 * rel + 2 ** -22) + want.abs() * own + least).all())
    assert bool((y[d == 0] == 0).all())
