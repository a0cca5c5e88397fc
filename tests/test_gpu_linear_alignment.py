"""States and gradients as slices of pools, which start off 16-byte boundaries when a
state has an odd number of elements: read ones are taken, written ones are
refused by name."""
from __future__ import annotations

import pytest
import torch

from ssd_chunked_forward_b200 import ssd
from tests.linear_cases import slopes

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def off(t):
    """t behind one element: contiguous, off a 16-byte boundary."""
    s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    assert s.data_ptr() % 16 and s.is_contiguous()
    return s


@pytest.mark.parametrize("dtype,K,V", [(BF, 64, 64), (F32, 5, 3)])
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
def test_read_from_anywhere(dtype, K, V, packed):
    B, T, H = 2, 300, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v, dy = rnd(B, T, H, K), rnd(B, T, H, K), rnd(B, T, H, V), rnd(B, T, H, V)
    init, dfinal, decay, cu = rnd(B, H, K, V, dt=F32), rnd(B, H, K, V, dt=F32), slopes(H), None
    if packed:
        q, k, v, dy = (t.flatten(0, 1) for t in (q, k, v, dy))
        cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")

    def run(move):
        y, final = ssd.linear_attention(q, k, v, decay, initial_state=move(init), cu_seqlens=cu)
        return {"y": y, "final": final, **ssd.linear_attention_backward(
            q, k, v, decay, move(dy), initial_state=move(init), dfinal=move(dfinal), cu_seqlens=cu)}

    a, b = run(lambda t: t), run(off)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_written_ones_are_refused_by_name():
    q, decay = torch.randn(2, 40, 2, 64, device="cuda", dtype=BF), slopes(2)
    y, state = ssd.linear_attention(q, q, q, decay)  # (a row of y is x below)
    for name, call in {
            "y": lambda: ssd.linear_attention(q, q, q, decay, y=off(y)),
            "final_state": lambda: ssd.linear_attention(q, q, q, decay, final_state=off(state)),
            "state": lambda: ssd.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], decay, off(state)),
            "workspace": lambda: ssd.linear_attention(q, q, q, decay, workspace=torch.empty(
                1 << 20, dtype=torch.uint8, device="cuda")[16:]),
            "stats": lambda: ssd.layer_norm_backward(y[0, :, 0], None, None, y[0, :, 0], off(torch.zeros(40, 1, 2, device="cuda"))),
    }.items():
        with pytest.raises(ValueError, match=f"^{name} must start"):
            call()
