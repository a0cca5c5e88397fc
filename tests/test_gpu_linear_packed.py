"""Packed rows of very many sequences, some of them long enough to be cut."""
from __future__ import annotations

import pytest
import torch

from ssd_chunked_forward_b200 import ssd
from tests.linear_cases import slopes
from tests.test_gpu_linear import both, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 128, 128), (F32, 24, 16)])
def test_long_ones_among_many(dtype, K, V):
    """1200 sequences of none to eight tokens with three of thousands between them, rows
    of no sequence in front: forward, gradients, states in and out."""
    cuts = [11]
    for i in range(1200):
        cuts.append(cuts[-1] + (i * 5) % 9)
        if i in (0, 33, 1100):
            cuts.append(cuts[-1] + 1500 + 700 * (i % 3))
    both(make(dtype, cuts, cuts[-1] + 5, 2, 1, K, V, outside=float("nan")), cuts, dtype)


@pytest.mark.parametrize("dtype,K,V", [(BF, 64, 64), (F32, 16, 16)])
def test_offsets_that_are_none_stay_inside(dtype, K, V):
    """Many offsets that decrease, are negative or too large: nothing outside the rows
    and the workspace is written."""
    T, H = 3000, 2
    c = make(dtype, [0, T], T, H, H, K, V, init=False)
    g = torch.Generator().manual_seed(1)
    for n in (2, 40, 900):
        cu = torch.randint(-T, 2 * T, (n + 1,), generator=g, dtype=torch.int32).cuda()
        code = ssd.SSD_DTYPE_BF16 if dtype == BF else ssd.SSD_DTYPE_F32
        need = ssd.linear_workspace_size(ssd.LinearShape(n, T, H, H, K, V, code, 1))
        ws = torch.full((need + 4096,), 5, dtype=torch.uint8, device="cuda")
        guard = torch.full((T + 256, H, V), 3.0, dtype=dtype, device="cuda")
        ssd.linear_attention(c["q"], c["k"], c["v"], c["decay"], cu_seqlens=cu, y=guard[128:128 + T], workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((guard[:128] == 3.0).all()) and bool((guard[128 + T:] == 3.0).all()) and bool((ws[need:] == 5).all())


def test_workspace_of_a_thousand_sequences():
    """1000 sequences in 100000 rows of 32 heads: in 54 MB."""
    shape = ssd.LinearShape(1000, 100000, 32, 32, 128, 128, ssd.SSD_DTYPE_BF16, 1)
    need = ssd.linear_workspace_size(shape)
    assert need < 100 << 20
    q = torch.randn(100000, 32, 128, device="cuda", dtype=BF)
    cu = torch.arange(0, 100001, 100, device="cuda", dtype=torch.int32)
    y, final = ssd.linear_attention(q, q, q, slopes(32), cu_seqlens=cu,
                                    workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    one = ssd.linear_attention(q[:100][None], q[:100][None], q[:100][None], slopes(32))
    assert torch.equal(y[:100], one[0][0]) and torch.equal(final[:1], one[1])
