"""The split of a weighted token into bf16 pieces, as the tensor-core scan makes it,
on the CPU: what the bound of the states' test tells apart."""
import torch


def test_one_piece_less_would_show():
    """The split of the weighted token on the CPU: three pieces hold the fp32 product, two
    leave more than tests/test_gpu_linear_long.py allows."""
    w = torch.exp(-0.03 * torch.arange(1, 300, dtype=torch.float64)).float()
    x = (w[:, None] * torch.randn(64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).float())
    for pieces, fits in ((3, True), (2, False)):
        rest, total = x.clone(), torch.zeros_like(x, dtype=torch.float64)
        for _ in range(pieces - 1):
            top = (rest.view(torch.int32) & -65536).view(torch.float32)
            total, rest = total + top, rest - top
        total += rest.to(torch.bfloat16)
        off = ((total - x.double()).abs() / x.double().abs()).max()
        assert (off == 0) if fits else (18 * 2 ** -24 < off <= 2 ** -16)
