"""Child of tests/test_gpu_linear_debug.py: with the index-checked build
(SSD_DEBUG_CHECKS=1) runs linear attention and layer norm on small in-bounds
cases; prints one JSON line with the largest error in units of its bound and
the record of failed checks."""
from __future__ import annotations

import json
import os

import torch

from tests.linear_cases import bounds, norm64, on_tensor_cores, reference, slopes
from ssd_chunked_forward_b200 import ssd


def main():
    assert os.environ.get("SSD_DEBUG_CHECKS") == "1"
    ssd.debug_record()
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    worst = {}
    cuts, total, H, G = [3, 3, 140, 1700], 1711, 4, 2
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    for dtype, K, V in ((torch.bfloat16, 128, 64), (torch.bfloat16, 64, 128), (torch.bfloat16, 128, 128),
                        (torch.bfloat16, 48, 56), (torch.float32, 33, 70)):
        q, k, v, dy = (rnd(total, h, d).to(dtype) for h, d in ((H, K), (G, K), (G, V), (H, V)))
        v[cuts[-1] - 3:cuts[-1]] = float("inf")  # mended rows
        init, dfinal, decay = rnd(3, H, K, V), rnd(3, H, K, V), slopes(H)
        args = (q, k, v, decay, K ** -0.5, init, cuts, dy, dfinal)
        ref, size = reference(*args), reference(*args, magnitude=True)
        y, final = ssd.linear_attention(q, k, v, decay, initial_state=init, cu_seqlens=cu)
        got = {"y": y, "final": final, **ssd.linear_attention_backward(q, k, v, decay, dy, initial_state=init,
                                                                       dfinal=dfinal, cu_seqlens=cu)}
        ssd.linear_attention(q[None], k[None], v[None], decay)
        ssd.linear_attention_step(q[:5], k[:5], v[:5], decay, rnd(5, H, K, V))
        for n, t in got.items():
            b = bounds(ref, size, n, dtype, K, V, 1560, on_tensor_cores(dtype, K, V))
            live = torch.isfinite(ref[n])
            worst[f"{n} {K} {V}"] = float(((t.double() - ref[n]).abs() / b)[live].max())
    for dtype, width, groups in ((torch.bfloat16, 512, 8), (torch.bfloat16, 2570, 1), (torch.float32, 455, 1)):
        x, z, dy = (rnd(37, width).to(dtype) for _ in range(3))
        w, b = rnd(width), rnd(width)
        y, stats = ssd.layer_norm(x, w, b, groups=groups, gate=z)
        out = ssd.layer_norm_backward(x, w, b, dy, stats, groups=groups, gate=z)
        ref = norm64(x, w, b, groups, z, 1e-5, dy)
        worst[f"norm {width}"] = float((y.double() - ref["y"]).abs().max() / ref["y"].abs().max())
        worst[f"norm dw {width}"] = float((out["dweight"].double() - ref["dweight"]).abs().max() /
                                          ref["dweight"].abs().max())
    torch.cuda.synchronize()
    print(json.dumps({"worst": worst, "record": list(ssd.debug_record())}))


if __name__ == "__main__":
    main()
