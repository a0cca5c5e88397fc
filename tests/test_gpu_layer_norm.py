"""Layer norm on the GPU against float64: rows and heads, gate, gradients."""
from __future__ import annotations

import pytest
import torch

from tests.linear_cases import norm64
from ssd_chunked_forward_b200 import ssd
from ssd_chunked_forward_b200.autograd import layer_norm_autograd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U32, U16 = 2.0 ** -24, 2.0 ** -8


def make(dtype, rows, width, gate, seed=2, mean=0.5, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return {"x": (rnd(rows, width) * std + mean).to(dtype), "weight": 1 + 0.3 * rnd(width), "bias": 0.2 * rnd(width),
            "gate": rnd(rows, width).to(dtype) if gate else None, "dy": rnd(rows, width).to(dtype)}


def close(name, got, want, size, dtype, steps):
    """size: the magnitudes that were added up; steps: fp32 roundings on the way."""
    b = steps * U32 * size + (U16 * 1.01 * want.abs() + 2.0 ** -18 * size if dtype == BF else 0.0) + 1e-30
    d = (got.double() - want).abs()
    assert bool((d <= b).all()), f"{name}: {float((d / b).max()):.2f} of its bound"


def run(c, dtype, groups, eps=1e-5):
    n = c["x"].shape[-1] // groups
    ref = norm64(c["x"], c["weight"], c["bias"], groups, c["gate"], eps, c["dy"])
    y, stats = ssd.layer_norm(c["x"], c["weight"], c["bias"], groups=groups, gate=c["gate"], eps=eps)
    g = ssd.layer_norm_backward(c["x"], c["weight"], c["bias"], c["dy"], stats, groups=groups, gate=c["gate"])
    part = lambda t: t.reshape(-1, groups, n)  # noqa: E731
    big = part(c["x"].double()).abs().amax(-1)  # the largest number of a part
    rstd = ref["stats"][..., 1]
    # sums over a part are trees of log2 n additions and a few per thread: 40 roundings cover 16384 numbers
    steps = 40.0
    assert bool(((stats[..., 0].double() - ref["stats"][..., 0]).abs() <= steps * U32 * big + 1e-30).all())
    # rstd = (mean (x-m)^2 + eps)^-1/2: relative error of the distances, twice, over two
    rel = steps * U32 * (1 + big * rstd)
    assert bool(((stats[..., 1].double() - rstd).abs() <= rel * rstd).all())
    wide = lambda t: t[..., None].expand(-1, -1, n).reshape(c["x"].shape)  # noqa: E731
    w, b = c["weight"].double().abs(), c["bias"].double().abs()
    xh = (c["x"].double().abs() + wide(big)) * wide(rstd) * wide(1 + big * rstd)
    u = xh * w + b
    z = torch.ones_like(u) if c["gate"] is None else c["gate"].double().abs()
    close("y", y, ref["y"], u * z, dtype, steps)
    d = c["dy"].double().abs()
    if c["gate"] is not None:
        # silu' is at most 1.1; exp of |z| up to 6 in fp32 costs a few roundings more
        close("dgate", g["dgate"], ref["dgate"], 1.1 * d * u, dtype, steps)
    du = d * z
    dxh = part(du * w)
    size = wide(rstd) * (dxh + dxh.mean(-1, keepdim=True) + part(xh) * (dxh * part(xh)).mean(-1, keepdim=True)).reshape(u.shape)
    close("dx", g["dx"], ref["dx"], size, dtype, 3 * steps)
    rows = c["x"].shape[0]
    more = min(rows, 400)  # rows that one thread adds up one after the other, then the blocks' sums
    close("dweight", g["dweight"], ref["dweight"], (du * xh).sum(0), F32, steps + more)
    close("dbias", g["dbias"], ref["dbias"], du.sum(0), F32, steps + more)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gate"])
@pytest.mark.parametrize("rows,width,groups", [
    (1, 1, 1), (1, 64, 1), (5, 64, 1), (37, 256, 4), (9, 300, 3), (300, 5120, 80), (3, 100, 1), (64, 2560, 1),
    (700, 1536, 24), (11, 455, 1), (4, 4096, 1), (5, 8192, 1), (2, 16384, 1), (3, 7777, 1), (2, 16383, 1),
    (33, 520, 13), (2100, 96, 1), (6, 4100, 1), (3, 12000, 1), (1000, 8, 8)])
def test_forward_and_gradients(dtype, gate, rows, width, groups):
    run(make(dtype, rows, width, gate), dtype, groups)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_far_mean_and_constant_rows(dtype):
    """A mean far from zero, and rows without any variance."""
    c = make(dtype, 20, 512, True, mean=300.0, std=1.0)
    c["x"][3:6] = 42.0
    run(c, dtype, 1)


def test_no_weight_no_bias_no_sums():
    c = make(F32, 10, 96, True)
    ref = norm64(c["x"], None, None, 2, c["gate"], 1e-5, c["dy"])
    y, stats = ssd.layer_norm(c["x"], groups=2, gate=c["gate"])
    g = ssd.layer_norm_backward(c["x"], None, None, c["dy"], stats, groups=2, gate=c["gate"], want_dweight=False,
                                want_dbias=False)
    assert g["dweight"] is None and g["dbias"] is None
    for got, want in ((y, ref["y"]), (g["dx"], ref["dx"]), (g["dgate"], ref["dgate"])):
        assert float((got.double() - want).norm() / want.norm()) <= 60 * U32
    one = ssd.layer_norm_backward(c["x"], c["weight"], None, c["dy"], stats, groups=2, want_dbias=False)
    ref = norm64(c["x"], c["weight"], None, 2, None, 1e-5, c["dy"])
    assert one["dbias"] is None and float((one["dweight"].double() - ref["dweight"]).norm() / ref["dweight"].norm()) <= 60 * U32


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("left", [0, 8, 3])
def test_slices(dtype, left):
    """x, gate and dy as slices of wider rows, on and off 16-byte boundaries;
    leading dimensions."""
    c = make(dtype, 12, 128, True)
    y0, s0 = ssd.layer_norm(c["x"], c["weight"], c["bias"], groups=2, gate=c["gate"])
    g0 = ssd.layer_norm_backward(c["x"], c["weight"], c["bias"], c["dy"], s0, groups=2, gate=c["gate"])

    def wide(t):
        b = torch.full((3, 4, left + 128 + 16), float("nan"), dtype=dtype, device="cuda")
        b[..., left:left + 128] = t.view(3, 4, 128)
        return b[..., left:left + 128]

    x, z, dy = wide(c["x"]), wide(c["gate"]), wide(c["dy"])
    y, s = ssd.layer_norm(x, c["weight"], c["bias"], groups=2, gate=z)
    g = ssd.layer_norm_backward(x, c["weight"], c["bias"], dy, s, groups=2, gate=z)
    # another vector width adds in another order
    tol = (2 * U16 if dtype == BF else 60 * U32)
    for a, b in ((y, y0), (g["dx"], g0["dx"]), (g["dgate"], g0["dgate"])):
        assert a.shape == (3, 4, 128)
        assert float((a.double().view(12, 128) - b.double()).norm() / b.double().norm()) <= tol
    assert float((g["dweight"] - g0["dweight"]).norm() / g0["dweight"].norm()) <= 60 * U32


def test_same_result_every_time_and_in_a_graph():
    c = make(BF, 3000, 768, True)
    call = lambda: ssd.layer_norm_backward(  # noqa: E731
        c["x"], c["weight"], c["bias"], c["dy"],
        ssd.layer_norm(c["x"], c["weight"], c["bias"], groups=12, gate=c["gate"])[1], groups=12, gate=c["gate"])
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n], held[n]) and torch.equal(want[n], other[n])


def test_autograd_and_differences():
    c = make(F32, 6, 80, True)
    leaves = [c[n].clone().requires_grad_() for n in ("x", "weight", "bias", "gate")]
    y = layer_norm_autograd(leaves[0], leaves[1], leaves[2], groups=5, gate=leaves[3])
    got = torch.autograd.grad(y, leaves, c["dy"].t().contiguous().t())
    ref = norm64(c["x"], c["weight"], c["bias"], 5, c["gate"], 1e-5, c["dy"])
    for a, n in zip(got, ("dx", "dweight", "dbias", "dgate")):
        assert float((a.double() - ref[n]).norm() / ref[n].norm()) <= 100 * U32
    g = torch.Generator(device="cuda").manual_seed(9)
    d = [torch.randn(t.shape, generator=g, device="cuda").double() for t in leaves]
    f = lambda s: (norm64(*(t.detach().double() + s * u for t, u in zip(leaves[:3], d)), 5,  # noqa: E731
                          leaves[3].detach().double() + s * d[3], 1e-5)["y"] * c["dy"]).sum()
    slope = float((f(1e-5) - f(-1e-5)) / 2e-5)
    along = float(sum((a.double() * u).sum() for a, u in zip(got, d)))
    assert abs(slope - along) <= 1e-5 * sum(float(a.double().norm() * u.norm()) for a, u in zip(got, d))


@pytest.mark.parametrize("dtype,rows,width,groups,gate", [(BF, 32768, 5120, 80, True), (BF, 50000, 640, 1, False),
                                                          (F32, 9000, 2048, 16, True), (BF, 70001, 24, 1, True)])
def test_rows_do_not_know_of_each_other(dtype, rows, width, groups, gate):
    """Many rows (blocks take several turns, threads many rows): each row's results are
    to the bit those of a call with a few of them, whatever the others hold."""
    c = make(dtype, rows, width, gate)
    c["x"][7::1000] = float("nan")
    c["dy"][11::1000] = float("inf")
    y, stats = ssd.layer_norm(c["x"], c["weight"], c["bias"], groups=groups, gate=c["gate"])
    g = ssd.layer_norm_backward(c["x"], c["weight"], c["bias"], c["dy"], stats, groups=groups, gate=c["gate"])
    for a in (0, 1, rows // 2, rows - 5):
        s = slice(a, a + 5)
        part = {n: None if c[n] is None else c[n][s] for n in ("x", "gate", "dy")}
        y2, stats2 = ssd.layer_norm(part["x"], c["weight"], c["bias"], groups=groups, gate=part["gate"])
        g2 = ssd.layer_norm_backward(part["x"], c["weight"], c["bias"], part["dy"], stats2, groups=groups,
                                     gate=part["gate"])
        same = lambda p, q: torch.equal(torch.nan_to_num(p), torch.nan_to_num(q))  # noqa: E731
        assert same(y[s], y2) and same(stats[s], stats2) and same(g["dx"][s], g2["dx"])
        assert gate is False or same(g["dgate"][s], g2["dgate"])
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[7::1000] = False
    assert bool(torch.isfinite(y[fine]).all())


def test_refusals_on_the_gpu():
    """Wrong types, shapes, devices and layouts are errors of the call."""
    c = make(BF, 12, 64, True)
    x, w, b, z = c["x"], c["weight"], c["bias"], c["gate"]
    ok, stats = ssd.layer_norm(x, w, b, groups=2, gate=z)
    for bad in [dict(x=x.half()), dict(weight=w.double()), dict(weight=w[:32]), dict(bias=b.cpu()), dict(gate=z.float()),
                dict(gate=z[:6]), dict(groups=5), dict(groups=0), dict(x=x.t()), dict(x=x[:0], gate=z[:0]),
                dict(y=ok.float()), dict(y=ok[:6]), dict(eps=float("nan")), dict(eps=-1.0)]:
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.layer_norm(**{**dict(x=x, weight=w, bias=b, groups=2, gate=z), **bad})
    for bad in [dict(dy=c["dy"].float()), dict(stats=stats[:6]), dict(stats=stats.double()), dict(dy=c["dy"].cpu())]:
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.layer_norm_backward(**{**dict(x=x, weight=w, bias=b, dy=c["dy"], stats=stats, groups=2, gate=z), **bad})
    torch.cuda.synchronize()
    assert torch.equal(ssd.layer_norm(x, w, b, groups=2, gate=z)[0], ok)


def test_squares_that_overflow():
    """Numbers whose squares leave fp32: rstd is 0, as the formula in fp32 has it, not NaN."""
    x = torch.randn(3, 256, device="cuda") * 1e25
    y, stats = ssd.layer_norm(x, None, None)
    assert bool((stats[..., 1] == 0).all()) and bool((y == 0).all())


@pytest.mark.parametrize("dtype,rows,width,groups", [(BF, 5000, 2560, 1), (BF, 3000, 1536, 24), (F32, 700, 455, 1),
                                                     (BF, 900, 455, 1)])
def test_in_place(dtype, rows, width, groups):
    """y may be x itself, or the gate."""
    c = make(dtype, rows, width, True)
    want, stats = ssd.layer_norm(c["x"], c["weight"], c["bias"], groups=groups, gate=c["gate"])
    for n in ("x", "gate"):
        t = {m: c[m].clone() for m in ("x", "gate")}
        y, s2 = ssd.layer_norm(t["x"], c["weight"], c["bias"], groups=groups, gate=t["gate"], y=t[n])
        assert y is t[n] and torch.equal(y, want) and torch.equal(s2, stats)


def test_two_streams_at_once():
    """Calls side by side on two streams, gradients among them."""
    c = make(BF, 6000, 1536, True)
    want, stats = ssd.layer_norm(c["x"], c["weight"], c["bias"], groups=24, gate=c["gate"])
    back = lambda s: ssd.layer_norm_backward(c["x"], c["weight"], c["bias"], c["dy"], stats, groups=24,  # noqa: E731
                                             gate=c["gate"], stream=s)
    g = back(None)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(10):
        with torch.cuda.stream(streams[i % 2]):
            got.append(back(None))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(r[n], g[n]) for n in g)
