"""Linear attention with a decay for each head on the GPU, against the
recurrence in 64 bits: prompts, gradients, single tokens, and their runs
together."""
from __future__ import annotations

import pytest
import torch

from tests.linear_cases import bounds, heads64, on_tensor_cores, reference, slopes
from ssd_chunked_forward_b200 import ssd
from ssd_chunked_forward_b200.autograd import layer_norm_autograd, linear_attention_autograd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(dtype, cuts, total, H, G, K, V, seed=1, init=True, fused=False, outside=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    S = len(cuts) - 1
    if fused:
        q, k, v = rnd(total, H * K + G * (K + V)).split([H * K, G * K, G * V], -1)
        q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V))
    else:
        q, k, v = rnd(total, H, K), rnd(total, G, K), rnd(total, G, V)
    out = {"q": q, "k": k, "v": v, "dy": rnd(total, H, V), "decay": slopes(H),
           "init": rnd(S, H, K, V, dt=F32) if init else None, "dfinal": rnd(S, H, K, V, dt=F32) if init else None}
    if outside is not None:  # rows of no sequence
        dead = torch.ones(total, dtype=torch.bool, device="cuda")
        for a, b in zip(cuts, cuts[1:]):
            dead[a:b] = False
        for n in ("q", "k", "v", "dy"):
            out[n][dead] = outside
    return out


def check(got, ref, size, dtype, K, V, longest, tc):
    for name, t in got.items():
        if t is None:
            continue
        live = ~torch.isnan(ref[name])
        d = (t.double() - ref[name]).abs()
        b = bounds(ref, size, name, dtype, K, V, longest, tc)
        bad = (d > b) | torch.isnan(d)
        assert not bool((bad & live).any()), f"{name}: {int((bad & live).sum())} of {live.sum()} off, worst {float((d / b)[live].max()):.2f} of its bound"


def both(c, cuts, dtype, scale=None, tc=None):
    """Runs the forward and the backward as packed rows and checks every output."""
    K, V = c["q"].shape[-1], c["v"].shape[-1]
    longest = max(b - a for a, b in zip(cuts, cuts[1:]))
    tc = on_tensor_cores(dtype, K, V) if tc is None else tc
    sc = K ** -0.5 if scale is None else scale
    args = (c["q"], c["k"], c["v"], c["decay"], sc, c["init"], cuts, c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    y, final = ssd.linear_attention(c["q"], c["k"], c["v"], c["decay"], scale=scale, initial_state=c["init"],
                                    cu_seqlens=cu)
    g = ssd.linear_attention_backward(c["q"], c["k"], c["v"], c["decay"], c["dy"], scale=scale,
                                      initial_state=c["init"], dfinal=c["dfinal"], cu_seqlens=cu)
    check({"y": y, "final": final, **g}, ref, size, dtype, K, V, longest, tc)
    return y, final, g


DIMS = [(64, 64), (128, 64), (64, 128), (128, 128), (96, 80), (16, 48), (8, 8), (100, 36), (1, 1), (33, 7)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("K,V", DIMS)
@pytest.mark.parametrize("T", [1, 2, 33, 128, 129, 300])
def test_rows_of_one_length(dtype, K, V, T):
    """[B,T] rows: forward and gradients, shared heads, states in and out."""
    B, H, G = 2, 4, 2
    c = make(dtype, [0, T, 2 * T], B * T, H, G, K, V)
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, c["init"], [0, T, 2 * T], c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    r = lambda t: t.view(B, T, *t.shape[1:])  # noqa: E731
    y, final = ssd.linear_attention(r(c["q"]), r(c["k"]), r(c["v"]), c["decay"], initial_state=c["init"])
    g = ssd.linear_attention_backward(r(c["q"]), r(c["k"]), r(c["v"]), c["decay"], r(c["dy"]),
                                      initial_state=c["init"], dfinal=c["dfinal"])
    got = {n: t.flatten(0, 1) if n not in ("final", "dinit") else t for n, t in {"y": y, "final": final, **g}.items()}
    check(got, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))


@pytest.mark.parametrize("K,V", [(256, 256), (200, 136), (128, 256)])
def test_wide_heads(K, V):
    for dtype in (F32, BF):
        both(make(dtype, [0, 150], 150, 2, 1, K, V), [0, 150], dtype)


PACKED = [[0, 5], [0, 0, 7, 7, 135, 300, 300], [0, 128, 256, 257, 700], [3, 60, 260]]


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 128), (BF, 128, 64), (BF, 64, 64), (BF, 40, 112), (F32, 48, 64)])
@pytest.mark.parametrize("cuts", PACKED, ids=str)
def test_packed(dtype, K, V, cuts):
    """Empty sequences, one token, ends inside a chunk; rows behind and before
    the sequences hold NaN: they are not read, and a given y keeps its own."""
    total = cuts[-1] + 37
    c = make(dtype, cuts, total, 4, 4, K, V, outside=float("nan"), fused=True)
    both(c, cuts, dtype)
    y = torch.full((total, 4, V), 7.0, dtype=dtype, device="cuda")
    ssd.linear_attention(c["q"], c["k"], c["v"], c["decay"], y=y, want_final=False,
                         cu_seqlens=torch.tensor(cuts, dtype=torch.int32, device="cuda"))
    assert bool((y[cuts[-1]:] == 7.0).all()) and bool((y[:cuts[0]] == 7.0).all())
    assert bool(torch.isfinite(y[cuts[0]:cuts[-1]]).all())


@pytest.mark.parametrize("dtype,K,V,T", [(BF, 128, 64, 3000), (BF, 128, 128, 2049), (BF, 64, 64, 5000),
                                         (BF, 64, 128, 2500), (F32, 64, 32, 2000)])
def test_long_cut_chains(dtype, K, V, T):
    """Few chains: every chain is cut into items and its states combined; rows
    of one length and packed ones give the same sums in other orders."""
    c = make(dtype, [0, T], T, 2, 1, K, V)
    y, final, g = both(c, [0, T], dtype)
    e = lambda t: t[None]  # noqa: E731
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, c["init"], [0, T], c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    y2, f2 = ssd.linear_attention(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], initial_state=c["init"])
    g2 = ssd.linear_attention_backward(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], e(c["dy"]),
                                       initial_state=c["init"], dfinal=c["dfinal"])
    got = {"y": y2[0], "final": f2, "dq": g2["dq"][0], "dk": g2["dk"][0], "dv": g2["dv"][0], "dinit": g2["dinit"]}
    check(got, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 64, 128), (F32, 20, 24)])
def test_some_chains_cut(dtype, K, V):
    """More chains than run at a time: whole ones, then cut ones."""
    B, T, H = 3, 1100, 52
    c = make(dtype, [0, T, 2 * T, 3 * T], B * T, H, H, K, V, init=False)
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, None, [0, T, 2 * T, 3 * T])
    ref, size = reference(*args), reference(*args, magnitude=True)
    r = lambda t: t.view(B, T, *t.shape[1:])  # noqa: E731
    y, final = ssd.linear_attention(r(c["q"]), r(c["k"]), r(c["v"]), c["decay"])
    check({"y": y.flatten(0, 1), "final": final}, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decays_at_the_ends(dtype):
    """No decay, decays that leave one token, and a head that keeps nothing."""
    c = make(dtype, [0, 290], 290, 4, 4, 64, 64)
    c["decay"] = torch.tensor([0.0, -3.0, -90.0, float("-inf")], device="cuda")
    both(c, [0, 290], dtype)


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 72, 40), (F32, 64, 64), (BF, 50, 30)])
def test_strides(dtype, K, V):
    """Batch of slices of one projection, heads before tokens, a broadcast batch,
    and rows that start off a 16-byte boundary."""
    B, T, H, G = 2, 200, 4, 2
    cuts = [0, T, 2 * T]
    c = make(dtype, cuts, B * T, H, G, K, V)
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, c["init"], cuts, c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    rows = {n: c[n].view(B, T, *c[n].shape[1:]) for n in ("q", "k", "v", "dy")}

    def wide(t, left):  # a slice of a wider projection
        b = torch.full(t.shape[:2] + (left + t.shape[2] * t.shape[3] + 24,), float("nan"), dtype=dtype, device="cuda")
        s = b[..., left:left + t.shape[2] * t.shape[3]].unflatten(-1, t.shape[2:])
        s.copy_(t)
        return s

    forms = {"slices": lambda t: wide(t, 8), "odd start": lambda t: wide(t, 3),
             "heads first": lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)}
    for name, form in forms.items():
        q, k, v = (form(rows[n]) for n in "qkv")
        y, final = ssd.linear_attention(q, k, v, c["decay"], initial_state=c["init"])
        g = ssd.linear_attention_backward(q, k, v, c["decay"], rows["dy"], initial_state=c["init"], dfinal=c["dfinal"])
        got = {n: t.flatten(0, 1) if n not in ("final", "dinit") else t for n, t in {"y": y, "final": final, **g}.items()}
        check(got, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))
    one = rows["k"][:1].expand(B, -1, -1, -1)
    y, _ = ssd.linear_attention(rows["q"], one, rows["v"], c["decay"])
    y2, _ = ssd.linear_attention(rows["q"], one.contiguous(), rows["v"], c["decay"])
    longest = (y.double() - y2.double()).abs().max()
    assert longest <= 4 * 2 ** -8 * y2.double().abs().max()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,K,V", [(1, 1, 1, 1, 1), (3, 4, 2, 128, 64), (2, 6, 1, 64, 128), (5, 2, 2, 128, 128),
                                       (2, 2, 2, 256, 256), (2, 4, 4, 100, 36), (3, 2, 1, 33, 7), (1, 2, 2, 17, 130)])
def test_step(dtype, B, H, G, K, V):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k, v = rnd(B, H * K + G * (K + V) + 5).to(dtype)[:, 5:].split([H * K, G * K, G * V], -1)
    q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V))
    state, decay = rnd(B, H, K, V), slopes(H)
    lam = torch.exp(decay.double())[:, None, None]
    kv = heads64(k, H)[..., None] * heads64(v, H)[..., None, :]
    h = lam * state.double() + kv
    y = 0.7 * torch.einsum("bhk,bhkv->bhv", q.double(), h)
    size_h = lam * state.double().abs() + kv.abs()
    size = 0.7 * torch.einsum("bhk,bhkv->bhv", q.double().abs(), size_h)
    got = ssd.linear_attention_step(q, k, v, decay, state, scale=0.7)
    # state: product, factor and sum round once each; y: K additions more
    assert bool(((state.double() - h).abs() <= 4 * 2 ** -24 * size_h).all())
    b = size * (K + 8) * 2 ** -24 + (2 ** -8 * 1.01 * y.abs() + size * 2 ** -20 if dtype == BF else 0.0)
    assert bool(((got.double() - y).abs() <= b).all())


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (F32, 64, 64), (BF, 128, 128)])
def test_prompt_then_tokens(dtype, K, V):
    """A prompt in two calls and single tokens behind it are one sequence."""
    T, n1, n2, B, H = 210, 130, 70, 2, 4
    c = make(dtype, [0, T, 2 * T], B * T, H, 2, K, V, init=False)
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, None, [0, T, 2 * T])
    ref, size = reference(*args), reference(*args, magnitude=True)
    q, k, v = (c[n].view(B, T, *c[n].shape[1:]) for n in "qkv")
    y1, state = ssd.linear_attention(q[:, :n1], k[:, :n1], v[:, :n1], c["decay"])
    # the state updated in place: final_state is initial_state
    y2, state2 = ssd.linear_attention(q[:, n1:n1 + n2], k[:, n1:n1 + n2], v[:, n1:n1 + n2], c["decay"],
                                      initial_state=state, final_state=state)
    assert state2 is state
    ys = [y1, y2]
    for t in range(n1 + n2, T):
        ys.append(ssd.linear_attention_step(q[:, t], k[:, t], v[:, t], c["decay"], state)[:, None])
    y = torch.cat(ys, 1).flatten(0, 1)
    check({"y": y, "final": state}, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))


def test_streams_and_graphs():
    """On another stream, and captured into a graph that replays with new inputs
    (cut chains, so several kernels and the workspace are in it)."""
    T = 2300
    c = make(BF, [0, T], T, 2, 2, 128, 64)
    e = lambda t: t[None]  # noqa: E731
    call = lambda: (ssd.linear_attention(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], initial_state=c["init"]),  # noqa: E731
                    ssd.linear_attention_backward(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], e(c["dy"]),
                                                  initial_state=c["init"], dfinal=c["dfinal"]))
    flat = lambda r: list(r[0]) + [r[1][n] for n in sorted(r[1])]  # noqa: E731
    want = flat(call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = flat(call())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = flat(call())
    graph.replay()
    for a, b, d in zip(want, other, held):
        assert torch.equal(a, b) and torch.equal(a, d)
    c["q"].mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], -want[0])
    # two streams at once, a workspace each
    ws = [torch.empty(ssd.linear_workspace_size(ssd.LinearShape(1, T, 2, 2, 128, 64, ssd.SSD_DTYPE_BF16, 0)),
                      dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = []
    torch.cuda.synchronize()
    for w in ws:
        s = torch.cuda.Stream()
        ys.append(ssd.linear_attention(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], initial_state=c["init"],
                                       workspace=w, stream=s)[0])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], held[0]) and torch.equal(ys[1], held[0])
    assert ssd.device_status(ws[0]) == ssd.SSD_OK


def test_autograd_block():
    """A block as a model has it: projection, linear attention, norm over the
    heads with a gate; gradients against float64 autograd and differences."""
    B, T, H, G, D, W = 2, 70, 4, 2, 32, 48
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = rnd(B, T, W), (rnd(W, H * D + 2 * G * D + H * D) / W ** 0.5).requires_grad_()
    nw, nb = (1 + 0.1 * rnd(H * D)).requires_grad_(), (0.1 * rnd(H * D)).requires_grad_()
    h0 = rnd(B, H, D, D).requires_grad_()
    decay, out = slopes(H), rnd(B, T, H * D)

    def block(w, nw, nb, h0, lib):
        q, k, v, z = (x.to(w.dtype) @ w).split([H * D, G * D, G * D, H * D], -1)
        q, k, v = q.unflatten(-1, (H, D)), k.unflatten(-1, (G, D)), v.unflatten(-1, (G, D))
        if lib:
            y, fin = linear_attention_autograd(q, k, v, decay, initial_state=h0)
            y = layer_norm_autograd(y.flatten(2), nw, nb, groups=H, gate=z)
        else:
            k, v = k.repeat_interleave(H // G, 2), v.repeat_interleave(H // G, 2)
            h, ys = h0, []
            for t in range(T):
                h = torch.exp(decay.double())[:, None, None] * h + k[:, t, :, :, None] * v[:, t, :, None]
                ys.append(D ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], h))
            y, fin = torch.stack(ys, 1), h
            y = (y - y.mean(-1, keepdim=True)) / torch.sqrt(y.var(-1, unbiased=False, keepdim=True) + 1e-5)
            y = (y.flatten(2) * nw + nb) * z * torch.sigmoid(z)
        return (y * out.to(y.dtype)).sum() + (fin * 0.1).sum()

    loss = block(w, nw, nb, h0, True)
    got = torch.autograd.grad(loss, [w, nw, nb, h0])
    leaves = [t.detach().double().requires_grad_() for t in (w, nw, nb, h0)]
    ref_loss = block(*leaves, False)
    want = torch.autograd.grad(ref_loss, leaves)
    # products over W, K, T and rows in fp32: some hundred roundings, the norm's
    # division amplifies by rstd at most tenfold here
    for a, b in zip(got, want):
        assert float((a.double() - b).norm() / b.norm()) <= 4000 * 2 ** -24
    # differences, in float64 on the definition and once through the kernels
    d = [torch.randn_like(t) for t in leaves]
    eps = 1e-5
    hi = block(*[t + eps * u for t, u in zip(leaves, d)], False)
    lo = block(*[t - eps * u for t, u in zip(leaves, d)], False)
    slope = float((hi - lo) / (2 * eps))
    along = float(sum((a.double() * u).sum() for a, u in zip(got, d)))
    assert abs(slope - along) <= 1e-4 * sum(float(a.double().norm() * u.norm()) for a, u in zip(got, d))


def test_backward_captured_while_an_eager_graph_lives():
    """Gradients by the explicit call inside a capture, with an autograd graph of
    the same tensors alive."""
    c = make(BF, [0, 100], 100, 2, 2, 64, 64)
    q = c["q"][None].detach().requires_grad_()
    y, _ = linear_attention_autograd(q, c["k"][None], c["v"][None], c["decay"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ssd.linear_attention_backward(q.detach(), c["k"][None], c["v"][None], c["decay"], c["dy"][None])
    graph.replay()
    (eager,) = torch.autograd.grad(y, q, c["dy"][None])
    assert torch.equal(eager, g["dq"])


def test_offsets_that_are_none_stay_inside():
    """Decreasing, negative and too large offsets: clamped, nothing outside the
    rows is written."""
    T = 700
    c = make(BF, [0, T], T, 2, 2, 64, 64, init=False)
    for cuts in ([0, 600, 100, 700], [-50, 300, 5000], [700, 0, 700]):
        cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        guard = torch.full((T + 256, 2, 64), 3.0, dtype=BF, device="cuda")
        y, _ = ssd.linear_attention(c["q"], c["k"], c["v"], c["decay"], cu_seqlens=cu, y=guard[128:128 + T])
        torch.cuda.synchronize()
        assert bool((guard[:128] == 3.0).all()) and bool((guard[128 + T:] == 3.0).all())


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 64, 64), (F32, 30, 24)])
def test_packed_shared_heads(dtype, K, V):
    """Keys and values shared by the heads of a group, rows of no sequence before
    and behind, a workspace that held something else: the gradients of those rows are
    zero, and nothing of the workspace reaches any."""
    cuts, total, H, G = [5, 140, 140, 900], 960, 6, 2
    c = make(dtype, cuts, total, H, G, K, V, outside=float("nan"))
    both(c, cuts, dtype)
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    code = ssd.SSD_DTYPE_BF16 if dtype == BF else ssd.SSD_DTYPE_F32
    need = ssd.linear_backward_workspace_size(ssd.LinearShape(3, total, H, G, K, V, code, 1))
    call = lambda fill: ssd.linear_attention_backward(  # noqa: E731
        c["q"], c["k"], c["v"], c["decay"], c["dy"], initial_state=c["init"], dfinal=c["dfinal"], cu_seqlens=cu,
        workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
    a, b = call(0xFF), call(0)
    for n in a:
        assert torch.equal(a[n], b[n]), n
        if n != "dinit":
            assert bool((a[n][:5] == 0).all()) and bool((a[n][900:] == 0).all()) and bool(torch.isfinite(a[n]).all())


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 64, 128), (BF, 128, 128), (BF, 64, 64), (F32, 16, 16)])
def test_many_chains(dtype, K, V):
    """More chains than the GPU runs at a time, several chunks each, uncut in both
    directions; gradients of all of them."""
    B, T, H = 2, 515, 160
    cuts = [0, T, 2 * T]
    c = make(dtype, cuts, B * T, H, H, K, V)
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, c["init"], cuts, c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    r = {n: c[n].view(B, T, *c[n].shape[1:]) for n in ("q", "k", "v", "dy")}
    y, final = ssd.linear_attention(r["q"], r["k"], r["v"], c["decay"], initial_state=c["init"])
    g = ssd.linear_attention_backward(r["q"], r["k"], r["v"], c["decay"], r["dy"], initial_state=c["init"],
                                      dfinal=c["dfinal"])
    got = {n: t if n in ("final", "dinit") else t.flatten(0, 1) for n, t in {"y": y, "final": final, **g}.items()}
    check(got, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))


@pytest.mark.parametrize("dtype,K,V", [(BF, 64, 64), (BF, 128, 128), (F32, 24, 16)])
def test_many_short_sequences(dtype, K, V):
    """Hundreds of sequences of none to nine tokens."""
    cuts = [0]
    for i in range(300):
        cuts.append(cuts[-1] + (i * 7) % 10)
    c = make(dtype, cuts, cuts[-1], 2, 1, K, V)
    both(c, cuts, dtype)


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 64, 128), (BF, 128, 128), (BF, 64, 64), (F32, 64, 64)])
def test_a_spoiled_sequence_stays_alone(dtype, K, V):
    """NaN and infinities in one sequence, its ends inside the neighbours' chunks:
    the others' results are to the bit what they are without."""
    cuts = [0, 70, 150, 333]
    c = make(dtype, cuts, 333, 4, 2, K, V)
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")

    def run():
        y, f = ssd.linear_attention(c["q"], c["k"], c["v"], c["decay"], initial_state=c["init"], cu_seqlens=cu)
        g = ssd.linear_attention_backward(c["q"], c["k"], c["v"], c["decay"], c["dy"], initial_state=c["init"],
                                          dfinal=c["dfinal"], cu_seqlens=cu)
        return {"y": y, "final": f, **g}

    want = run()
    for n in ("q", "k", "v", "dy"):
        c[n][70:110] = float("nan")
        c[n][110:150] = float("inf")
    got = run()
    for n, t in got.items():
        for keep in ([slice(0, 1), slice(2, 3)] if n in ("final", "dinit") else [slice(0, 70), slice(150, 333)]):
            assert torch.equal(t[keep], want[n][keep]), n


def test_refusals_on_the_gpu():
    """Wrong types, shapes, devices and layouts are errors of the call."""
    c = make(BF, [0, 40], 40, 4, 2, 64, 64)
    q, k, v, decay = c["q"][None], c["k"][None], c["v"][None], c["decay"]
    ok = ssd.linear_attention(q, k, v, decay)[0]
    for bad in [dict(q=q.half()), dict(k=k.float()), dict(v=v[:, :30]), dict(k=k[:, :, :1].expand(1, 40, 3, 64)),
                dict(decay=decay.double()), dict(decay=decay[:3]), dict(decay=decay.cpu()), dict(q=q[..., :40]),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(initial_state=c["init"].half()),
                dict(initial_state=c["init"][:, :2]), dict(y=torch.empty_like(ok).transpose(1, 2)),
                dict(y=ok.float()), dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda")),
                dict(cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(scale=float("nan")), dict(q=q[:, :0], k=k[:, :0], v=v[:, :0])]:
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.linear_attention(**{**dict(q=q, k=k, v=v, decay=decay), **bad})
    with pytest.raises((ValueError, ssd.SSDError)):
        ssd.linear_attention_backward(q, k, v, decay, c["dy"][None], scale=0.0)
    with pytest.raises((ValueError, ssd.SSDError)):
        ssd.linear_attention_backward(q, k, v, decay, c["dy"][None].float())
    with pytest.raises((ValueError, ssd.SSDError)):
        ssd.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], decay, c["init"].transpose(2, 3))
    torch.cuda.synchronize()
    assert torch.equal(ssd.linear_attention(q, k, v, decay)[0], ok)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 64, 128), (BF, 128, 128), (BF, 40, 56), (F32, 64, 64),
                                       (F32, 20, 70)])
def test_later_tokens_reach_no_earlier_ones(dtype, K, V, bad):
    """Infinities and NaN from token 40, and from token 300, on (a batch's padding, say):
    outputs before them are those without, and gradients where dy is spoiled only
    before a token are those without behind it."""
    B, T, H, G = 3, 333, 4, 2
    c = make(dtype, [0, T, 2 * T, 3 * T], B * T, H, G, K, V)
    r = {n: c[n].view(B, T, *c[n].shape[1:]).clone() for n in ("q", "k", "v", "dy")}
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, c["init"], [0, T, 2 * T, 3 * T], c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    for n in ("q", "k", "v"):
        r[n][0, 40:] = bad
        r[n][1, 300:] = bad
    r["v"][2, 200] = bad  # one token's values alone
    y, _ = ssd.linear_attention(r["q"], r["k"], r["v"], c["decay"], initial_state=c["init"])
    y = y.clone()
    for b, first in ((0, 40), (1, 300), (2, 200)):
        assert not bool(torch.isfinite(y[b, first:]).all())
        ref["y"].view(B, T, H, V)[b, first:] = float("nan")  # checked above
    check({"y": y.flatten(0, 1)}, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))
    clean = {n: c[n].view(B, T, *c[n].shape[1:]) for n in ("q", "k", "v", "dy")}
    clean["dy"] = clean["dy"].clone()
    clean["dy"][0, :250] = bad
    g = ssd.linear_attention_backward(clean["q"], clean["k"], clean["v"], c["decay"], clean["dy"],
                                      initial_state=c["init"], dfinal=c["dfinal"])
    for n, d in (("dk", K), ("dv", V)):
        ref[n].view(B, T, G, d)[0, :250] = float("nan")
    check({n: g[n].flatten(0, 1) for n in ("dk", "dv")}, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))


@pytest.mark.parametrize("dtype,K,V,packed", [(BF, 128, 64, False), (BF, 128, 128, True), (F32, 20, 24, False),
                                              (F32, 20, 24, True)])
def test_cut_chains_update_the_state_in_place(dtype, K, V, packed):
    """final_state is initial_state, in chains that are cut into items: the first item
    starts from what the state held."""
    T = 3000
    c = make(dtype, [0, T], T, 2, 2, K, V)
    e = (lambda t: t) if packed else (lambda t: t[None])
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda") if packed else None
    y, final = ssd.linear_attention(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], initial_state=c["init"], cu_seqlens=cu)
    for _ in range(3):
        state = c["init"].clone()
        y2, _ = ssd.linear_attention(e(c["q"]), e(c["k"]), e(c["v"]), c["decay"], initial_state=state,
                                     final_state=state, cu_seqlens=cu)
        assert torch.equal(y2, y) and torch.equal(state, final)


def test_autograd_of_packed_rows_and_unaligned_gradients():
    """Rows of no sequence are zero in y and in the gradients; a gradient that starts off
    a 16-byte boundary is taken."""
    cuts, total, H, K, V = [4, 60, 200], 230, 2, 64, 64
    c = make(BF, cuts, total, H, H, K, V, outside=float("nan"))
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    q, k, v = (c[n].requires_grad_() for n in "qkv")
    y, _ = linear_attention_autograd(q, k, v, c["decay"], initial_state=c["init"], cu_seqlens=cu)
    assert bool((y[:4] == 0).all()) and bool((y[200:] == 0).all()) and bool(torch.isfinite(y).all())
    dy = torch.empty(total * H * V + 1, dtype=BF, device="cuda")[1:].view(total, H, V).copy_(c["dy"])
    assert dy.data_ptr() % 16 != 0
    got = torch.autograd.grad(y, [q, k, v], dy)
    want = ssd.linear_attention_backward(q.detach(), k.detach(), v.detach(), c["decay"], c["dy"], cu_seqlens=cu,
                                         initial_state=c["init"], want_dinit=False)
    for t, n in zip(got, ("dq", "dk", "dv")):
        assert torch.equal(t, want[n]) and bool((t[:4] == 0).all()) and bool((t[200:] == 0).all())


@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 64), (BF, 128, 128), (F32, 64, 64)])
def test_spoiled_queries_hide_nothing(dtype, K, V):
    """Queries that are not finite spoil their own outputs only, and values that are not,
    behind them in the sequence, still no earlier output."""
    T, H = 400, 2
    c = make(dtype, [0, T], T, H, H, K, V)
    args = (c["q"], c["k"], c["v"], c["decay"], K ** -0.5, c["init"], [0, T], c["dy"], c["dfinal"])
    ref, size = reference(*args), reference(*args, magnitude=True)
    c["q"][0:64] = float("nan")
    c["q"][140] = float("inf")
    c["v"][350:] = float("nan")
    y, _ = ssd.linear_attention(c["q"][None], c["k"][None], c["v"][None], c["decay"], initial_state=c["init"])
    for s in (slice(0, 64), slice(140, 141), slice(350, T)):
        ref["y"][s] = float("nan")
        assert not bool(torch.isfinite(y[0, s]).any())
    check({"y": y[0]}, ref, size, dtype, K, V, T, on_tensor_cores(dtype, K, V))
