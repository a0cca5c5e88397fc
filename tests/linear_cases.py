"""The definitions of linear attention with a decay for each head and of layer
norm in 64 bits, token by token and row by row, with the bounds that the tests
hold the kernels to.

Bounds.  Every result is a sum of terms; with the same recurrence over the
absolute values it is `size`, the sum of the terms' magnitudes, and a term that
passes through m roundings of unit u is off by at most (about) m u times its
magnitude.  In fp32 (u = 2^-24) a term passes through one rounding for each
addition behind it: at most the K products of a score, the chunk's tokens, the
chunks that carry it and a few factors.  On tensor cores a term is rounded to
bf16 (u = 2^-8) once more, as a masked score or as part of the state operand,
and a bf16 result once at the end.
"""
from __future__ import annotations

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8


def scan64(q, k, v, decay, init=None, reverse=False):
    """q, k [T,H,K], v [T,H,V] float64: out_t = q_t^T h_t of the scan and its last
    state.  Backwards, the initial state meets the last token undecayed."""
    T, H, K = q.shape
    lam = torch.exp(decay.double())[:, None, None]
    h = torch.zeros(H, K, v.shape[-1], dtype=torch.float64, device=q.device) if init is None else init.clone()
    out = torch.empty(T, H, v.shape[-1], dtype=torch.float64, device=q.device)
    order = range(T - 1, -1, -1) if reverse else range(T)
    for n, t in enumerate(order):
        h = (h if reverse and n == 0 else lam * h) + k[t][:, :, None] * v[t][:, None, :]
        out[t] = torch.einsum("hk,hkv->hv", q[t], h)
    return out, h


def heads64(t, H):
    return t.double().repeat_interleave(H // t.shape[-2], -2)


def reference(q, k, v, decay, scale, init, cuts, dy=None, dfinal=None, magnitude=False):
    """Rows [T,heads,d] of sequences [cuts[i], cuts[i+1]): dict of y, final and,
    with dy, dq, dk, dv, dinit in float64; NaN in rows outside every sequence.
    magnitude: the same of the absolute values."""
    H, G = q.shape[1], k.shape[1]
    m = (lambda t: t.abs()) if magnitude else (lambda t: t)
    none = float("nan")
    S, K, V = len(cuts) - 1, q.shape[2], v.shape[2]
    new = lambda *s: torch.full(s, none, dtype=torch.float64, device=q.device)  # noqa: E731
    out = {"y": new(q.shape[0], H, V), "final": new(S, H, K, V)}
    if dy is not None:
        out |= {"dq": new(*q.shape), "dk": new(*k.shape), "dv": new(*v.shape), "dinit": new(S, H, K, V)}
    scale = abs(scale) if magnitude else scale
    lam = torch.exp(decay.double())[:, None, None]
    for s in range(S):
        a, b = cuts[s], cuts[s + 1]
        qs, ks, vs = m(q[a:b].double()), m(heads64(k[a:b], H)), m(heads64(v[a:b], H))
        h0 = None if init is None else m(init[s].double())
        y, h = scan64(qs, ks, vs, decay, h0)
        out["y"][a:b], out["final"][s] = scale * y, h
        if dy is None:
            continue
        d = m(dy[a:b].double())
        g0 = None if dfinal is None else m(dfinal[s].double()) / scale
        dq, _ = scan64(d, vs, ks, decay, None if h0 is None else h0.transpose(1, 2))
        dk, _ = scan64(vs, d, qs, decay, None if g0 is None else g0.transpose(1, 2), reverse=True)
        dv, adj = scan64(ks, qs, d, decay, g0, reverse=True)
        share = lambda t: t.unflatten(1, (G, H // G)).sum(2)  # noqa: E731
        out["dq"][a:b], out["dk"][a:b], out["dv"][a:b] = scale * dq, scale * share(dk), scale * share(dv)
        out["dinit"][s] = scale * (lam * adj if b > a else adj)
    return out


def bounds(ref, size, name, dtype, K, V, longest, tensor_cores):
    """Elementwise bound for output `name`."""
    steps = max(K, V) + 128 + longest / 32 + 32  # roundings in fp32 along one term
    b = size[name] * (steps * U32)
    if name in ("final", "dinit"):
        return b + 1e-30
    if tensor_cores:
        b = b + size[name] * (U16 * 1.01)
    if dtype == torch.bfloat16:
        b = b + ref[name].abs() * (U16 * 1.01) + size[name] * U16 * (U16 if tensor_cores else steps * U32)
    return b + 1e-30


def on_tensor_cores(dtype, K, V):
    return dtype == torch.bfloat16 and K <= 128 and V <= 128 and K % 8 == 0 and V % 8 == 0


def slopes(H, device="cuda"):
    """Memories of two tokens to a thousand."""
    return -torch.exp2(-torch.linspace(0.5, 10.0, H, device=device))


def norm64(x, weight, bias, groups, gate, eps, dy=None):
    """y, stats and, with dy, the gradients, by float64 autograd."""
    leaves = {"dx": x.double(), "dweight": None if weight is None else weight.double(),
              "dbias": None if bias is None else bias.double(), "dgate": None if gate is None else gate.double()}
    leaves = {n: None if t is None else t.clone().requires_grad_() for n, t in leaves.items()}
    xg = leaves["dx"].reshape(-1, groups, x.shape[-1] // groups)
    mean = xg.mean(-1, keepdim=True)
    var = (xg - mean).square().mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    y = ((xg - mean) * rstd).reshape(x.shape)
    if weight is not None:
        y = y * leaves["dweight"]
    if bias is not None:
        y = y + leaves["dbias"]
    if gate is not None:
        y = y * (leaves["dgate"] * torch.sigmoid(leaves["dgate"]))
    out = {"y": y.detach(), "stats": torch.cat([mean, rstd], -1).detach()}
    if dy is not None:
        names = [n for n, t in leaves.items() if t is not None]
        got = torch.autograd.grad(y, [leaves[n] for n in names], dy.double())
        out |= dict(zip(names, got))
    return out
