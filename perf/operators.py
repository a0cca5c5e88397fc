"""Measured cases of linear attention with a decay for each head and of layer norm.

Five operators: linear attention over prompts (``linear``), its gradients
(``linear_backward``), its step for single tokens (``linear_step``), layer norm
(``norm``) and its gradients (``norm_backward``).  ``run`` makes the library's
calls where ``own`` is true, and computes the same in elementary torch
operations where it is not.

    h_t = exp(decay[h]) h_{t-1} + k_t v_t^T,     y_t = scale q_t^T h_t
    y = ((x - mean) rstd weight + bias) * silu(gate)
"""
import math
import random

import torch

own = False

_CHUNK = 128


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # the prompt of one short chat turn: latency
        _linear("prompt short", "bf16", 1, 200, 8, 8, 64, 64),
        # a training layer with the sizes of the 2.7B-shaped workload (80 heads of 64, state 128)
        _linear("layer 2.7b", "bf16", 4, 8192, 80, 80, 128, 64),
        # one long document, few chains, four query heads to a key/value head
        _linear("document long", "bf16", 1, 65536, 32, 8, 128, 128),
        # prompts of a serving batch packed one behind the other, resumed from their states
        _linear("prompts packed", "bf16", 24, 18011, 16, 16, 128, 128, init=True, packed=True),
        # training step of the 130M-shaped workload (24 heads of 64, state 128)
        _linear("backward 130m", "bf16", 8, 2048, 24, 24, 128, 64, op="linear_backward"),
        # fp32 check run with shared heads, odd length and a loss on the final state
        _linear("backward fp32", "f32", 2, 333, 8, 2, 48, 64, op="linear_backward", init=True),
        # one sequence being generated: latency
        _linear("step one", "bf16", 1, 1, 24, 24, 128, 64, op="linear_step"),
        # a full serving batch of the 2.7B-shaped layer
        _linear("step batch", "bf16", 128, 1, 80, 80, 128, 64, op="linear_step"),
        # the gated norm over each head behind the 2.7B-shaped layer
        _norm("norm heads gated", "bf16", 32768, 5120, 80, True),
        # the norm in front of a block while generating for 64 sequences, fp32
        _norm("norm rows small", "f32", 64, 2560, 1, False),
        # gradients of the norm over whole rows of the 2.7B-shaped model's width
        _norm("norm backward rows", "bf16", 32768, 2560, 1, False, op="norm_backward"),
        # gradients of the gated norm over heads, 130M-shaped
        _norm("norm backward heads", "bf16", 16384, 1536, 24, True, op="norm_backward"),
    ]


def _linear(name, dtype, B, T, H, G, K, V, op="linear", init=False, packed=False):
    c = {"op": op, "dtype": dtype, "B": B, "T": T, "H": H, "G": G, "K": K, "V": V, "init": init, "packed": packed}
    return dict(c, name=name) if name else c


def _norm(name, dtype, rows, width, groups, gate, op="norm"):
    c = {"op": op, "dtype": dtype, "rows": rows, "width": width, "groups": groups, "gate": gate}
    return dict(c, name=name) if name else c


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["linear", "linear", "linear_backward", "linear_step", "norm", "norm_backward"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op in ("norm", "norm_backward"):
        per_head = rng.random() < 0.5
        groups = rng.choice([2, 8, 16, 32, 80]) if per_head else 1
        n = rng.choice([32, 64, 80, 128, 100]) if per_head else log(64, 8192)
        rows = min(log(1, 40000), 160_000_000 // (n * groups))
        return _norm(None, dtype, max(1, rows), n * groups, groups, rng.random() < 0.5, op=op)
    G = rng.choice([1, 2, 4, 8, 16, 24])
    H = G * rng.choice([1, 1, 1, 2, 4])
    dims = [64, 64, 128, 128, 32, 48, 80, 96, 112, 100]
    K, V = rng.choice(dims), rng.choice(dims)
    init = rng.random() < 0.5
    if op == "linear_step":
        return _linear(None, dtype, log(1, 256), 1, H, G, K, V, op=op)
    # CUDA-core types and sizes: fewer tokens
    most = 2_000_000 if dtype == "f32" or K % 8 or V % 8 else 100_000_000
    if op == "linear_backward":
        most //= 4
    packed = rng.random() < 0.3
    B = log(2, 40) if packed else log(1, 16)
    T = log(2, 32768)
    T = min(T, most // (H * (K + V) * (1 if packed else B)))
    return _linear(None, dtype, B, max(2, T), H, G, K, V, op=op, init=init, packed=packed)


def _cuts(case):
    """Row offsets of a packed case's sequences: from its sizes alone, lengths of zero among them by chance."""
    r = random.Random(case["B"] * 1000003 + case["T"])
    return [0] + sorted(r.randint(0, case["T"]) for _ in range(case["B"] - 1)) + [case["T"]]


# ----------------------------------------------------------------- inputs ----
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    normal = lambda *shape, dtype=dt: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)  # noqa: E731
    s = {"case": case}
    if "rows" in case:
        rows, width, groups = case["rows"], case["width"], case["groups"]
        s["x"] = (normal(rows, width, dtype=torch.float32) * 1.5 + 0.3).to(dt)
        s["weight"] = 1.0 + 0.2 * normal(width, dtype=torch.float32)
        s["bias"] = 0.1 * normal(width, dtype=torch.float32)
        s["gate"] = normal(rows, width) if case["gate"] else None
        if case["op"] == "norm_backward":
            s["dy"] = normal(rows, width)
            x = s["x"].float().view(rows, groups, width // groups)
            mean = x.mean(-1)
            rstd = torch.rsqrt((x - mean[..., None]).square().mean(-1) + 1e-5)
            s["stats"] = torch.stack([mean, rstd], -1).contiguous()
        return s
    B, T, H, G, K, V = (case[n] for n in ("B", "T", "H", "G", "K", "V"))
    # slopes spread over the heads, memories of a few tokens to some thousands
    s["decay"] = -torch.exp2(-1.0 - 11.0 * torch.arange(H, device="cuda", dtype=torch.float32) / max(1, H - 1))
    lead = (T,) if case["packed"] else (B,) if case["op"] == "linear_step" else (B, T)
    if case["packed"]:
        cuts = _cuts(case)
        s["cu_seqlens"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        s["longest"] = max(b - a for a, b in zip(cuts, cuts[1:]))
    if case["op"] == "linear_backward":
        s["q"], s["k"], s["v"], s["dy"] = normal(*lead, H, K), normal(*lead, G, K), normal(*lead, G, V), normal(*lead, H, V)
        s["dfinal"] = normal(B, H, K, V, dtype=torch.float32) if case["init"] else None
    else:
        s["qkv"] = normal(*lead, H * K + G * K + G * V)  # one fused projection
    if case["op"] == "linear_step":
        s["state"] = normal(B, H, K, V, dtype=torch.float32)
    else:
        s["init"] = normal(B, H, K, V, dtype=torch.float32) if case["init"] else None
    return s


def _split(s):
    """q, k, v as views of the fused projection's output."""
    c, x = s["case"], s["qkv"]
    H, G, K, V = c["H"], c["G"], c["K"], c["V"]
    q, k, v = x.split([H * K, G * K, G * V], dim=-1)
    return q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V))


# -------------------------------------------------------------------- run ----
def run(s):
    return _OPS[s["case"]["op"]](s)


def _run_linear(s):
    q, k, v = _split(s)
    c = s["case"]
    scale = c["K"] ** -0.5
    if own:
        from ssd_chunked_forward_b200 import ssd

        y, final = ssd.linear_attention(q, k, v, s["decay"], scale=scale, initial_state=s["init"],
                                        cu_seqlens=s.get("cu_seqlens"))
        return {"y": y, "final": final}
    qp, kp, vp = _pad(s, q), _heads(_pad(s, k), c), _heads(_pad(s, v), c)
    lens, la = _lens(s), s["decay"].double()
    y = _unpad(s, _scan(qp, kp, vp, la, s["init"]) * scale)
    final = _whole_state(kp, vp, la, _to_end(la, lens, qp.shape[1]))
    if s["init"] is not None:
        final = final + torch.exp(la * lens[:, None].double()).float()[..., None, None] * s["init"]
    return {"y": y.to(q.dtype), "final": final}


def _run_linear_backward(s):
    q, k, v, dy, c = s["q"], s["k"], s["v"], s["dy"], s["case"]
    scale = c["K"] ** -0.5
    if own:
        from ssd_chunked_forward_b200 import ssd

        return ssd.linear_attention_backward(q, k, v, s["decay"], dy, scale=scale, initial_state=s["init"],
                                             dfinal=s["dfinal"], cu_seqlens=s.get("cu_seqlens"))
    qp, dyp, kp, vp = _pad(s, q), _pad(s, dy), _heads(_pad(s, k), c), _heads(_pad(s, v), c)
    lens, la, T = _lens(s), s["decay"].double(), qp.shape[1]
    dq = scale * _scan(dyp, vp, kp, la, None if s["init"] is None else s["init"].transpose(-1, -2))
    dk = scale * _scan(vp.flip(1), dyp.flip(1), qp.flip(1), la, None).flip(1)
    dv = scale * _scan(kp.flip(1), qp.flip(1), dyp.flip(1), la, None).flip(1)
    since = torch.exp(la * (torch.arange(T, device=q.device).double()[:, None] + 1))  # [T, H]: exp(decay (t + 1))
    dinit = scale * _whole_state(qp, dyp, la, since.float().expand(c["B"], -1, -1))
    if s["dfinal"] is not None:
        w = _to_end(la, lens, T)[..., None]
        dk = dk + w * torch.einsum("bthv,bhkv->bthk", vp, s["dfinal"])
        dv = dv + w * torch.einsum("bthk,bhkv->bthv", kp, s["dfinal"])
        dinit = dinit + torch.exp(la * lens[:, None].double()).float()[..., None, None] * s["dfinal"]
    share = lambda t: t.unflatten(2, (c["G"], c["H"] // c["G"])).sum(3)  # noqa: E731
    return {"dq": _unpad(s, dq).to(q.dtype), "dk": _unpad(s, share(dk)).to(q.dtype),
            "dv": _unpad(s, share(dv)).to(q.dtype), "dinit": dinit}


def _run_linear_step(s):
    q, k, v = _split(s)
    c, h = s["case"], s["state"]
    scale = c["K"] ** -0.5
    if own:
        from ssd_chunked_forward_b200 import ssd

        return {"y": ssd.linear_attention_step(q, k, v, s["decay"], h, scale=scale), "state": h}
    r = c["H"] // c["G"]
    kf, vf = k.float().repeat_interleave(r, 1), v.float().repeat_interleave(r, 1)
    h.mul_(torch.exp(s["decay"].double()).float()[:, None, None]).add_(kf[..., None] * vf[..., None, :])
    y = scale * torch.einsum("bhk,bhkv->bhv", q.float(), h)
    return {"y": y.to(q.dtype), "state": h}


def _run_norm(s):
    c = s["case"]
    if own:
        from ssd_chunked_forward_b200 import ssd

        y, stats = ssd.layer_norm(s["x"], s["weight"], s["bias"], groups=c["groups"], gate=s["gate"], eps=1e-5)
        return {"y": y, "stats": stats}
    x = s["x"].float().unflatten(-1, (c["groups"], -1))
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = torch.rsqrt(d.square().mean(-1) + 1e-5)
    y = (d * rstd[..., None]).flatten(1) * s["weight"] + s["bias"]
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * (z / (1 + torch.exp(-z)))
    return {"y": y.to(s["x"].dtype), "stats": torch.stack([mean, rstd], -1)}


def _run_norm_backward(s):
    c = s["case"]
    if own:
        from ssd_chunked_forward_b200 import ssd

        return ssd.layer_norm_backward(s["x"], s["weight"], s["bias"], s["dy"], s["stats"], groups=c["groups"],
                                       gate=s["gate"])
    mean, rstd = s["stats"][..., :1], s["stats"][..., 1:]
    group = lambda t: t.unflatten(-1, (c["groups"], -1))  # noqa: E731
    xh = ((group(s["x"].float()) - mean) * rstd).flatten(1)
    du, out = s["dy"].float(), {}
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = 1 / (1 + torch.exp(-z))
        u = xh * s["weight"] + s["bias"]
        out["dgate"] = (du * u * (sig * (1 + z * (1 - sig)))).to(s["x"].dtype)
        du = du * (z * sig)
    dxh, xg = group(du * s["weight"]), group(xh)
    dx = rstd * (dxh - dxh.mean(-1, keepdim=True) - xg * (dxh * xg).mean(-1, keepdim=True))
    out["dx"] = dx.flatten(1).to(s["x"].dtype)
    out["dweight"] = (du * xh).sum(0, dtype=torch.float64).float()
    out["dbias"] = du.sum(0, dtype=torch.float64).float()
    return out


_OPS = {"linear": _run_linear, "linear_backward": _run_linear_backward, "linear_step": _run_linear_step,
        "norm": _run_norm, "norm_backward": _run_norm_backward}


# ------------------------------------------------ the plain form's pieces ----
def _lens(s):
    if s["case"]["packed"]:
        cu = s["cu_seqlens"].long()
        return cu[1:] - cu[:-1]
    return torch.full((s["case"]["B"],), s["case"]["T"], device="cuda", dtype=torch.long)


def _pad(s, t):
    """[B, longest, heads, d] in fp32, zeros behind each sequence."""
    if not s["case"]["packed"]:
        return t.float()
    cu = s["cu_seqlens"].long()
    at = torch.arange(s["longest"], device=t.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at).clamp(max=s["case"]["T"] - 1)
    return torch.where(there[..., None, None], t[rows].float(), 0.0)


def _unpad(s, t):
    if not s["case"]["packed"]:
        return t
    cu, T = s["cu_seqlens"].long(), s["case"]["T"]
    seq = torch.repeat_interleave(cu[1:] - cu[:-1], output_size=T)
    return t[seq, torch.arange(T, device=t.device) - cu[seq]]


def _heads(t, c):
    return t.repeat_interleave(c["H"] // c["G"], 2)


def _to_end(la, lens, T):
    """[B, T, H]: exp(decay * tokens from t to the sequence's last), zero behind it."""
    left = lens[:, None] - 1 - torch.arange(T, device=la.device)
    w = torch.exp(la * left.clamp(min=0)[..., None].double()).float()
    return torch.where((left >= 0)[..., None], w, 0.0)


def _whole_state(k, v, la, w):
    """sum over t of w[b,t,h] k_t v_t^T."""
    return torch.matmul((k * w[..., None]).permute(0, 2, 3, 1), v.transpose(1, 2))


def _scan(q, k, v, la, init):
    """sum over s <= t of exp(decay (t - s)) (q_t . k_s) v_s + exp(decay (t + 1)) q_t . init, in
    chunks: masked products inside each, its state passed to every later one by one matrix."""
    T, C, dev = q.shape[1], _CHUNK, q.device
    nc = -(-T // C)
    cut = lambda t: torch.nn.functional.pad(t, (0, 0, 0, 0, 0, nc * C - T)).unflatten(1, (nc, C)).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v = cut(q), cut(k), cut(v)  # [B, H, nc, C, d]
    i = torch.arange(C, device=dev)
    apart = i[:, None] - i
    e = lambda d: torch.exp(la[:, None] * d.double().flatten()).float().unflatten(1, d.shape)  # noqa: E731
    inside = torch.where(apart >= 0, e(apart.clamp(min=0)), 0.0)  # [H, C, C]
    y = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * inside[:, None], v)
    own_state = torch.matmul((k * e(C - 1 - i)[:, None, :, None]).transpose(-1, -2), v)  # [B, H, nc, K, V]
    c = torch.arange(nc, device=dev)
    gap = c[:, None] - 1 - c
    carry = torch.where(gap >= 0, e(C * gap.clamp(min=0)), 0.0)  # [H, nc, nc]
    entering = torch.matmul(carry, own_state.flatten(-2)).unflatten(-1, own_state.shape[-2:])
    if init is not None:
        entering = entering + e(C * c)[..., None, None] * init[:, :, None]
    y = y + torch.matmul(q * e(i + 1)[:, None, :, None], entering)
    return y.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :T]


# ------------------------------------------------------------------- work ----
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if "rows" in case:
        n = case["rows"] * case["width"]
        stats = case["rows"] * case["groups"] * 8
        if case["op"] == "norm":
            return {"bytes": n * e * (3 if case["gate"] else 2) + stats + case["width"] * 8,
                    "flops": n * (12 if case["gate"] else 8)}
        return {"bytes": n * e * (5 if case["gate"] else 3) + stats + case["width"] * 16,
                "flops": n * (30 if case["gate"] else 14)}
    B, T, H, G, K, V = (case[n] for n in ("B", "T", "H", "G", "K", "V"))
    tokens = T if case["packed"] else B * T
    state = B * H * K * V * 4
    q_k_v = tokens * (H * K + G * K + G * V) * e
    out = tokens * H * V * e
    if case["op"] == "linear_backward":
        return {"bytes": 2 * q_k_v + out + state * (3 if case["init"] else 1), "flops": 10.0 * tokens * H * K * V}
    if case["op"] == "linear_step":
        return {"bytes": q_k_v + out + 2 * state, "flops": 5.0 * tokens * H * K * V}
    return {"bytes": q_k_v + out + state * (2 if case["init"] else 1), "flops": 4.0 * tokens * H * K * V}


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    """The operators token by token and row by row, in 64 bits."""
    s = prepare(case, seed)
    if "rows" in case:
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        shape = (case["rows"], case["groups"], case["width"] // case["groups"])
        if case["op"] == "norm":
            var, mean = torch.var_mean(x.reshape(shape), dim=-1, unbiased=False)
            r = (var + 1e-5) ** -0.5
            y = ((x.reshape(shape) - mean[..., None]) * r[..., None]).reshape(x.shape) * w + b
            if s["gate"] is not None:
                y *= s["gate"].double() * torch.sigmoid(s["gate"].double())
            return {"y": y, "stats": torch.stack([mean, r], dim=-1)}
        m, r = s["stats"].double().unbind(-1)
        # autograd of the definition with the given mean and rstd put in for those of x: their own
        # derivatives come from the identity that each is a function of its part of the row
        xh = ((x.reshape(shape) - m[..., None]) * r[..., None]).reshape(x.shape)
        z = None if s["gate"] is None else s["gate"].double().requires_grad_()
        wl, bl, xl = w.clone().requires_grad_(), b.clone().requires_grad_(), xh.clone().requires_grad_()
        y = xl * wl + bl
        if z is not None:
            y = y * z * torch.sigmoid(z)
        leaves = [xl, wl, bl] + ([] if z is None else [z])
        got = torch.autograd.grad(y, leaves, s["dy"].double())
        d, h = got[0].reshape(shape), xh.reshape(shape)
        n = shape[-1]
        dx = r[..., None] * (d - d.sum(-1, keepdim=True) / n - h * ((d * h).sum(-1, keepdim=True) / n))
        out = {"dx": dx.reshape(x.shape), "dweight": got[1], "dbias": got[2]}
        if z is not None:
            out["dgate"] = got[3]
        return out
    B, T, H, G, K, V = (case[n] for n in ("B", "T", "H", "G", "K", "V"))
    group = torch.arange(H, device="cuda") // (H // G)
    lam = torch.exp(s["decay"].double())[:, None, None]
    scale = K ** -0.5
    if case["op"] == "linear_step":
        q, k, v = _split(s)
        k, v = k.double()[:, group], v.double()[:, group]
        h = lam * s["state"].double() + torch.einsum("bhk,bhv->bhkv", k, v)
        return {"y": scale * torch.einsum("bhk,bhkv->bhv", q.double(), h), "state": h}
    if case["op"] == "linear":
        q, k, v = _split(s)
    else:
        q, k, v = s["q"], s["k"], s["v"]
    cuts = _cuts(case) if case["packed"] else [b * T for b in range(B + 1)]
    flat = lambda t: t.reshape(-1, *t.shape[-2:])  # noqa: E731
    q, k, v = flat(q), flat(k), flat(v)
    starts = torch.tensor(cuts[:-1], device="cuda")
    lens = torch.tensor([b - a for a, b in zip(cuts, cuts[1:])], device="cuda")
    longest = int(lens.max())
    last = q.shape[0] - 1
    h = torch.zeros(B, H, K, V, dtype=torch.float64, device="cuda") if s["init"] is None else s["init"].double()
    dy = flat(s["dy"]) if case["op"] == "linear_backward" else None
    if dy is None:
        y = torch.zeros(last + 2, H, V, dtype=torch.float64, device="cuda")
    else:
        y = torch.zeros(last + 2, H, K, dtype=torch.float64, device="cuda")
    for t in range(longest):
        live = t < lens
        row = (starts + t).clamp(max=last)
        kt, vt = k[row].double()[:, group], v[row].double()[:, group]
        new = torch.einsum("bhk,bhv->bhkv", kt, vt).addcmul_(lam.expand_as(h), h)
        h = new if longest == T and not case["packed"] else torch.where(live[:, None, None, None], new, h)
        if dy is None:
            got = torch.einsum("bhk,bhkv->bhv", q[row].double(), h)
        else:
            got = torch.einsum("bhv,bhkv->bhk", dy[row].double(), h)
        y[torch.where(live, row, last + 1)] = scale * got  # ended sequences write the spare row
    if dy is None:
        return {"y": y[:-1].reshape(*s["qkv"].shape[:-1], H, V), "final": h}
    adj = torch.zeros(B, H, K, V, dtype=torch.float64, device="cuda")
    dfinal = torch.zeros_like(adj) if s["dfinal"] is None else s["dfinal"].double()
    dk = torch.zeros(last + 2, H, K, dtype=torch.float64, device="cuda")
    dv = torch.zeros(last + 2, H, V, dtype=torch.float64, device="cuda")
    for t in range(longest - 1, -1, -1):
        live = (t < lens)[:, None, None, None]
        row = (starts + t).clamp(max=last)
        down = torch.where((t == lens - 1)[:, None, None, None], dfinal, lam * adj)
        new = down + scale * torch.einsum("bhk,bhv->bhkv", q[row].double(), dy[row].double())
        adj = torch.where(live, new, adj)
        kt, vt = k[row].double()[:, group], v[row].double()[:, group]
        to = torch.where(live.flatten(), row, last + 1)
        dk[to] = torch.einsum("bhkv,bhv->bhk", adj, vt)
        dv[to] = torch.einsum("bhkv,bhk->bhv", adj, kt)
    dinit = torch.where((lens > 0)[:, None, None, None], lam * adj, dfinal)
    share = lambda t: t[:-1].unflatten(1, (G, H // G)).sum(2)  # noqa: E731
    return {"dq": y[:-1].reshape(s["q"].shape), "dk": share(dk).reshape(s["k"].shape),
            "dv": share(dv).reshape(s["v"].shape), "dinit": dinit}
