"""Linear attention and layer norm without a GPU: the C ABI's argument checks
(every call is refused before any work is queued, or fails by the test hook), the
workspace arithmetic, and the autograd functions over the definitions."""
from __future__ import annotations

import ctypes

import pytest
import torch

from ssd_chunked_forward_b200 import ssd
from ssd_chunked_forward_b200.autograd import layer_norm_autograd, linear_attention_autograd
from tests.linear_cases import norm64, reference, slopes

OK = 1 << 20  # an aligned address that is never used


@pytest.fixture(scope="module")
def lib():
    from ssd_chunked_forward_b200.build import build
    build()
    return ssd.load()


def shape(**kw):
    base = dict(B=2, T=512, H=4, G=2, K=64, V=64, dtype=ssd.SSD_DTYPE_BF16, packed=0)
    base.update(kw)
    return ssd.LinearShape(*(base[n] for n, _ in ssd.LinearShape._fields_))


BAD = [dict(B=0), dict(T=0), dict(H=0), dict(G=0), dict(G=3), dict(K=0), dict(K=257), dict(V=0), dict(V=300),
       dict(dtype=2), dict(packed=2), dict(packed=-1), dict(T=2 ** 31 - 1), dict(B=2 ** 30, H=1 << 20, G=1)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_shapes(lib, bad):
    s = shape(**bad)
    assert ssd.linear_workspace_size(s) == 0 and ssd.linear_backward_workspace_size(s) == 0
    r = ctypes.byref(s)
    qkv = [OK, None, OK, None, OK, None]
    assert lib.ssd_linear_attention(r, *qkv, OK, None, None, 1.0, OK, None, OK, 1 << 50, None) == ssd.SSD_ERR_INVALID_ARG
    assert lib.ssd_linear_attention_step(r, *qkv, OK, 1.0, OK, OK, None) == ssd.SSD_ERR_INVALID_ARG
    assert lib.ssd_linear_attention_backward(r, *qkv, OK, None, None, 1.0, OK, None, OK, OK, OK, None, OK, 1 << 50,
                                             None) == ssd.SSD_ERR_INVALID_ARG


def refused(call, args, changes):
    for at, value, code in changes:
        bad = list(args)
        bad[at] = value
        assert call(*bad) == code, (at, value)


def test_forward_arguments(lib):
    s = shape()
    r, need = ctypes.byref(s), ssd.linear_workspace_size(s)
    neg, nan = ctypes.byref(ssd.Strides(1, -8, 8)), float("nan")
    args = [r, OK, None, OK, None, OK, None, OK, None, None, 1.0, OK, None, OK, need, None]
    I, W = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_WORKSPACE
    changes = [(0, None, I), (1, None, I), (1, OK + 1, I), (2, neg, I), (3, None, I), (4, neg, I), (5, None, I),
               (6, neg, I), (7, None, I), (8, OK, I), (9, OK + 4, I), (10, nan, I), (10, float("inf"), I), (11, None, I),
               (11, OK + 2, I), (12, OK + 8, I), (13, None, W), (13, OK + 16, W), (14, need - 1, W)]
    refused(lib.ssd_linear_attention, args, changes)
    p = shape(packed=1)
    pargs = list(args)
    pargs[0], pargs[14] = ctypes.byref(p), ssd.linear_workspace_size(p)
    refused(lib.ssd_linear_attention, pargs, [(8, None, I), (8, OK + 2, I)])


def test_step_and_backward_arguments(lib):
    I, W = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_WORKSPACE
    one = shape(T=1)
    args = [ctypes.byref(one), OK, None, OK, None, OK, None, OK, 1.0, OK, OK, None]
    refused(lib.ssd_linear_attention_step, args,
            [(0, ctypes.byref(shape(T=2)), I), (0, ctypes.byref(shape(T=1, packed=1)), I), (1, None, I), (3, None, I),
             (5, OK + 1, I), (7, None, I), (8, float("nan"), I), (9, None, I), (9, OK + 4, I), (10, None, I)])
    s = shape()
    need = ssd.linear_backward_workspace_size(s)
    args = [ctypes.byref(s), OK, None, OK, None, OK, None, OK, None, None, 1.0, OK, None, OK, OK, OK, None, OK, need,
            None]
    refused(lib.ssd_linear_attention_backward, args,
            [(8, OK, I), (9, OK + 4, I), (10, 0.0, I), (10, float("inf"), I), (11, None, I), (11, OK + 2, I),
             (12, OK + 4, I), (13, None, I), (14, None, I), (15, OK + 8, I), (16, OK + 4, I), (17, None, W),
             (17, OK + 64, W), (18, need - 1, W)])


def test_norm_arguments(lib):
    I, W = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_WORKSPACE
    ns = lambda *a: ctypes.byref(ssd.NormShape(*a))  # noqa: E731
    args = [ns(8, 128, 2, 1), OK, 128, OK, OK, None, 0, 1e-5, OK, OK, None]
    refused(lib.ssd_layer_norm, args,
            [(0, None, I), (0, ns(0, 128, 2, 1), I), (0, ns(8, 128, 3, 1), I), (0, ns(8, 128, 0, 1), I),
             (0, ns(8, 0, 1, 1), I), (0, ns(8, 32768, 1, 1), I), (0, ns(8, 128, 2, 5), I), (1, None, I), (1, OK + 1, I),
             (2, -1, I), (3, OK + 2, I), (7, 0.0, I), (7, -1.0, I), (7, float("nan"), I), (8, None, I), (9, OK + 4, I)])
    s = ssd.NormShape(8, 128, 2, 1)
    need = lib.ssd_layer_norm_backward_workspace_size(ctypes.byref(s))
    assert need >= 2 * 128 * 4 and lib.ssd_layer_norm_backward_workspace_size(ns(8, 128, 3, 1)) == 0
    args = [ctypes.byref(s), OK, 128, OK, OK, OK, 128, OK, 128, OK, OK, OK, OK, OK, OK, need, None]
    refused(lib.ssd_layer_norm_backward, args,
            [(0, ns(8, 32768, 1, 1), I), (1, None, I), (7, None, I), (8, -4, I), (9, None, I), (10, None, I),
             (11, OK + 2, I), (13, None, I), (5, None, I), (14, None, W), (14, OK + 4, W), (15, need - 1, W)])


def test_failed_launch_is_reported(lib):
    s = shape()
    lib.ssd_test_fail_calls(4)
    qkv = [OK, None, OK, None, OK, None]
    E = ssd.SSD_ERR_CUDA
    assert lib.ssd_linear_attention(ctypes.byref(s), *qkv, OK, None, None, 1.0, OK, None, OK, 1 << 40, None) == E
    assert lib.ssd_linear_attention_backward(ctypes.byref(s), *qkv, OK, None, None, 1.0, OK, None, OK, OK, OK, None,
                                             OK, 1 << 40, None) == E
    assert lib.ssd_linear_attention_step(ctypes.byref(shape(T=1)), *qkv, OK, 1.0, OK, OK, None) == E
    n = ssd.NormShape(8, 128, 2, 1)
    assert lib.ssd_layer_norm(ctypes.byref(n), OK, 128, None, None, None, 0, 1e-5, OK, None, None) == E
    assert lib.ssd_test_pending_failures() == 0


def test_workspace_holds_the_cut_chains(lib):
    """Whole rounds of chains are run whole; a few long chains are cut into
    items with a state each; the shared heads' gradients add fp32 partials."""
    whole = ssd.linear_workspace_size(shape(B=74, H=4, T=512))  # 296 chains: two rounds of 148
    assert whole == 256
    few = ssd.linear_workspace_size(shape(B=1, H=4, T=8192))
    assert few > 256 and (few - 256) % 256 == 0
    assert few <= 256 + 4 * 64 * 64 * 64 * 4  # a state for each chunk at most
    a = ssd.linear_backward_workspace_size(shape(G=4, T=128))
    b = ssd.linear_backward_workspace_size(shape(G=2, T=128))
    assert b - a == 2 * (2 * 128 * 4 * 64 * 4)


def test_python_refuses_cpu_tensors_and_bad_layouts():
    q, decay = torch.zeros(1, 4, 2, 8), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.linear_attention(q, q, q, decay)
    with pytest.raises(ValueError, match="dimensions"):
        ssd.linear_attention(q, q, q, decay, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ssd.linear_attention(q.half(), q.half(), q.half(), decay)
    with pytest.raises(ValueError, match="dimensions"):
        ssd.linear_attention_step(q, q, q, decay, q)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.layer_norm(q)


class _Linear:
    """The definition in place of the kernels."""

    @staticmethod
    def _run(q, k, v, decay, scale, init, cu, dy=None, dfinal=None):
        T = q.shape[-3]
        cuts = cu.tolist() if cu is not None else [T * b for b in range(q.shape[0] + 1)]
        flat = lambda t: t if t is None or cu is not None else t.flatten(0, 1)  # noqa: E731
        return reference(flat(q), flat(k), flat(v), decay, scale, init, cuts, flat(dy), dfinal)

    @classmethod
    def forward(cls, q, k, v, decay, *, scale, initial_state, cu_seqlens):
        r = cls._run(q, k, v, decay, scale, initial_state, cu_seqlens)
        return r["y"].view(*q.shape[:-1], v.shape[-1]), r["final"]

    @classmethod
    def backward(cls, q, k, v, decay, dy, *, scale, initial_state, dfinal, cu_seqlens, want_dinit):
        r = cls._run(q, k, v, decay, scale, initial_state, cu_seqlens, dy, dfinal)
        return {"dq": r["dq"].view(q.shape), "dk": r["dk"].view(k.shape), "dv": r["dv"].view(v.shape),
                "dinit": r["dinit"] if want_dinit else None}


@pytest.mark.parametrize("packed", [False, True])
def test_linear_autograd_against_differences(packed):
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()  # noqa: E731
    lead = (9,) if packed else (2, 5)
    cu = torch.tensor([0, 4, 4, 9], dtype=torch.int32) if packed else None
    S = 3 if packed else 2
    q, k, v, h = rnd(*lead, 4, 3), rnd(*lead, 2, 3), rnd(*lead, 2, 5), rnd(S, 4, 3, 5)
    f = lambda q, k, v, h: linear_attention_autograd(q, k, v, slopes(4, "cpu"), scale=0.4, initial_state=h,  # noqa: E731
                                                     cu_seqlens=cu, ops=_Linear)
    assert torch.autograd.gradcheck(f, (q, k, v, h))
    y, _ = f(q, k, v, h.detach())
    assert torch.autograd.grad(y.sum(), q)[0].shape == q.shape
    _, final = f(q, k, v, h)  # a loss on the state alone
    assert torch.autograd.grad(final.sum(), k)[0].abs().sum() > 0
    with pytest.raises(ValueError, match="no gradient"):
        linear_attention_autograd(q, k, v, slopes(4, "cpu").requires_grad_(), ops=_Linear)


class _Norm:
    @staticmethod
    def forward(x, weight, bias, *, groups, gate, eps):
        r = norm64(x, weight, bias, groups, gate, eps)
        return r["y"], r["stats"]

    @staticmethod
    def backward(x, weight, bias, dy, stats, *, groups, gate, want_dweight, want_dbias):
        with torch.enable_grad():
            r = norm64(x, weight, bias, groups, gate, 1e-5, dy)
        return {n: r.get(n) for n in ("dx", "dweight", "dbias", "dgate")}


def test_norm_autograd_against_differences():
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()  # noqa: E731
    f = lambda x, w, b, z: layer_norm_autograd(x, w, b, groups=2, gate=z, ops=_Norm)  # noqa: E731
    assert torch.autograd.gradcheck(f, (rnd(3, 8), rnd(8), rnd(8), rnd(3, 8)))
    assert torch.autograd.gradcheck(lambda x: layer_norm_autograd(x, ops=_Norm), (rnd(2, 6),))
