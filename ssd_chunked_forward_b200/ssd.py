"""ctypes binding of libssd (include/ssd.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
turns torch tensors into device pointers, the current torch stream into a
``cudaStream_t`` and status codes into exceptions.  There is no fallback: if
``libssd.so`` is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssd.so")
# the index-checked build, loaded instead when SSD_DEBUG_CHECKS=1
DEBUG_LIB_PATH = os.path.join(_HERE, "libssd_debug.so")

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_WORKSPACE, SSD_ERR_CUDA, SSD_ERR_TIMEOUT = range(6)
SSD_DTYPE_F32, SSD_DTYPE_BF16 = 0, 1
PATH_AUTO, PATH_MODULAR, PATH_SIMT, PATH_FUSED, PATH_SPLIT = 0, 1, 2, 3, 4
IMPL_AUTO, IMPL_SIMT, IMPL_TC = 0, 1, 2
FLAG_TEST_STALL = 0x100

EXPORTS = [
    "ssd_status_string", "ssd_workspace_size", "ssd_path_supported", "ssd_forward",
    "ssd_forward_path", "ssd_device_status", "ssd_chunk_cumsum", "ssd_chunk_state",
    "ssd_state_pass", "ssd_chunk_scan", "ssd_diag_scan", "ssd_forward_host_bytes",
    "ssd_forward_host", "ssd_forward_noalloc", "ssd_auto_path", "ssd_forward_init",
    "ssd_decode_step", "ssd_discretize", "ssd_decay_total", "ssd_state_combine",
    "ssd_segment_state", "ssd_backward", "ssd_backward_workspace_size",
    "ssd_test_fail_calls", "ssd_test_pending_failures", "ssd_split_pieces",
    "ssd_device_status_where", "ssd_forward_discretized", "ssd_debug_build", "ssd_debug_record",
    "ssd_debug_fail_all", "ssd_linear_attention", "ssd_linear_workspace_size",
    "ssd_linear_attention_step", "ssd_linear_attention_backward", "ssd_linear_backward_workspace_size",
    "ssd_layer_norm", "ssd_layer_norm_backward", "ssd_layer_norm_backward_workspace_size",
]


class SSDError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)}")


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "H", "P", "G", "N", "chunk", "a_per_state", "dtype")]

    def __repr__(self):
        return "Shape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class LinearShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "H", "G", "K", "V", "dtype", "packed")]


class Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_longlong) for n in ("batch", "token", "head")]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("width", ctypes.c_int), ("groups", ctypes.c_int),
                ("dtype", ctypes.c_int)]


_lib = None


def load(path: str = None):
    """Open libssd.so (built by ``ssd_chunked_forward_b200.build``), or the
    index-checked libssd_debug.so when the environment sets SSD_DEBUG_CHECKS=1."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = DEBUG_LIB_PATH if os.environ.get("SSD_DEBUG_CHECKS") == "1" else LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libssd.so not built ({path}); run python -m ssd_chunked_forward_b200.build")
    lib = ctypes.CDLL(path)
    vp, fp, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
    sp = ctypes.POINTER(Shape)
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_workspace_size.argtypes = [sp]
    lib.ssd_workspace_size.restype = sz
    lib.ssd_path_supported.argtypes = [sp, ctypes.c_uint]
    lib.ssd_path_supported.restype = ctypes.c_int
    lib.ssd_auto_path.argtypes = [sp]
    lib.ssd_auto_path.restype = ctypes.c_int
    lib.ssd_split_pieces.argtypes = [sp]
    lib.ssd_split_pieces.restype = ctypes.c_int
    lib.ssd_forward.argtypes = [sp, vp, fp, vp, vp, fp, vp, fp, vp, sz, vp]
    lib.ssd_forward_path.argtypes = [sp, vp, fp, vp, vp, fp, vp, fp, vp, sz, vp, ctypes.c_uint, ctypes.c_uint]
    lib.ssd_forward_init.argtypes = [sp, vp, fp, vp, vp, fp, fp, vp, fp, vp, sz, vp, ctypes.c_uint,
                                     ctypes.c_uint]
    lib.ssd_device_status.argtypes = [vp, vp]
    ip = ctypes.POINTER(ctypes.c_int)
    lib.ssd_device_status_where.argtypes = [vp, vp, ip, ip, ip]
    lib.ssd_debug_build.argtypes = []
    lib.ssd_debug_build.restype = ctypes.c_int
    lib.ssd_debug_record.argtypes = [ip, ip, ip, ip]
    lib.ssd_debug_fail_all.argtypes = [ctypes.c_int]
    lib.ssd_chunk_cumsum.argtypes = [sp, fp, fp, vp]
    lib.ssd_chunk_state.argtypes = [sp, vp, vp, fp, fp, vp, ctypes.c_uint]
    lib.ssd_state_pass.argtypes = [sp, fp, fp, fp, vp]
    lib.ssd_chunk_scan.argtypes = [sp, vp, vp, vp, fp, fp, fp, vp, vp, ctypes.c_uint]
    lib.ssd_diag_scan.argtypes = [sp, vp, vp, vp, fp, fp, fp, vp, vp, ctypes.c_uint]
    lib.ssd_forward_host_bytes.argtypes = [sp]
    lib.ssd_forward_host_bytes.restype = sz
    lib.ssd_forward_host.argtypes = [sp, vp, fp, vp, vp, fp, vp, fp, vp, sz, vp]
    lib.ssd_forward_noalloc.argtypes = [sp, vp, fp, vp, vp, fp, vp, fp, vp]
    lib.ssd_decode_step.argtypes = [sp, vp, fp, vp, vp, fp, fp, vp, vp]
    lib.ssd_discretize.argtypes = [sp, fp, fp, fp, vp, fp, vp, vp]
    lib.ssd_forward_discretized.argtypes = [sp, vp, fp, fp, fp, vp, vp, fp, vp, fp, vp, sz, vp]
    lib.ssd_decay_total.argtypes = [sp, fp, fp, vp]
    lib.ssd_state_combine.argtypes = [sp, ctypes.c_int, fp, fp, fp, fp, vp]
    lib.ssd_segment_state.argtypes = [sp, vp, fp, vp, fp, fp, vp, sz, vp]
    lib.ssd_test_fail_calls.argtypes = [ctypes.c_int]
    lib.ssd_test_fail_calls.restype = None
    lib.ssd_test_pending_failures.argtypes = []
    lib.ssd_test_pending_failures.restype = ctypes.c_int
    lib.ssd_backward.argtypes = [sp, vp, fp, vp, vp, fp, fp, vp, fp, vp, fp, vp, vp, fp, fp, vp, sz, vp]
    lib.ssd_backward_workspace_size.argtypes = [sp]
    lib.ssd_backward_workspace_size.restype = sz
    lp, np_, stp, ll = ctypes.POINTER(LinearShape), ctypes.POINTER(NormShape), ctypes.POINTER(Strides), ctypes.c_longlong
    qkv = [vp, stp, vp, stp, vp, stp]
    lib.ssd_linear_attention.argtypes = [lp] + qkv + [fp, vp, fp, ctypes.c_float, vp, fp, vp, sz, vp]
    lib.ssd_linear_attention_step.argtypes = [lp] + qkv + [fp, ctypes.c_float, fp, vp, vp]
    lib.ssd_linear_attention_backward.argtypes = ([lp] + qkv + [fp, vp, fp, ctypes.c_float, vp, fp, vp, vp, vp, fp,
                                                               vp, sz, vp])
    lib.ssd_layer_norm.argtypes = [np_, vp, ll, fp, fp, vp, ll, ctypes.c_float, vp, fp, vp]
    lib.ssd_layer_norm_backward.argtypes = [np_, vp, ll, fp, fp, vp, ll, vp, ll, fp, vp, fp, fp, vp, vp, sz, vp]
    for name, arg in (("ssd_linear_workspace_size", lp), ("ssd_linear_backward_workspace_size", lp),
                      ("ssd_layer_norm_backward_workspace_size", np_)):
        getattr(lib, name).argtypes = [arg]
        getattr(lib, name).restype = sz
    for name in ("ssd_linear_attention", "ssd_linear_attention_step", "ssd_linear_attention_backward",
                 "ssd_layer_norm", "ssd_layer_norm_backward"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("ssd_forward_noalloc", "ssd_forward", "ssd_forward_path", "ssd_forward_init",
                 "ssd_device_status", "ssd_chunk_cumsum", "ssd_decode_step", "ssd_discretize",
                 "ssd_decay_total", "ssd_state_combine", "ssd_segment_state", "ssd_backward",
                 "ssd_chunk_state", "ssd_state_pass", "ssd_chunk_scan", "ssd_diag_scan",
                 "ssd_forward_host", "ssd_device_status_where", "ssd_forward_discretized"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().ssd_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != SSD_OK:
        raise SSDError(code, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _torch_stream(stream, device):
    """``stream`` (a torch stream, another object with a ``cuda_stream``, or a
    raw handle) as a torch stream of ``device``."""
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            raise ValueError(f"stream must be on {device}")
        return stream
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if handle in (0, 1):  # the legacy default stream by its two names
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def _on(stream, fn, *args, **kw):
    """fn(*args, **kw), a call that allocates, as under ``torch.cuda.stream(stream)``:
    what it allocates, clears and copies is queued there like its kernels, and
    temporary memory goes back to that stream's pool, whose next user runs behind
    them.  New results are also marked as used by the caller's own stream, so that
    dropping them there is safe while it still reads them."""
    given = [t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)]
    if not given or not given[0].is_cuda:  # (fn refuses them)
        return fn(*args, **kw)
    here, side = torch.cuda.current_stream(given[0].device), _torch_stream(stream, given[0].device)
    with torch.cuda.stream(side):
        out = fn(*args, **kw)
    if side != here:
        for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
            if t is not None and not any(t is g for g in given):
                t.record_stream(here)
    return out


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_shape(B, T, H, P, G, N, chunk, a_per_state=False, dtype="bf16") -> Shape:
    dt = SSD_DTYPE_BF16 if dtype in ("bf16", torch.bfloat16) else SSD_DTYPE_F32
    return Shape(int(B), int(T), int(H), int(P), int(G), int(N), int(chunk), int(bool(a_per_state)), dt)


def shape_of(x: torch.Tensor, a: torch.Tensor, Bm: torch.Tensor, chunk: int) -> Shape:
    B, T, H, P = x.shape
    G, N = Bm.shape[2], Bm.shape[3]
    return make_shape(B, T, H, P, G, N, chunk, a.dim() == 4, x.dtype)


def workspace_size(shape: Shape) -> int:
    return int(load().ssd_workspace_size(ctypes.byref(shape)))


def path_supported(shape: Shape, path: int) -> bool:
    return bool(load().ssd_path_supported(ctypes.byref(shape), int(path)))


def auto_path(shape: Shape) -> int:
    """The path SSD_PATH_AUTO takes for this shape (PATH_FUSED, PATH_SPLIT or
    PATH_MODULAR)."""
    return int(load().ssd_auto_path(ctypes.byref(shape)))


def split_pieces(shape: Shape) -> int:
    """Pieces per sequence of the split path (1: not split, 0: invalid)."""
    return int(load().ssd_split_pieces(ctypes.byref(shape)))


def alloc_workspace(shape: Shape, device=None) -> torch.Tensor:
    n = workspace_size(shape)
    if n == 0:
        raise SSDError(SSD_ERR_INVALID_ARG, "ssd_workspace_size")
    # torch's caching allocator returns >= 512-byte aligned blocks
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _check_inputs(x, a, Bm, Cm, D):
    for name, t in (("x", x), ("a", a), ("Bm", Bm), ("Cm", Cm)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if a.dtype != torch.float32:
        raise ValueError("a must be float32")
    if x.dtype not in (torch.float32, torch.bfloat16) or Bm.dtype != x.dtype or Cm.dtype != x.dtype:
        raise ValueError("x, Bm, Cm must share dtype float32 or bfloat16")
    if D is not None and (D.dtype != torch.float32 or not D.is_cuda or not D.is_contiguous()):
        raise ValueError("D must be a contiguous float32 CUDA tensor")


def forward(x, a, Bm, Cm, D=None, chunk=256, *, y=None, final_state=None, want_final=True,
            workspace=None, path=PATH_AUTO, flags=0, stream=None, initial_state=None):
    """y[B,T,H,P] (and final state [B,H,N,P] fp32) of the chunked SSD forward.

    x [B,T,H,P], Bm/Cm [B,T,G,N] (float32 or bfloat16, same dtype), a [B,T,H]
    or [B,T,H,N] float32 log-decays, D [H] float32 or None, initial_state
    [B,H,N,P] float32 or None (zero).  Asynchronous on the current torch
    stream, or on ``stream``, where what it allocates then belongs too; the order
    of that stream with the inputs is the caller's, as for every call here."""
    if stream is not None:
        return _on(stream, forward, x, a, Bm, Cm, D, chunk, y=y, final_state=final_state, want_final=want_final,
                   workspace=workspace, path=path, flags=flags, initial_state=initial_state)
    _check_inputs(x, a, Bm, Cm, D)
    if initial_state is not None and (initial_state.dtype != torch.float32 or not initial_state.is_cuda
                                      or not initial_state.is_contiguous()):
        raise ValueError("initial_state must be a contiguous float32 CUDA tensor")
    shape = shape_of(x, a, Bm, chunk)
    B, T, H, P = x.shape
    N = Bm.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and want_final:
        final_state = torch.empty((B, H, N, P), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(shape, x.device)
    if initial_state is not None:
        if tuple(initial_state.shape) != (B, H, N, P):
            raise ValueError("initial_state must be [B,H,N,P]")
        code = load().ssd_forward_init(ctypes.byref(shape), _ptr(x), _ptr(a), _ptr(Bm), _ptr(Cm),
                                       _ptr(D), _ptr(initial_state), _ptr(y), _ptr(final_state),
                                       _ptr(workspace), workspace.numel(), _stream(stream), int(path),
                                       int(flags))
        _check(code, "ssd_forward_init")
        return y, final_state
    code = load().ssd_forward_path(ctypes.byref(shape), _ptr(x), _ptr(a), _ptr(Bm), _ptr(Cm),
                                   _ptr(D), _ptr(y), _ptr(final_state), _ptr(workspace),
                                   workspace.numel(), _stream(stream), int(path), int(flags))
    _check(code, "ssd_forward_path")
    return y, final_state


def device_status(workspace, stream=None) -> int:
    """Synchronise and return the workspace status word (SSD_OK or an error)."""
    return int(load().ssd_device_status(_ptr(workspace), _stream(stream)))


def debug_build() -> bool:
    """True when the loaded library is the index-checked debug build."""
    return bool(load().ssd_debug_build())


def debug_record():
    """(failed checks, line, block, thread) since the last call, then cleared;
    debug build only (raises SSDError otherwise)."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    _check(load().ssd_debug_record(*(ctypes.byref(v) for v in vals)), "ssd_debug_record")
    return tuple(v.value for v in vals)


def debug_fail_all(on: bool) -> None:
    """Debug build only: make every index check fail (and skip its access)."""
    _check(load().ssd_debug_fail_all(1 if on else 0), "ssd_debug_fail_all")


def device_status_where(workspace, stream=None):
    """(status, source line, block, thread) of the first bounded wait that ran
    out in a fused-path kernel; zeros when none did."""
    line, block, thread = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = int(load().ssd_device_status_where(_ptr(workspace), _stream(stream), ctypes.byref(line),
                                            ctypes.byref(block), ctypes.byref(thread)))
    return st, line.value, block.value, thread.value


def chunk_cumsum(shape: Shape, a, cum=None, stream=None):
    if stream is not None and cum is None:
        return _on(stream, chunk_cumsum, shape, a, None)
    nc = -(-shape.T // shape.chunk)  # the last chunk may end past T
    if cum is None:
        dims = (shape.B, shape.H, nc, shape.chunk) + ((shape.N,) if shape.a_per_state else ())
        cum = torch.empty(dims, dtype=torch.float32, device=a.device)
    _check(load().ssd_chunk_cumsum(ctypes.byref(shape), _ptr(a), _ptr(cum), _stream(stream)),
           "ssd_chunk_cumsum")
    return cum


def chunk_state(shape: Shape, x, Bm, cum, states=None, impl=IMPL_AUTO, stream=None):
    if stream is not None and states is None:
        return _on(stream, chunk_state, shape, x, Bm, cum, None, impl)
    nc = -(-shape.T // shape.chunk)  # the last chunk may end past T
    if states is None:
        states = torch.empty((shape.B, shape.H, nc, shape.N, shape.P), dtype=torch.float32,
                             device=x.device)
    _check(load().ssd_chunk_state(ctypes.byref(shape), _ptr(x), _ptr(Bm), _ptr(cum), _ptr(states),
                                  _stream(stream), int(impl)), "ssd_chunk_state")
    return states


def state_pass(shape: Shape, cum, states, final_state=None, stream=None):
    _check(load().ssd_state_pass(ctypes.byref(shape), _ptr(cum), _ptr(states), _ptr(final_state),
                                 _stream(stream)), "ssd_state_pass")
    return states, final_state


def chunk_scan(shape: Shape, x, Bm, Cm, cum, Hin, D=None, y=None, impl=IMPL_AUTO, stream=None):
    if stream is not None and y is None:
        return _on(stream, chunk_scan, shape, x, Bm, Cm, cum, Hin, D, None, impl)
    if y is None:
        y = torch.empty_like(x)
    fn = load().ssd_diag_scan if shape.a_per_state else load().ssd_chunk_scan
    _check(fn(ctypes.byref(shape), _ptr(x), _ptr(Bm), _ptr(Cm), _ptr(cum), _ptr(Hin), _ptr(D),
              _ptr(y), _stream(stream), int(impl)),
           "ssd_diag_scan" if shape.a_per_state else "ssd_chunk_scan")
    return y


def forward_host_bytes(shape: Shape) -> int:
    return int(load().ssd_forward_host_bytes(ctypes.byref(shape)))


def forward_host(shape: Shape, x_h, a_h, Bm_h, Cm_h, D_h, y_h, final_h, dev_buf, stream=None):
    """The forward from HOST buffers (pinned for asynchrony): the library copies
    the inputs to ``dev_buf``, runs, and copies y (and the final state) back,
    all queued on the stream.  The caller synchronises."""
    _check(load().ssd_forward_host(ctypes.byref(shape), _ptr(x_h), _ptr(a_h), _ptr(Bm_h), _ptr(Cm_h),
                                   _ptr(D_h), _ptr(y_h), _ptr(final_h), _ptr(dev_buf),
                                   dev_buf.numel(), _stream(stream)), "ssd_forward_host")


def forward_noalloc(x, a, Bm, Cm, D=None, chunk=256, *, y=None, final_state=None, stream=None):
    """The fused forward with the library's own fixed scratch (no workspace,
    nothing allocated by the library); see ssd_forward_noalloc in ssd.h."""
    if stream is not None:
        return _on(stream, forward_noalloc, x, a, Bm, Cm, D, chunk, y=y, final_state=final_state)
    _check_inputs(x, a, Bm, Cm, D)
    shape = shape_of(x, a, Bm, chunk)
    B, T, H, P = x.shape
    N = Bm.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if final_state is None:
        final_state = torch.empty((B, H, N, P), dtype=torch.float32, device=x.device)
    _check(load().ssd_forward_noalloc(ctypes.byref(shape), _ptr(x), _ptr(a), _ptr(Bm), _ptr(Cm),
                                      _ptr(D), _ptr(y), _ptr(final_state), _stream(stream)),
           "ssd_forward_noalloc")
    return y, final_state


def decode_step(x, a, Bm, Cm, D, state, *, y=None, stream=None):
    """One recurrent step for a batch of single tokens, in place on ``state``.

    x [B,H,P], Bm/Cm [B,G,N] (float32 or bfloat16), a [B,H] or [B,H,N] float32
    log-decays, D [H] float32 or None, state [B,H,N,P] float32 (updated).
    Returns y [B,H,P]."""
    if stream is not None:
        return _on(stream, decode_step, x, a, Bm, Cm, D, state, y=y)
    for name, t in (("x", x), ("a", a), ("Bm", Bm), ("Cm", Cm), ("state", state)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if a.dtype != torch.float32 or state.dtype != torch.float32:
        raise ValueError("a and state must be float32")
    if Bm.dtype != x.dtype or Cm.dtype != x.dtype:
        raise ValueError("x, Bm, Cm must share dtype")
    B, H, P = x.shape
    G, N = Bm.shape[1], Bm.shape[2]
    if tuple(state.shape) != (B, H, N, P):
        raise ValueError("state must be [B,H,N,P]")
    shape = make_shape(B, 1, H, P, G, N, 1, a.dim() == 3, x.dtype)
    if y is None:
        y = torch.empty_like(x)
    _check(load().ssd_decode_step(ctypes.byref(shape), _ptr(x), _ptr(a), _ptr(Bm), _ptr(Cm), _ptr(D),
                                  _ptr(state), _ptr(y), _stream(stream)), "ssd_decode_step")
    return y


def discretize(dt_raw, dt_bias, A_log, x, *, a_out=None, x_out=None, stream=None):
    """dt = softplus(dt_raw + dt_bias); returns (a, x_out): a = -dt exp(A_log)
    ([B,T,H], or [B,T,H,N] when A_log is [H,N]) and x_out = dt x ([B,T,H,P],
    x's dtype), the inputs of forward()."""
    if stream is not None:
        return _on(stream, discretize, dt_raw, dt_bias, A_log, x, a_out=a_out, x_out=x_out)
    for name, t in (("dt_raw", dt_raw), ("A_log", A_log), ("x", x)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dt_raw.dtype != torch.float32 or A_log.dtype != torch.float32:
        raise ValueError("dt_raw and A_log must be float32")
    B, T, H, P = x.shape
    per_state = A_log.dim() == 2
    N = A_log.shape[1] if per_state else 1
    shape = make_shape(B, T, H, P, 1, N, 1, per_state, x.dtype)
    if a_out is None:
        a_out = torch.empty((B, T, H) + ((N,) if per_state else ()), dtype=torch.float32, device=x.device)
    if x_out is None:
        x_out = torch.empty_like(x)
    _check(load().ssd_discretize(ctypes.byref(shape), _ptr(dt_raw), _ptr(dt_bias), _ptr(A_log), _ptr(x),
                                 _ptr(a_out), _ptr(x_out), _stream(stream)), "ssd_discretize")
    return a_out, x_out


def forward_discretized(x, dt_raw, dt_bias, A_log, Bm, Cm, D=None, chunk=256, *, y=None, final_state=None,
                        want_final=True, workspace=None, stream=None):
    """discretize() followed by forward() in one fused pass (x_out and a are never
    written): y = SSD(dt x, -dt exp(A_log), Bm, Cm) + D (dt x), dt = softplus(dt_raw
    + dt_bias).  x [B,T,H,P] bf16, dt_raw [B,T,H] float32, dt_bias [H] or None,
    A_log [H] float32 (scalar decay only)."""
    if stream is not None:
        return _on(stream, forward_discretized, x, dt_raw, dt_bias, A_log, Bm, Cm, D, chunk, y=y,
                   final_state=final_state, want_final=want_final, workspace=workspace)
    for name, t in (("dt_raw", dt_raw), ("A_log", A_log)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    B, T, H, P = x.shape
    if tuple(dt_raw.shape) != (B, T, H) or tuple(A_log.shape) != (H,):
        raise ValueError("dt_raw must be [B,T,H] and A_log [H]")
    _check_inputs(x, dt_raw, Bm, Cm, D)
    shape = shape_of(x, dt_raw, Bm, chunk)
    N = Bm.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and want_final:
        final_state = torch.empty((B, H, N, P), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(shape, x.device)
    _check(load().ssd_forward_discretized(ctypes.byref(shape), _ptr(x), _ptr(dt_raw), _ptr(dt_bias),
                                          _ptr(A_log), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(y),
                                          _ptr(final_state), _ptr(workspace), workspace.numel(),
                                          _stream(stream)), "ssd_forward_discretized")
    return y, final_state


def decay_total(a, *, out=None, stream=None):
    """Total log-decay of each chain over the sequence: a [B,T,H] -> [B,H]
    (a [B,T,H,N] -> [B,H,N])."""
    if stream is not None:
        return _on(stream, decay_total, a, out=out)
    if not a.is_cuda or not a.is_contiguous() or a.dtype != torch.float32:
        raise ValueError("a must be a contiguous float32 CUDA tensor")
    B, T, H = a.shape[:3]
    per_state = a.dim() == 4
    N = a.shape[3] if per_state else 1
    shape = make_shape(B, T, H, 1, 1, N, 1, per_state, torch.float32)
    if out is None:
        out = torch.empty((B, H) + ((N,) if per_state else ()), dtype=torch.float32, device=a.device)
    _check(load().ssd_decay_total(ctypes.byref(shape), _ptr(a), _ptr(out), _stream(stream)),
           "ssd_decay_total")
    return out


def state_combine(finals, totals, h0=None, *, out=None, stream=None):
    """finals [S,B,H,N,P] (each segment's final state from zero), totals
    [S,B,H] or [S,B,H,N] -> h_in [S+1,B,H,N,P]: h_in[s] enters segment s,
    h_in[S] is the state after all of them (h0, or zero, enters segment 0)."""
    if stream is not None:
        return _on(stream, state_combine, finals, totals, h0, out=out)
    for name, t in (("finals", finals), ("totals", totals)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    S, B, H, N, P = finals.shape
    per_state = totals.dim() == 4
    shape = make_shape(B, 1, H, P, 1, N, 1, per_state, torch.float32)
    if out is None:
        out = torch.empty((S + 1, B, H, N, P), dtype=torch.float32, device=finals.device)
    _check(load().ssd_state_combine(ctypes.byref(shape), int(S), _ptr(finals), _ptr(totals), _ptr(h0),
                                    _ptr(out), _stream(stream)), "ssd_state_combine")
    return out


def segment_state(x, a, Bm, chunk=256, *, final_state=None, total=None, workspace=None, stream=None):
    """The state a segment builds from a zero start, [B,H,N,P] fp32, and its
    total log-decay [B,H] (or [B,H,N]), without computing its outputs."""
    if stream is not None:
        return _on(stream, segment_state, x, a, Bm, chunk, final_state=final_state, total=total,
                   workspace=workspace)
    for name, t in (("x", x), ("a", a), ("Bm", Bm)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    shape = shape_of(x, a, Bm, chunk)
    B, T, H, P = x.shape
    N = Bm.shape[3]
    if final_state is None:
        final_state = torch.empty((B, H, N, P), dtype=torch.float32, device=x.device)
    if total is None:
        total = torch.empty((B, H) + ((N,) if a.dim() == 4 else ()), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(shape, x.device)
    _check(load().ssd_segment_state(ctypes.byref(shape), _ptr(x), _ptr(a), _ptr(Bm), _ptr(final_state),
                                    _ptr(total), _ptr(workspace), workspace.numel(), _stream(stream)),
           "ssd_segment_state")
    return final_state, total


def backward_workspace_size(shape: Shape) -> int:
    return int(load().ssd_backward_workspace_size(ctypes.byref(shape)))


def backward(x, a, Bm, Cm, D, dy, chunk=256, *, dfinal=None, initial_state=None, want_dD=True,
             want_dinit=True, workspace=None, stream=None):
    """Gradients of sum(dy * y) + <dfinal, final_state> for the forward of the
    same inputs (scalar decay, or per-state up to N = 128): returns dict dx,
    da, dBm, dCm, dD (or None), dinit (or None).  Shapes and dtypes as for
    forward(); dy like x; dfinal and initial_state [B,H,N,P] float32 or None.  Asynchronous on the current
    torch stream (or ``stream``)."""
    if stream is not None:
        return _on(stream, backward, x, a, Bm, Cm, D, dy, chunk, dfinal=dfinal, initial_state=initial_state,
                   want_dD=want_dD, want_dinit=want_dinit, workspace=workspace)
    _check_inputs(x, a, Bm, Cm, D)
    if dy.shape != x.shape or dy.dtype != x.dtype or not dy.is_contiguous():
        raise ValueError("dy must be a contiguous tensor of x's shape and dtype")
    B, T, H, P = x.shape
    N = Bm.shape[3]
    for name, t in (("dfinal", dfinal), ("initial_state", initial_state)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()
                              or tuple(t.shape) != (B, H, N, P)):
            raise ValueError(f"{name} must be a contiguous float32 [B,H,N,P] tensor")
    shape = shape_of(x, a, Bm, chunk)
    need = backward_workspace_size(shape)
    if need == 0:
        raise SSDError(SSD_ERR_UNSUPPORTED, "ssd_backward_workspace_size")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    out = {
        "dx": torch.empty_like(x), "da": torch.empty_like(a),
        "dBm": torch.empty_like(Bm), "dCm": torch.empty_like(Cm),
        "dD": torch.empty(H, dtype=torch.float32, device=x.device) if want_dD else None,
        "dinit": torch.empty((B, H, N, P), dtype=torch.float32, device=x.device) if want_dinit else None,
    }
    _check(load().ssd_backward(ctypes.byref(shape), _ptr(x), _ptr(a), _ptr(Bm), _ptr(Cm), _ptr(D),
                               _ptr(initial_state), _ptr(dy), _ptr(dfinal), _ptr(out["dx"]),
                               _ptr(out["da"]), _ptr(out["dBm"]), _ptr(out["dCm"]), _ptr(out["dD"]),
                               _ptr(out["dinit"]), _ptr(workspace), workspace.numel(), _stream(stream)),
           "ssd_backward")
    return out


# ---- linear attention with a decay for each head, and layer norm -------------
#
# These calls run on the device of their tensors, on its current torch stream
# unless another is given, whose order with the inputs is then the caller's.  A
# single token's step takes a few microseconds on the GPU, so the host's part is
# kept short: what follows from the tensors' shapes and strides alone is checked
# and laid out once for each combination of them.

def _on_device(name, t, device, dtype=None, shape=None, contiguous=True):
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_boundary(name, t, by):
    if t.data_ptr() % by:
        raise ValueError(f"{name} must start on a {by}-byte boundary")


def _aligned(t):
    """A tensor that is only read, on a 16-byte boundary: itself or a copy."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _dtype_code(dtype):
    if dtype == torch.bfloat16:
        return SSD_DTYPE_BF16
    if dtype == torch.float32:
        return SSD_DTYPE_F32
    raise ValueError("tensors must be float32 or bfloat16")


def _call(where, device, fn, *args):
    """fn(*args, device's current stream) with `device` current; raises SSDError."""
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code != SSD_OK:
        raise SSDError(code, where)


_PLANS_MOST = 4096
_plans = {}  # shapes, strides and types -> what is laid out for them


def _plan(key, make):
    plan = _plans.get(key)
    if plan is None:
        plan = make()
        if len(_plans) >= _PLANS_MOST:
            _plans.clear()
        _plans[key] = plan
    return plan


class _LinearPlan:
    """What the shapes and strides of q, k, v say."""

    def __init__(self, q, k, v, seqs, step):
        lead = 1 if step or seqs is not None else 2
        if q.dim() != lead + 2 or k.dim() != lead + 2 or v.dim() != lead + 2:
            raise ValueError(f"q, k, v must have {lead + 2} dimensions")
        dt = _dtype_code(q.dtype)
        for name, t in (("q", q), ("k", k), ("v", v)):
            if t.numel() == 0:
                raise ValueError(f"{name} is empty")
            if t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError(f"the last dimension of {name} must be contiguous")
        rows, H, K = tuple(q.shape[:lead]), q.shape[-2], q.shape[-1]
        G, V = k.shape[-2], v.shape[-1]
        if tuple(k.shape) != rows + (G, K) or tuple(v.shape) != rows + (G, V) or H % G:
            raise ValueError("k must be [..., G, K] and v [..., G, V] with q's leading dimensions and G dividing H")
        if seqs is not None:
            if len(seqs) != 1 or seqs[0] < 2:
                raise ValueError("cu_seqlens must be [sequences + 1]")
            B, T, packed = seqs[0] - 1, rows[0], 1
        else:
            B, T, packed = (rows[0], 1, 0) if step else (rows[0], rows[1], 0)
        self.keep = [LinearShape(B, T, H, G, K, V, dt, packed)]
        for t in (q, k, v):
            st = t.stride()
            self.keep.append(Strides(0 if packed else st[0], 0 if step else st[lead - 1], st[-2]))
        self.shape = self.keep[0]
        self.refs = [ctypes.byref(x) for x in self.keep]
        self.H, self.y, self.k, self.v = (H,), rows + (H, V), rows + (G, K), rows + (G, V)
        self.state = (B, H, K, V)
        self.scale = float(K) ** -0.5
        self.forward_bytes = linear_workspace_size(self.shape)
        self.backward_bytes = linear_backward_workspace_size(self.shape)
        if self.forward_bytes == 0:
            raise SSDError(SSD_ERR_INVALID_ARG, "ssd_linear_workspace_size")


def _linear_plan(q, k, v, decay, cu_seqlens, step=False):
    dev, dt = q.device, q.dtype
    seqs = None if cu_seqlens is None else cu_seqlens.shape
    plan = _plan((q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(), dt, seqs, step),
                 lambda: _LinearPlan(q, k, v, seqs, step))
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.device != dev or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor on {dev}")
        if t.dtype != dt:
            raise ValueError("q, k, v must share their type")
    _on_device("decay", decay, dev, torch.float32, plan.H)
    if cu_seqlens is not None:
        _on_device("cu_seqlens", cu_seqlens, dev, torch.int32)
    return plan


def _workspace_arg(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _on_device("workspace", workspace, device, torch.uint8)
    _on_boundary("workspace", workspace, 256)
    return workspace


def linear_workspace_size(shape: LinearShape) -> int:
    return int(load().ssd_linear_workspace_size(ctypes.byref(shape)))


def linear_backward_workspace_size(shape: LinearShape) -> int:
    return int(load().ssd_linear_backward_workspace_size(ctypes.byref(shape)))


def linear_attention(q, k, v, decay, *, scale=None, initial_state=None, cu_seqlens=None, y=None, final_state=None,
                     want_final=True, workspace=None, stream=None):
    """y and the final state of linear attention with a decay for each head:
    h_t = exp(decay[h]) h_{t-1} + k_t v_t^T, y_t = scale q_t^T h_t.

    q [B,T,H,K], k [B,T,G,K], v [B,T,G,V] (float32 or bfloat16; slices of one
    projection are taken as they are, only the last dimension has to be
    contiguous), decay [H] float32 log-decays, initial_state [B,H,K,V] float32
    or None (zero), scale (None: K**-0.5).  With cu_seqlens (int32 [S+1], on the device) the
    tensors are [T,heads,d] with S sequences one behind the other, the states
    [S,H,K,V]; rows of a given y outside every sequence stay as they are (those
    of a new y are not set).  A given y and final_state (which may be initial_state)
    start on 16-byte boundaries, other states are taken from anywhere.
    bfloat16 with K and V up to 128 and multiples of 8, and rows on 16-byte
    boundaries (no stride of 0), runs on tensor cores; other calls run on CUDA
    cores, some ten times slower.
    Returns y [B,T,H,V] and the state [B,H,K,V] float32 (None with
    want_final=False).  Asynchronous on the current stream of q's device; a kernel's
    wait that gave up leaves y undefined and says so in the workspace, if the caller
    gives one to ask (device_status)."""
    if stream is not None:
        return _on(stream, linear_attention, q, k, v, decay, scale=scale, initial_state=initial_state,
                   cu_seqlens=cu_seqlens, y=y, final_state=final_state, want_final=want_final, workspace=workspace)
    plan, dev = _linear_plan(q, k, v, decay, cu_seqlens), q.device
    if initial_state is not None:
        _on_device("initial_state", initial_state, dev, torch.float32, plan.state)
    if y is None:
        y = torch.empty(plan.y, dtype=q.dtype, device=dev)
    else:
        _on_device("y", y, dev, q.dtype, plan.y)
        _on_boundary("y", y, 16)
    if final_state is not None:
        _on_device("final_state", final_state, dev, torch.float32, plan.state)
        _on_boundary("final_state", final_state, 16)
    elif want_final:
        final_state = torch.empty(plan.state, dtype=torch.float32, device=dev)
    workspace = _workspace_arg(workspace, plan.forward_bytes, dev)
    initial_state = _aligned(initial_state)
    shape, sq, sk, sv = plan.refs
    _call("ssd_linear_attention", dev, load().ssd_linear_attention, shape, q.data_ptr(), sq, k.data_ptr(), sk,
          v.data_ptr(), sv, decay.data_ptr(), _ptr(cu_seqlens), _ptr(initial_state),
          plan.scale if scale is None else scale, y.data_ptr(), _ptr(final_state), workspace.data_ptr(),
          workspace.numel())
    return y, final_state


def linear_attention_step(q, k, v, decay, state, *, scale=None, y=None, stream=None):
    """One token of linear_attention() for a batch of sequences, in place on
    ``state`` [B,H,K,V] float32, on a 16-byte boundary: q [B,H,K], k [B,G,K],
    v [B,G,V], decay [H].
    Returns y [B,H,V]."""
    if stream is not None:
        return _on(stream, linear_attention_step, q, k, v, decay, state, scale=scale, y=y)
    plan, dev = _linear_plan(q, k, v, decay, None, True), q.device
    _on_device("state", state, dev, torch.float32, plan.state)
    _on_boundary("state", state, 16)
    if y is None:
        y = torch.empty(plan.y, dtype=q.dtype, device=dev)
    else:
        _on_device("y", y, dev, q.dtype, plan.y)
    shape, sq, sk, sv = plan.refs
    _call("ssd_linear_attention_step", dev, load().ssd_linear_attention_step, shape, q.data_ptr(), sq,
          k.data_ptr(), sk, v.data_ptr(), sv, decay.data_ptr(), plan.scale if scale is None else scale,
          state.data_ptr(), y.data_ptr())
    return y


def linear_attention_backward(q, k, v, decay, dy, *, scale=None, initial_state=None, dfinal=None, cu_seqlens=None,
                              want_dinit=True, workspace=None, stream=None):
    """Gradients of sum(dy * y) + <dfinal, final_state> of linear_attention()
    for the same inputs: a dict of dq, dk, dv (contiguous, in q's dtype; dk and
    dv summed over the query heads of their group) and dinit ([B,H,K,V]
    float32, or None).  dy like y; dfinal like the final state, or None.  The
    decay has no gradient.  Rows outside every packed sequence come back zero."""
    if stream is not None:
        return _on(stream, linear_attention_backward, q, k, v, decay, dy, scale=scale,
                   initial_state=initial_state, dfinal=dfinal, cu_seqlens=cu_seqlens, want_dinit=want_dinit,
                   workspace=workspace)
    plan, dev = _linear_plan(q, k, v, decay, cu_seqlens), q.device
    _on_device("dy", dy, dev, q.dtype, plan.y)
    for name, t in (("initial_state", initial_state), ("dfinal", dfinal)):
        if t is not None:
            _on_device(name, t, dev, torch.float32, plan.state)
    new = torch.empty if cu_seqlens is None else torch.zeros
    dq, dk, dv = (new(d, dtype=q.dtype, device=dev) for d in (q.shape, plan.k, plan.v))
    dinit = torch.empty(plan.state, dtype=torch.float32, device=dev) if want_dinit else None
    workspace = _workspace_arg(workspace, plan.backward_bytes, dev)
    dy, initial_state, dfinal = _aligned(dy), _aligned(initial_state), _aligned(dfinal)
    shape, sq, sk, sv = plan.refs
    _call("ssd_linear_attention_backward", dev, load().ssd_linear_attention_backward, shape, q.data_ptr(), sq,
          k.data_ptr(), sk, v.data_ptr(), sv, decay.data_ptr(), _ptr(cu_seqlens), _ptr(initial_state),
          plan.scale if scale is None else scale, dy.data_ptr(), _ptr(dfinal), dq.data_ptr(), dk.data_ptr(),
          dv.data_ptr(), _ptr(dinit), workspace.data_ptr(), workspace.numel())
    return {"dq": dq, "dk": dk, "dv": dv, "dinit": dinit}


def _row_stride(name, t):
    """Elements from row to row of t, whose leading dimensions must flatten to rows."""
    if t.dim() == 0 or t.numel() == 0:
        raise ValueError(f"{name} is empty")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    stride = want = None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if want is None:
            stride = s
        elif s != want:
            raise ValueError(f"the leading dimensions of {name} must flatten to rows")
        want = s * n
    return t.shape[-1] if stride is None else stride


class _NormPlan:
    """What the shapes and strides of x (gate, dy) say."""

    def __init__(self, x, groups, gate, dy):
        self.x_stride = _row_stride("x", x)
        for name, t in (("gate", gate), ("dy", dy)):
            if t is not None and t.shape != x.shape:
                raise ValueError(f"{name} must have x's shape and dtype")
        self.gate_stride = 0 if gate is None else _row_stride("gate", gate)
        self.dy_stride = 0 if dy is None else _row_stride("dy", dy)
        width = x.shape[-1]
        if groups < 1 or width % groups:
            raise ValueError("groups must divide x's last dimension")
        self.keep = NormShape(x.numel() // width, width, groups, _dtype_code(x.dtype))
        self.shape = ctypes.byref(self.keep)
        self.width = (width,)
        self.stats = (x.numel() // width, groups, 2)
        self.sums_bytes = int(load().ssd_layer_norm_backward_workspace_size(self.shape))


def _norm_plan(x, weight, bias, groups, gate, dy=None):
    dev, dt = x.device, x.dtype
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    for name, t in (("gate", gate), ("dy", dy)):
        if t is not None:
            if t.device != dev:
                raise ValueError(f"{name} must be a CUDA tensor on {dev}")
            if t.dtype != dt:
                raise ValueError(f"{name} must have x's shape and dtype")
    lay = lambda t: None if t is None else (t.shape, t.stride())  # noqa: E731
    groups = int(groups)
    plan = _plan((x.shape, x.stride(), dt, groups, lay(gate), lay(dy)), lambda: _NormPlan(x, groups, gate, dy))
    if weight is not None:
        _on_device("weight", weight, dev, torch.float32, plan.width)
    if bias is not None:
        _on_device("bias", bias, dev, torch.float32, plan.width)
    return plan


def layer_norm(x, weight=None, bias=None, *, groups=1, gate=None, eps=1e-5, y=None, stream=None):
    """Layer norm over each of the ``groups`` equal parts of x's last dimension
    (groups = heads: the norm behind a sequence mixer), times silu(gate):
    y = ((x - mean) rstd weight + bias) silu(gate).

    x [..., D] float32 or bfloat16 (leading dimensions that flatten to rows,
    the last contiguous), gate the same or None, weight and bias [D] float32 or
    None.  Returns y and stats [rows, groups, 2] float32 (mean and rstd, for
    layer_norm_backward)."""
    if stream is not None:
        return _on(stream, layer_norm, x, weight, bias, groups=groups, gate=gate, eps=eps, y=y)
    plan, dev = _norm_plan(x, weight, bias, groups, gate), x.device
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _on_device("y", y, dev, x.dtype, x.shape)
    stats = torch.empty(plan.stats, dtype=torch.float32, device=dev)
    _call("ssd_layer_norm", dev, load().ssd_layer_norm, plan.shape, x.data_ptr(), plan.x_stride, _ptr(weight),
          _ptr(bias), _ptr(gate), plan.gate_stride, eps, y.data_ptr(), stats.data_ptr())
    return y, stats


def layer_norm_backward(x, weight, bias, dy, stats, *, groups=1, gate=None, want_dweight=True, want_dbias=True,
                        workspace=None, stream=None):
    """Gradients of sum(dy * y) of layer_norm() for the same inputs and its
    stats: a dict of dx, dgate (None without a gate), dweight and dbias ([D]
    float32, or None)."""
    if stream is not None:
        return _on(stream, layer_norm_backward, x, weight, bias, dy, stats, groups=groups, gate=gate,
                   want_dweight=want_dweight, want_dbias=want_dbias, workspace=workspace)
    plan, dev = _norm_plan(x, weight, bias, groups, gate, dy), x.device
    _on_device("stats", stats, dev, torch.float32, plan.stats)
    _on_boundary("stats", stats, 8)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dgate = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    dweight = torch.empty(plan.width, dtype=torch.float32, device=dev) if want_dweight else None
    dbias = torch.empty(plan.width, dtype=torch.float32, device=dev) if want_dbias else None
    if want_dweight or want_dbias:
        workspace = _workspace_arg(workspace, plan.sums_bytes, dev)
    _call("ssd_layer_norm_backward", dev, load().ssd_layer_norm_backward, plan.shape, x.data_ptr(),
          plan.x_stride, _ptr(weight), _ptr(bias), _ptr(gate), plan.gate_stride, dy.data_ptr(), plan.dy_stride,
          stats.data_ptr(), dx.data_ptr(), _ptr(dweight), _ptr(dbias), _ptr(dgate), _ptr(workspace),
          0 if workspace is None else workspace.numel())
    return {"dx": dx, "dgate": dgate, "dweight": dweight, "dbias": dbias}
