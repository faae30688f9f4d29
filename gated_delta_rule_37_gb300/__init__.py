"""GB300 (sm_103a) gated delta rule forward: thin Python binding of libgdr.so.

Every step of the computation runs in the library's CUDA kernels; this module
only marshals torch tensors (device memory, streams) into the C ABI declared in
``include/gdr.h`` and raises on a non-zero status.  There is no CPU fallback:
if ``libgdr.so`` is missing or no CUDA device is present, calls fail loudly.
Nothing is recorded for automatic differentiation: outputs carry no gradient
function, whatever the inputs require; gradients come from the ``*_bwd`` calls.

Entry points (same names as the C ABI, without the ``gdr_`` prefix):
  chunk_fwd           chunked prefill          -> o, final_state
  recurrent_fwd       slot-indexed decode / verify (pool in place, ibuf)
  gating_fwd          g, beta from raw projections
  chunk_workspace_size
  linrec_fwd          gated linear recurrence over packed sequences -> y, final_state
  linrec_bwd          its gradients                       -> dx, dg, d_initial_state
  linrec_step         the same over a slot-indexed state pool (decode / verify) -> y
  rmsnorm_fwd         RMS norm with the residual's addition, in the input's type or
                      e4m3 with scales                    -> y, residual_out, scales
  rmsnorm_bwd         its gradients                       -> dx, dweight
  linrec_workspace_size, rmsnorm_bwd_workspace_size
  kv_append           new keys and values into a paged cache, rotary positions
                      applied on the way                  -> q_out, k_out
  attn_fwd            causal softmax attention over packed prompts -> o
  attn_step           attention of a few tokens per sequence over the paged cache,
                      a shared prefix read once for the batch      -> o
  attn_step_workspace_size
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr.so")

GDR_BF16, GDR_F32, GDR_E4M3 = 0, 1, 2
GDR_GATE_SCALAR, GDR_GATE_CHANNEL = 0, 1
GDR_QK_L2NORM, GDR_NEG_EIGVAL, GDR_COMMIT, GDR_VALIDATE, GDR_CHANNEL_GATE = 0x1, 0x2, 0x4, 0x8, 0x10
GDR_CHUNK_SCAN, GDR_ROPE_PAIRS = 0x20, 0x40
CHUNK = 64

STATUS = {0: "GDR_OK", 1: "GDR_ERR_INVALID_ARG", 2: "GDR_ERR_UNSUPPORTED", 3: "GDR_ERR_WORKSPACE",
          4: "GDR_ERR_LAUNCH", 5: "GDR_ERR_DEVICE_TIMEOUT", 6: "GDR_ERR_VALIDATION"}

# every symbol include/gdr.h declares
EXPORTED = ("gdr_chunk_workspace_size", "gdr_chunk_fwd", "gdr_chunk_fwd_noalloc", "gdr_recurrent_fwd",
            "gdr_recurrent_fwd_gated", "gdr_recurrent_fwd_norm", "gdr_gating_fwd",
            "gdr_linrec_workspace_size", "gdr_linrec_fwd", "gdr_linrec_bwd", "gdr_linrec_step",
            "gdr_rmsnorm_fwd", "gdr_rmsnorm_bwd_workspace_size", "gdr_rmsnorm_bwd",
            "gdr_kv_append", "gdr_attn_fwd", "gdr_attn_step_workspace_size", "gdr_attn_step",
            "gdr_last_error", "gdr_get_device_status", "gdr_selftest_bounded_wait", "gdr_selftest_linrec_lost_copy",
            "gdr_selftest_rmsnorm_lost_copy", "gdr_profile_enable", "gdr_profile_read", "gdr_version")

_lib = None


class GdrError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


def load(path: str | None = None):
    """Load libgdr.so (built in-tree by ``build.build()``); raises if missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libgdr.so not found at {p}: build it with gated_delta_rule_37_gb300.build.build()")
    lib = ctypes.CDLL(p)
    P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.gdr_chunk_workspace_size.argtypes = [I, I64, I, I, I, I, I, I, I, ctypes.POINTER(SZ)]
    lib.gdr_chunk_workspace_size.restype = I
    lib.gdr_chunk_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I64, I, I, I, I, F, I, I, P, P, P, SZ, P]
    lib.gdr_chunk_fwd.restype = I
    lib.gdr_chunk_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, I, I64, I, I, I, I, F, I, I, P, P, P]
    lib.gdr_chunk_fwd_noalloc.restype = I
    lib.gdr_recurrent_fwd.argtypes = [P, P, P, P, P, P, I, I, P, P, I, I64, I, I, I, I, F, I, I, P, P, I, P]
    lib.gdr_recurrent_fwd.restype = I
    lib.gdr_recurrent_fwd_gated.argtypes = [P, P, P, P, P, P, P, P, I, I, P, P, I, I64, I, I, I, I, F, I, I, P, P, I, P]
    lib.gdr_recurrent_fwd_gated.restype = I
    lib.gdr_recurrent_fwd_norm.argtypes = [P, P, P, P, P, P, I, I, P, P, I, I64, I, I, I, I, F, I, I, P, P, F, P, P, I,
                                           P]
    lib.gdr_recurrent_fwd_norm.restype = I
    lib.gdr_gating_fwd.argtypes = [P, P, P, P, I64, I, I, I, P, P, P]
    lib.gdr_gating_fwd.restype = I
    lib.gdr_linrec_workspace_size.argtypes = [I, I64, I, I, I, ctypes.POINTER(SZ)]
    lib.gdr_linrec_workspace_size.restype = I
    lib.gdr_linrec_fwd.argtypes = [P, I64, P, I64, P, P, I, I64, I, I, I, I, P, I64, P, P, SZ, P]
    lib.gdr_linrec_fwd.restype = I
    lib.gdr_linrec_bwd.argtypes = [P, I64, P, I64, P, I64, P, P, P, I, I64, I, I, I, I, P, I64, P, I64, P, P, SZ, P]
    lib.gdr_linrec_bwd.restype = I
    lib.gdr_linrec_step.argtypes = [P, I64, P, I64, P, I, I, P, P, I, I64, I, I, I, I, P, I64, P, I, P]
    lib.gdr_linrec_step.restype = I
    lib.gdr_rmsnorm_fwd.argtypes = [P, I64, P, I64, P, I64, I, F, I, P, I64, P, I64, I, P, I, P]
    lib.gdr_rmsnorm_fwd.restype = I
    lib.gdr_rmsnorm_bwd_workspace_size.argtypes = [I64, I, ctypes.POINTER(SZ)]
    lib.gdr_rmsnorm_bwd_workspace_size.restype = I
    lib.gdr_rmsnorm_bwd.argtypes = [P, I64, P, I64, P, P, I64, I64, I, F, I, P, I64, P, P, SZ, P]
    lib.gdr_rmsnorm_bwd.restype = I
    lib.gdr_kv_append.argtypes = [P, I64, P, I64, P, I64, P, I, P, P, I64, I, P, I, I64, I, I, I, I, I, P, I64, P, I64,
                                  P, P, I, I, P]
    lib.gdr_kv_append.restype = I
    lib.gdr_attn_fwd.argtypes = [P, I64, P, I64, P, I64, P, I, I64, I, I, I, F, I, I, P, I64, P]
    lib.gdr_attn_fwd.restype = I
    lib.gdr_attn_step_workspace_size.argtypes = [I, I64, I, I, I, I, I, ctypes.POINTER(SZ)]
    lib.gdr_attn_step_workspace_size.restype = I
    lib.gdr_attn_step.argtypes = [P, I64, P, P, I, I, P, I64, I, P, P, I, P, I, I64, I, I, I, F, I, I, P, I64, P, SZ, P]
    lib.gdr_attn_step.restype = I
    lib.gdr_last_error.argtypes = []
    lib.gdr_last_error.restype = ctypes.c_char_p
    lib.gdr_get_device_status.argtypes = [P, ctypes.POINTER(I)]
    lib.gdr_get_device_status.restype = I
    lib.gdr_selftest_bounded_wait.argtypes = [P]
    lib.gdr_selftest_bounded_wait.restype = I
    lib.gdr_selftest_linrec_lost_copy.argtypes = [P, P, P, I, I64, I, I, P, P, P, SZ, P]
    lib.gdr_selftest_linrec_lost_copy.restype = I
    lib.gdr_selftest_rmsnorm_lost_copy.argtypes = [P, P, P, I64, I, I64, P, P, P, SZ, P]
    lib.gdr_selftest_rmsnorm_lost_copy.restype = I
    lib.gdr_profile_enable.argtypes = [I]
    lib.gdr_profile_enable.restype = I
    lib.gdr_profile_read.argtypes = [I, ctypes.c_char_p, SZ, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(I), ctypes.POINTER(I)]
    lib.gdr_profile_read.restype = I
    lib.gdr_version.argtypes = []
    lib.gdr_version.restype = I
    if path is None:
        _lib = lib
    return lib


def _check(code: int):
    if code != 0:
        raise GdrError(code, load().gdr_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    if t.dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libgdr must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libgdr must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def chunk_workspace_size(N: int, T: int, Hk: int, Hv: int, K: int, V: int, *, gate_kind: int,
                         dtype: int, flags: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(load().gdr_chunk_workspace_size(N, T, Hk, Hv, K, V, gate_kind, dtype, flags, ctypes.byref(out)))
    return out.value


def chunk_fwd(q, k, v, beta, cu_seqlens, *, g=None, gk=None, initial_state=None, scale=None,
              flags: int = 0, o=None, final_state=None, output_final_state: bool = True,
              workspace=None, stream=None):
    """Chunked prefill.  q,k [T,Hk,K]; v [T,Hv,V]; g [T,Hv] fp32 or gk [T,Hv,K]
    fp32; beta [T,Hv]; initial_state [N,Hv,V,K] fp32 or None; cu_seqlens [N+1]
    int32 (device).  Returns (o, final_state or None)."""
    T, Hk, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty(T, Hv, V, dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, Hv, V, K, dtype=torch.float32, device=q.device)
    gate_kind = GDR_GATE_SCALAR if g is not None else GDR_GATE_CHANNEL
    need = chunk_workspace_size(N, T, Hk, Hv, K, V, gate_kind=gate_kind, dtype=dt, flags=flags)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(load().gdr_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(gk), _ptr(beta),
                                _ptr(initial_state), _ptr(cu_seqlens), N, T, Hk, Hv, K, V,
                                float(scale), dt, flags, _ptr(o), _ptr(final_state),
                                _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, final_state


NOALLOC_WORKSPACE_BYTES = 64 << 20


def chunk_fwd_noalloc(q, k, v, beta, cu_seqlens, *, g=None, gk=None, initial_state=None, scale=None,
                      flags: int = 0, o, final_state=None, stream=None):
    """Chunked prefill through gdr_chunk_fwd_noalloc: no workspace argument and
    no device allocation inside the call (the library's fixed scratch array of
    NOALLOC_WORKSPACE_BYTES is used).  For callers that cannot allocate device
    memory; they pass preallocated outputs ``o`` (and ``final_state``).  Calls
    that overlap on the GPU share the scratch and must be serialised."""
    T, Hk, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    _check(load().gdr_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(gk), _ptr(beta),
                                        _ptr(initial_state), _ptr(cu_seqlens), N, T, Hk, Hv, K, V,
                                        float(scale), _dtype_code(q), flags, _ptr(o), _ptr(final_state),
                                        _stream(stream)))
    return o, final_state


def recurrent_fwd(q, k, v, g, beta, state_pool, state_indices, cu_seqlens, *, scale=None,
                  flags: int = GDR_COMMIT, o=None, intermediate_states=None, stream=None):
    """Slot-indexed decode / verify.  ``g`` is the scalar log-decay [T, Hv] or
    the per-key-channel one [T, Hv, K] (sets GDR_CHANNEL_GATE).  The pool is
    updated in place only with GDR_COMMIT; ``intermediate_states`` [rows, steps,
    Hv, V, K] (pool dtype) receives per-token states.  Returns o."""
    T, Hk, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    N = cu_seqlens.numel() - 1
    if g.dim() == 3:
        if tuple(g.shape) != (T, Hv, K):
            raise ValueError("a per-channel gate must be [T, Hv, K]")
        flags |= GDR_CHANNEL_GATE
    if scale is None:
        scale = K ** -0.5
    if o is None:
        o = torch.empty(T, Hv, V, dtype=q.dtype, device=q.device)
    steps = 0
    if intermediate_states is not None:
        if intermediate_states.dim() != 5 or intermediate_states.shape[0] < N:
            raise ValueError("intermediate_states must be [rows >= N, steps, Hv, V, K]")
        if intermediate_states.dtype != state_pool.dtype:
            raise TypeError("intermediate_states must have the pool dtype")
        steps = intermediate_states.shape[1]
    _check(load().gdr_recurrent_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
                                    _dtype_code(state_pool), state_pool.shape[0], _ptr(state_indices),
                                    _ptr(cu_seqlens), N, T, Hk, Hv, K, V, float(scale), _dtype_code(q),
                                    flags, _ptr(o), _ptr(intermediate_states), steps, _stream(stream)))
    return o


def recurrent_fwd_norm(q, k, v, g, beta, state_pool, state_indices, cu_seqlens, norm_weight, norm_gate, *,
                       eps: float = 1e-6, scale=None, flags: int = GDR_COMMIT, o=None, intermediate_states=None,
                       stream=None):
    """recurrent_fwd with the gated RMSNorm output epilogue: each value row x of
    o becomes x / sqrt(mean(x^2) + eps) * norm_weight * sigmoid(norm_gate).
    norm_weight [V] fp32; norm_gate [T, Hv, V] (q's dtype).  Returns o."""
    T, Hk, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    if g.dim() == 3:
        flags |= GDR_CHANNEL_GATE
    if o is None:
        o = torch.empty(T, Hv, V, dtype=q.dtype, device=q.device)
    steps = 0
    if intermediate_states is not None:
        steps = intermediate_states.shape[1]
    if norm_gate.dtype != q.dtype or tuple(norm_gate.shape) != (T, Hv, V):
        raise ValueError("norm_gate must be [T, Hv, V] in q's dtype")
    _check(load().gdr_recurrent_fwd_norm(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
                                         _dtype_code(state_pool), state_pool.shape[0], _ptr(state_indices),
                                         _ptr(cu_seqlens), N, T, Hk, Hv, K, V, float(scale), _dtype_code(q), flags,
                                         _ptr(norm_weight), _ptr(norm_gate), float(eps), _ptr(o),
                                         _ptr(intermediate_states), steps, _stream(stream)))
    return o


def recurrent_fwd_gated(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, cu_seqlens, *, scale=None,
                        flags: int = GDR_COMMIT, o=None, intermediate_states=None, stream=None):
    """recurrent_fwd with the gates formed in the kernel from the raw
    projections: g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b) (x2
    with GDR_NEG_EIGVAL).  a, b [T, Hv] (q's dtype); A_log, dt_bias [Hv] fp32.
    Returns o."""
    T, Hk, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    N = cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    if o is None:
        o = torch.empty(T, Hv, V, dtype=q.dtype, device=q.device)
    steps = 0
    if intermediate_states is not None:
        if intermediate_states.dim() != 5 or intermediate_states.shape[0] < N:
            raise ValueError("intermediate_states must be [rows >= N, steps, Hv, V, K]")
        if intermediate_states.dtype != state_pool.dtype:
            raise TypeError("intermediate_states must have the pool dtype")
        steps = intermediate_states.shape[1]
    if a.dtype != q.dtype or b.dtype != q.dtype:
        raise TypeError("a and b must have q's dtype")
    _check(load().gdr_recurrent_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                          _ptr(state_pool), _dtype_code(state_pool), state_pool.shape[0],
                                          _ptr(state_indices), _ptr(cu_seqlens), N, T, Hk, Hv, K, V, float(scale),
                                          _dtype_code(q), flags, _ptr(o), _ptr(intermediate_states), steps,
                                          _stream(stream)))
    return o


def gating_fwd(a, dt_bias, A_log, b, *, flags: int = 0, g=None, beta=None, stream=None):
    """g = -exp(A_log) softplus(a + dt_bias) (fp32), beta = sigmoid(b) (x2 with
    GDR_NEG_EIGVAL).  a, b [T, Hv]; dt_bias, A_log [Hv] fp32."""
    T, Hv = a.shape
    if g is None:
        g = torch.empty(T, Hv, dtype=torch.float32, device=a.device)
    if beta is None:
        beta = torch.empty(T, Hv, dtype=a.dtype, device=a.device)
    _check(load().gdr_gating_fwd(_ptr(a), _ptr(dt_bias), _ptr(A_log), _ptr(b), T, Hv, _dtype_code(a),
                                 flags, _ptr(g), _ptr(beta), _stream(stream)))
    return g, beta


# ---- gated linear recurrence and RMS norm -----------------------------------
#
# Rows are 2-D tensors whose last axis is dense; their row stride is free (a
# column block of a wider matrix, an expanded row).  Everything runs on the
# tensors' device; `stream` defaults to that device's current stream, and what
# a call allocates belongs to the stream it runs on.  What a call costs on the
# host is the latency of a decode step: every tensor is checked once, and the
# current stream is asked for its handle without making a Stream object.

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_CODES = {torch.bfloat16: GDR_BF16, torch.float32: GDR_F32}

_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(t, shape, dtype, device, what):
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    raise ValueError(f"{what} must be on {device}, not {t.device}")


def _dense(t, shape, dtype, device, what):
    """Address of a dense tensor of this shape, dtype and device."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _refuse(t, shape, dtype, device, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, shape, dtype, device, what):
    """(address, row stride) of a [rows, D] tensor with a dense last axis."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _refuse(t, shape, dtype, device, what)
    row, col = t.stride()
    rows, D = shape
    if col != 1 and D > 1:
        raise ValueError(f"{what} must be dense along its last axis")
    return t.data_ptr(), row if rows > 1 else D


def _like(t, shape, dtype, device):
    """(tensor, address, row stride) of a new dense [rows, D] tensor; `t` has its shape."""
    if t.dtype is dtype:
        new = torch.empty_like(t)  # costs less than empty(); laid out as t where that is dense
        if new.is_contiguous():
            return new, new.data_ptr(), shape[1]
    new = torch.empty(shape, dtype=dtype, device=device)
    return new, new.data_ptr(), shape[1]


def _not_a_code(*dtypes):
    bad = next(d for d in dtypes if d not in _CODES)
    raise TypeError(f"unsupported dtype {bad} (bf16 or fp32)")


def _elsewhere(t, what, stream):
    """The context to enter first where a call does not run on the current
    device's current stream; refuses tensors that no call takes."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def _scratch(workspace, size, device):
    """(tensor, address, bytes) of the given workspace, or of a new one of `size` bytes."""
    if workspace is None:
        if size == 0:
            return None, None, 0
        workspace = torch.empty(size, dtype=_U8, device=device)
    elif workspace.device != device or workspace.dtype != _U8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a dense uint8 tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel()


@functools.lru_cache(maxsize=4096)
def _linrec_bytes(N, T, D, dtype, gate_dtype):
    out = ctypes.c_size_t(0)
    _check(load().gdr_linrec_workspace_size(N, T, D, dtype, gate_dtype, ctypes.byref(out)))
    return out.value


def linrec_workspace_size(N: int, T: int, D: int, *, dtype: int, gate_dtype: int) -> int:
    return _linrec_bytes(N, T, D, dtype, gate_dtype)


def linrec_fwd(x, g, cu_seqlens, *, initial_state=None, flags: int = 0, y=None, final_state=None,
               output_final_state: bool = True, workspace=None, stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over packed
    sequences.  x [T, D] bf16 or fp32; g [T, D] bf16 or fp32, <= 0; cu_seqlens
    [N+1] int32; initial_state [N, D] fp32 or None.  Rows from cu_seqlens[N] on
    are neither read nor written.  Returns (y, final_state or None)."""
    if stream is not None or not x.is_cuda or x.get_device() != _current_device() or x.dim() != 2:
        with _elsewhere(x, "x", stream):
            return linrec_fwd(x, g, cu_seqlens, initial_state=initial_state, flags=flags, y=y, final_state=final_state,
                              output_final_state=output_final_state, workspace=workspace)
    dev, shape, xt, gt = x.device, x.shape, x.dtype, g.dtype
    T, D = shape
    xc, gc = _CODES.get(xt), _CODES.get(gt)
    if xc is None or gc is None:
        _not_a_code(xt, gt)
    N = cu_seqlens.numel() - 1
    state = (N, D)
    xp, xs = _rows(x, shape, xt, dev, "x")
    gp, gs = _rows(g, shape, gt, dev, "g")
    hp = _dense(initial_state, state, _F32, dev, "initial_state")
    cp = _dense(cu_seqlens, (N + 1,), _I32, dev, "cu_seqlens")
    if y is None:
        y, yp, ys = _like(x, shape, xt, dev)
    else:
        yp, ys = _rows(y, shape, xt, dev, "y")
    if final_state is not None or not output_final_state:
        fp = _dense(final_state, state, _F32, dev, "final_state")
    else:
        final_state = torch.empty(N, D, dtype=_F32, device=dev) if hp is None else torch.empty_like(initial_state)
        fp = final_state.data_ptr()
    ws, wp, wn = _scratch(workspace, _linrec_bytes(N, T, D, xc, gc), dev)
    code = (_lib or load()).gdr_linrec_fwd(xp, xs, gp, gs, hp, cp, N, T, D, xc, gc, flags, yp, ys, fp, wp, wn,
                                           _current_handle(dev.index))
    if code:
        _check(code)
    return y, final_state


def linrec_bwd(dy, g, y, cu_seqlens, *, initial_state=None, d_final_state=None, flags: int = 0, dx=None, dg=None,
               d_initial_state=None, output_d_initial_state: bool = True, workspace=None, stream=None):
    """Gradients of linrec_fwd: dy [T, D] is the gradient of y, d_final_state
    [N, D] fp32 (or None) that of the final state; g, y, initial_state are the
    forward's.  Returns (dx, dg, d_initial_state or None)."""
    if stream is not None or not dy.is_cuda or dy.get_device() != _current_device() or dy.dim() != 2:
        with _elsewhere(dy, "dy", stream):
            return linrec_bwd(dy, g, y, cu_seqlens, initial_state=initial_state, d_final_state=d_final_state,
                              flags=flags, dx=dx, dg=dg, d_initial_state=d_initial_state,
                              output_d_initial_state=output_d_initial_state, workspace=workspace)
    dev, shape, xt, gt = dy.device, dy.shape, dy.dtype, g.dtype
    T, D = shape
    xc, gc = _CODES.get(xt), _CODES.get(gt)
    if xc is None or gc is None:
        _not_a_code(xt, gt)
    N = cu_seqlens.numel() - 1
    state = (N, D)
    dp, ds = _rows(dy, shape, xt, dev, "dy")
    gp, gs = _rows(g, shape, gt, dev, "g")
    yp, ys = _rows(y, shape, xt, dev, "y")
    hp = _dense(initial_state, state, _F32, dev, "initial_state")
    fp = _dense(d_final_state, state, _F32, dev, "d_final_state")
    cp = _dense(cu_seqlens, (N + 1,), _I32, dev, "cu_seqlens")
    if dx is None:
        dx, xp, xs = _like(dy, shape, xt, dev)
    else:
        xp, xs = _rows(dx, shape, xt, dev, "dx")
    if dg is None:
        dg, ap, as_ = _like(g, shape, gt, dev)
    else:
        ap, as_ = _rows(dg, shape, gt, dev, "dg")
    if d_initial_state is not None or not output_d_initial_state:
        ip = _dense(d_initial_state, state, _F32, dev, "d_initial_state")
    else:
        d_initial_state = torch.empty(N, D, dtype=_F32, device=dev) if hp is None else torch.empty_like(initial_state)
        ip = d_initial_state.data_ptr()
    ws, wp, wn = _scratch(workspace, _linrec_bytes(N, T, D, xc, gc), dev)
    code = (_lib or load()).gdr_linrec_bwd(dp, ds, gp, gs, yp, ys, hp, fp, cp, N, T, D, xc, gc, flags, xp, xs, ap, as_,
                                           ip, wp, wn, _current_handle(dev.index))
    if code:
        _check(code)
    return dx, dg, d_initial_state


def linrec_step(x, g, state_pool, state_indices, cu_seqlens, *, flags: int = GDR_COMMIT, y=None,
                intermediate_states=None, stream=None):
    """The recurrence over a few tokens per sequence from state_pool [slots, D]
    (fp32 or bf16) at state_indices [N] int32 (< 0: skipped).  The pool is
    updated in place only with GDR_COMMIT; intermediate_states [rows >= N,
    steps, D] (pool dtype) receives the state after every token.  Returns y."""
    if stream is not None or not x.is_cuda or x.get_device() != _current_device() or x.dim() != 2:
        with _elsewhere(x, "x", stream):
            return linrec_step(x, g, state_pool, state_indices, cu_seqlens, flags=flags, y=y,
                               intermediate_states=intermediate_states)
    dev, shape, xt, gt, pt = x.device, x.shape, x.dtype, g.dtype, state_pool.dtype
    T, D = shape
    xc, gc, pc = _CODES.get(xt), _CODES.get(gt), _CODES.get(pt)
    if xc is None or gc is None or pc is None:
        _not_a_code(xt, gt, pt)
    N = cu_seqlens.numel() - 1
    slots = state_pool.shape[0]
    xp, xs = _rows(x, shape, xt, dev, "x")
    gp, gs = _rows(g, shape, gt, dev, "g")
    pp = _dense(state_pool, (slots, D), pt, dev, "state_pool")
    ip = _dense(state_indices, (N,), _I32, dev, "state_indices")
    cp = _dense(cu_seqlens, (N + 1,), _I32, dev, "cu_seqlens")
    steps, bp = 0, None
    if intermediate_states is not None:
        if intermediate_states.dim() != 3 or intermediate_states.shape[0] < N:
            raise ValueError("intermediate_states must be [rows >= N, steps, D]")
        rows, steps = intermediate_states.shape[:2]
        bp = _dense(intermediate_states, (rows, steps, D), pt, dev, "intermediate_states")
    if y is None:
        y, yp, ys = _like(x, shape, xt, dev)
    else:
        yp, ys = _rows(y, shape, xt, dev, "y")
    code = (_lib or load()).gdr_linrec_step(xp, xs, gp, gs, pp, pc, slots, ip, cp, N, T, D, xc, gc, flags, yp, ys, bp,
                                            steps, _current_handle(dev.index))
    if code:
        _check(code)
    return y


def rmsnorm_fwd(x, weight, *, residual=None, eps: float = 1e-6, y_dtype=None, scale_group: int = 0, y=None,
                residual_out=None, scales=None, stream=None):
    """s = x + residual (rounded to x's dtype; x without a residual), y = s /
    sqrt(mean(s^2) + eps) * weight per row of x [M, D] (bf16 or fp32); weight
    [D] fp32.  y_dtype None: y in x's dtype; torch.float8_e4m3fn: codes, with
    one fp32 scale per scale_group (32, 64, 128; 0: the row) elements of a row.
    residual_out may be residual (or x) itself.  Returns (y, residual_out or
    None, scales or None)."""
    if stream is not None or not x.is_cuda or x.get_device() != _current_device() or x.dim() != 2:
        with _elsewhere(x, "x", stream):
            return rmsnorm_fwd(x, weight, residual=residual, eps=eps, y_dtype=y_dtype, scale_group=scale_group, y=y,
                               residual_out=residual_out, scales=scales)
    dev, shape, xt = x.device, x.shape, x.dtype
    M, D = shape
    xc = _CODES.get(xt)
    if xc is None:
        _not_a_code(xt)
    if y_dtype is None:
        y_dtype = xt if y is None else y.dtype
    xp, xs = _rows(x, shape, xt, dev, "x")
    wp = _dense(weight, (D,), _F32, dev, "weight")
    sp = None
    if y_dtype is torch.float8_e4m3fn:
        yc = GDR_E4M3
        groups = -(-D // scale_group) if scale_group > 0 else 1
        if scales is None:
            scales = torch.empty(M, groups, dtype=_F32, device=dev)
            sp = scales.data_ptr()
        else:
            sp = _dense(scales, (M, groups), _F32, dev, "scales")
    else:
        yc = _CODES.get(y_dtype, -1)
        if scales is not None:
            raise ValueError("scales go with y_dtype torch.float8_e4m3fn only")
    if y is None:
        y, yp, ys = _like(x, shape, y_dtype, dev)
    else:
        yp, ys = _rows(y, shape, y_dtype, dev, "y")
    if residual is not None:
        rp, rs = _rows(residual, shape, xt, dev, "residual")
        if residual_out is None:
            residual_out, op, os_ = _like(x, shape, xt, dev)
        else:
            op, os_ = _rows(residual_out, shape, xt, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    else:
        rp, rs, op, os_ = None, 0, None, 0
    code = (_lib or load()).gdr_rmsnorm_fwd(xp, xs, rp, rs, wp, M, D, eps, xc, op, os_, yp, ys, yc, sp, scale_group,
                                            _current_handle(dev.index))
    if code:
        _check(code)
    return y, residual_out, scales


@functools.lru_cache(maxsize=4096)
def rmsnorm_bwd_workspace_size(M: int, D: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().gdr_rmsnorm_bwd_workspace_size(M, D, ctypes.byref(out)))
    return out.value


def rmsnorm_bwd(dy, s, weight, *, eps: float = 1e-6, d_residual_out=None, dx=None, dweight=None,
                output_dweight: bool = True, workspace=None, stream=None):
    """Gradients of rmsnorm_fwd from dy [M, D]; s [M, D] is the forward's
    residual_out (x without a residual), d_residual_out the gradient arriving
    at s along the residual stream.  Returns (dx, dweight): dx is the gradient
    of x and of residual alike, dweight [D] fp32."""
    if stream is not None or not dy.is_cuda or dy.get_device() != _current_device() or dy.dim() != 2:
        with _elsewhere(dy, "dy", stream):
            return rmsnorm_bwd(dy, s, weight, eps=eps, d_residual_out=d_residual_out, dx=dx, dweight=dweight,
                               output_dweight=output_dweight, workspace=workspace)
    dev, shape, xt = dy.device, dy.shape, dy.dtype
    M, D = shape
    xc = _CODES.get(xt)
    if xc is None:
        _not_a_code(xt)
    dp, ds = _rows(dy, shape, xt, dev, "dy")
    sp, ss = _rows(s, shape, xt, dev, "s")
    wp = _dense(weight, (D,), _F32, dev, "weight")
    rp, rs = (None, 0) if d_residual_out is None else _rows(d_residual_out, shape, xt, dev, "d_residual_out")
    if dx is None:
        dx, xp, xs = _like(dy, shape, xt, dev)
    else:
        xp, xs = _rows(dx, shape, xt, dev, "dx")
    ws = kp = gp = None
    kn = 0
    if dweight is None and output_dweight:
        dweight = torch.empty_like(weight)
    if dweight is not None:
        gp = _dense(dweight, (D,), _F32, dev, "dweight")
        ws, kp, kn = _scratch(workspace, rmsnorm_bwd_workspace_size(M, D), dev)
    code = (_lib or load()).gdr_rmsnorm_bwd(dp, ds, sp, ss, wp, rp, rs, M, D, eps, xc, xp, xs, gp, kp, kn,
                                            _current_handle(dev.index))
    if code:
        _check(code)
    return dx, dweight


# ---- softmax attention and its paged cache -----------------------------------
#
# Token tensors are [T, heads, D] with dense heads and a token stride of their
# own (a column block of one projection's output); the rest as above.


def _tokens(t, shape, dtype, device, what):
    """(address, token stride) of a [T, heads, D] tensor with dense heads."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _refuse(t, shape, dtype, device, what)
    token, head, col = t.stride()
    T, H, D = shape
    if col != 1 or (head != D and H > 1):
        raise ValueError(f"{what} must have dense heads")
    return t.data_ptr(), token if T > 1 else H * D


def _attention_elsewhere(t, what, stream):
    """As _elsewhere, for [T, heads, D] tensors."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{what} must be [T, heads, D]")
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def _caches(k_cache, v_cache, block_table, cache_lens, N, Hkv, D, dtype, device):
    """The paged cache's arguments: addresses and sizes."""
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("caches must be [pages, Hkv, page_size, D], block_table [N, max_pages]")
    pages, _, page_size, _ = shape = k_cache.shape
    if shape != (pages, Hkv, page_size, D):
        raise ValueError(f"caches must be [pages, {Hkv}, page_size, {D}], not {tuple(shape)}")
    kp = _dense(k_cache, shape, dtype, device, "k_cache")
    vp = _dense(v_cache, shape, dtype, device, "v_cache")
    columns = block_table.shape[1]
    tp, ts = _rows(block_table, (N, columns), _I32, device, "block_table")
    return kp, vp, pages, page_size, tp, ts, columns, _dense(cache_lens, (N,), _I32, device, "cache_lens")


def kv_append(k, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens, *, q=None, freqs=None, flags: int = 0,
              q_out=None, k_out=None, output_k: bool = False, stream=None):
    """Appends k and v [T, Hkv, D] to the caches [pages, Hkv, page_size, D]:
    token i of sequence n goes to position cache_lens[n] + i, in the page
    block_table[n, position // page_size].  freqs [R / 2] fp32 (radians per
    position; None: no rotation) turns the first R channels of k and of q
    [T, Hq, D] (GDR_ROPE_PAIRS: neighbouring pairs).  cache_lens[n] < 0: the
    sequence is skipped.  Returns (q_out or None, k_out or None): q turned, and
    with output_k or k_out the turned k as dense rows; both may be in place."""
    if stream is not None or not k.is_cuda or k.get_device() != _current_device() or k.dim() != 3:
        with _attention_elsewhere(k, "k", stream):
            return kv_append(k, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens, q=q, freqs=freqs,
                             flags=flags, q_out=q_out, k_out=k_out, output_k=output_k)
    dev, shape, kt = k.device, k.shape, k.dtype
    T, Hkv, D = shape
    code = _CODES.get(kt)
    if code is None:
        _not_a_code(kt)
    N = cu_seqlens.numel() - 1
    kp, ks = _tokens(k, shape, kt, dev, "k")
    vp, vs = _tokens(v, shape, kt, dev, "v")
    cp = _dense(cu_seqlens, (N + 1,), _I32, dev, "cu_seqlens")
    ckp, cvp, pages, page_size, tp, ts, columns, lp = _caches(k_cache, v_cache, block_table, cache_lens, N, Hkv, D, kt,
                                                              dev)
    Hq, qp, qs, qop, qos = 0, None, 0, None, 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T, Hq, D]")
        Hq = q.shape[1]
        wide = (T, Hq, D)
        qp, qs = _tokens(q, wide, kt, dev, "q")
        if q_out is None:
            q_out = torch.empty(wide, dtype=kt, device=dev)
        qop, qos = _tokens(q_out, wide, kt, dev, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    kop, kos = None, 0
    if k_out is None and output_k:
        k_out = torch.empty(shape, dtype=kt, device=dev)
    if k_out is not None:
        kop, kos = _tokens(k_out, shape, kt, dev, "k_out")
    R, fp = 0, None
    if freqs is not None:
        R = 2 * freqs.numel()
        fp = _dense(freqs, (R // 2,), _F32, dev, "freqs")
    rc = (_lib or load()).gdr_kv_append(qp, qs, kp, ks, vp, vs, fp, R, lp, tp, ts, columns, cp, N, T, Hq, Hkv, D, code,
                                        flags, qop, qos, kop, kos, ckp, cvp, pages, page_size,
                                        _current_handle(dev.index))
    if rc:
        _check(rc)
    return q_out, k_out


def attn_fwd(q, k, v, cu_seqlens, *, scale=None, flags: int = 0, o=None, stream=None):
    """Causal softmax attention over packed prompts: q [T, Hq, D], k and v
    [T, Hkv, D] bf16 or fp32, D 64 or 128; query head h reads key head h /
    (Hq / Hkv); scale defaults to D ** -0.5.  Rows from cu_seqlens[N] on are not
    written.  Returns o [T, Hq, D]."""
    if stream is not None or not q.is_cuda or q.get_device() != _current_device() or q.dim() != 3:
        with _attention_elsewhere(q, "q", stream):
            return attn_fwd(q, k, v, cu_seqlens, scale=scale, flags=flags, o=o)
    dev, shape, qt = q.device, q.shape, q.dtype
    T, Hq, D = shape
    code = _CODES.get(qt)
    if code is None:
        _not_a_code(qt)
    if k.dim() != 3:
        raise ValueError("k must be [T, Hkv, D]")
    Hkv = k.shape[1]
    N = cu_seqlens.numel() - 1
    narrow = (T, Hkv, D)
    qp, qs = _tokens(q, shape, qt, dev, "q")
    kp, ks = _tokens(k, narrow, qt, dev, "k")
    vp, vs = _tokens(v, narrow, qt, dev, "v")
    cp = _dense(cu_seqlens, (N + 1,), _I32, dev, "cu_seqlens")
    if o is None:
        o = torch.empty(shape, dtype=qt, device=dev)
    op, os_ = _tokens(o, shape, qt, dev, "o")
    rc = (_lib or load()).gdr_attn_fwd(qp, qs, kp, ks, vp, vs, cp, N, T, Hq, Hkv, D,
                                       D ** -0.5 if scale is None else scale, code, flags, op, os_,
                                       _current_handle(dev.index))
    if rc:
        _check(rc)
    return o


@functools.lru_cache(maxsize=4096)
def _attn_step_bytes(N, T, Hq, Hkv, D, prefix_len, dtype):
    out = ctypes.c_size_t(0)
    # (ctypes would wrap a length of more than 32 bits; the largest int is refused)
    _check(load().gdr_attn_step_workspace_size(N, T, Hq, Hkv, D, min(prefix_len, 2 ** 31 - 1), dtype, ctypes.byref(out)))
    return out.value


def attn_step_workspace_size(N: int, T: int, Hq: int, Hkv: int, D: int, *, prefix_len: int = 0, dtype: int) -> int:
    return _attn_step_bytes(N, T, Hq, Hkv, D, prefix_len, dtype)


def attn_step(q, k_cache, v_cache, block_table, cache_lens, cu_seqlens, *, prefix_pages=None, prefix_len: int = 0,
              scale=None, flags: int = 0, o=None, workspace=None, stream=None):
    """Attention of a few tokens per sequence over the paged cache, after
    kv_append of the same tokens: token i of sequence n sees the keys 0 ..
    cache_lens[n] + i (cache_lens as kv_append took it; < 0: skipped).  The first
    prefix_len keys are the same for every sequence, in the pages prefix_pages
    [ceil(prefix_len / page_size)] int32, and are read once for the batch.
    Returns o [T, Hq, D]."""
    if stream is not None or not q.is_cuda or q.get_device() != _current_device() or q.dim() != 3:
        with _attention_elsewhere(q, "q", stream):
            return attn_step(q, k_cache, v_cache, block_table, cache_lens, cu_seqlens, prefix_pages=prefix_pages,
                             prefix_len=prefix_len, scale=scale, flags=flags, o=o, workspace=workspace)
    dev, shape, qt = q.device, q.shape, q.dtype
    T, Hq, D = shape
    code = _CODES.get(qt)
    if code is None:
        _not_a_code(qt)
    N = cu_seqlens.numel() - 1
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, Hkv, page_size, D]")
    Hkv = k_cache.shape[1]
    qp, qs = _tokens(q, shape, qt, dev, "q")
    cp = _dense(cu_seqlens, (N + 1,), _I32, dev, "cu_seqlens")
    ckp, cvp, pages, page_size, tp, ts, columns, lp = _caches(k_cache, v_cache, block_table, cache_lens, N, Hkv, D, qt,
                                                              dev)
    pp = _dense(prefix_pages, (-(-prefix_len // max(page_size, 1)),), _I32, dev, "prefix_pages")
    if o is None:
        o = torch.empty(shape, dtype=qt, device=dev)
    op, os_ = _tokens(o, shape, qt, dev, "o")
    ws, wp, wn = _scratch(workspace, _attn_step_bytes(N, T, Hq, Hkv, D, prefix_len, code), dev)
    rc = (_lib or load()).gdr_attn_step(qp, qs, ckp, cvp, pages, page_size, tp, ts, columns, lp, pp, prefix_len, cp, N,
                                        T, Hq, Hkv, D, D ** -0.5 if scale is None else scale, code, flags, op, os_, wp,
                                        wn, _current_handle(dev.index))
    if rc:
        _check(rc)
    return o


def device_status(stream=None) -> int:
    """Synchronise and read/clear the library's device error word."""
    w = ctypes.c_int(0)
    code = load().gdr_get_device_status(_stream(stream), ctypes.byref(w))
    if code not in (0, 5):
        _check(code)
    return w.value


def profile_enable(on: bool = True):
    """Bracket every library kernel launch with CUDA events on its stream."""
    _check(load().gdr_profile_enable(1 if on else 0))


def profile_read(max_kernels: int = 32):
    """{kernel name: (total device ms, launches)} since the previous read."""
    names = ctypes.create_string_buffer(4096)
    ms = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_int * max_kernels)()
    n = ctypes.c_int(0)
    _check(load().gdr_profile_read(max_kernels, names, 4096, ms, cnt, ctypes.byref(n)))
    keys = [k for k in names.value.decode().split(",") if k]
    return {keys[i]: (ms[i], cnt[i]) for i in range(n.value)}
