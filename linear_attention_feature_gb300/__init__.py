"""GB300-native kernelised (elu+1) linear attention.

Thin Python binding over the C ABI of ``liblinattn.so`` (declared in
``include/linattn.h``): argument marshalling only.  Every step of the
computation runs in the library's CUDA kernels; PyTorch is used for device
memory and streams.  There is no CPU fallback: if the library has not been
built (``python -m linear_attention_feature_gb300.build``) or a tensor is not
on a CUDA device, the call raises.

A call goes to the current stream, or to the one given as ``stream``.  What it
allocates is then that stream's memory; inputs have to stay until the stream
has passed the call (``record_stream``), and another stream has to wait for it
before it reads the results.

Automatic differentiation does not record the calls: results are detached.  The
backward_* functions are the gradients of their forwards.
"""
from __future__ import annotations

import array
import ctypes
import os
import struct

from . import build as _build

__all__ = ["forward", "forward_variant", "forward_gated", "decode_step_gated",
           "decode_step_delta",
           "forward_causal_state", "forward_host",
           "host_workspace_bytes", "decode_step",
           "rope_frequencies", "qk_norm_rope", "backward_qk_norm_rope",
           "forward_recurrence", "backward_recurrence", "decode_step_recurrence",
           "check_device_status",
           "kernel_launch_count", "LinAttnError",
           "load_library", "LA_F32", "LA_BF16", "STATUS", "EXPORTED"]

LA_F32 = 0
LA_BF16 = 1
STATUS = {0: "LA_OK", 1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED",
          3: "LA_ERR_CUDA", 4: "LA_ERR_NO_MEMORY", 5: "LA_ERR_TIMEOUT",
          6: "LA_ERR_INTERNAL"}
EXPORTED = ("la_forward", "la_forward_ex", "la_decode_step",
            "la_check_device_status", "la_status_string", "la_last_error",
            "la_abi_version", "la_kernel_launch_count",
            "la_forward_causal_noalloc", "la_forward_host",
            "la_forward_host_workspace_bytes", "la_forward_causal_state",
            "la_decode_step_ex", "la_forward_variant", "la_decode_step_variant",
            "la_forward_gated", "la_decode_step_gated", "la_decode_step_delta",
            "la_debug_inject_timeout", "la_debug_fail_next_allocs", "la_forward_delta",
            "la_qk_norm_rope", "la_backward_qk_norm_rope",
            "la_backward_qk_norm_rope_workspace_bytes", "la_recurrence_workspace_bytes",
            "la_forward_recurrence",
            "la_backward_recurrence", "la_decode_step_recurrence")

FEATURE_MAPS = {"elu1": 0, "identity": 1}
GATES = {"value": 0, "log": 1, "logit": 2}


class _Variant(ctypes.Structure):
    _fields_ = [("feature_map", ctypes.c_int), ("normalise", ctypes.c_int)]


def _variant(feature_map, normalise):
    if feature_map not in FEATURE_MAPS:
        raise ValueError(f"feature_map must be one of {sorted(FEATURE_MAPS)}")
    return ctypes.byref(_Variant(FEATURE_MAPS[feature_map], int(bool(normalise))))

_lib = None


class LinAttnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {detail}")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load liblinattn.so (built in-tree).  Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build the CUDA library first "
            "(python -m linear_attention_feature_gb300.build)")
    lib = ctypes.CDLL(p)
    V, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_float)
    lib.la_forward.argtypes = [V, V, V, V, I, I, I, I, I, F, I, V]
    lib.la_forward_ex.argtypes = [V, V, V, V, I, I, I, I, I, F, I, I, I, V]
    lib.la_decode_step.argtypes = [V, V, V, V, V, V, I, I, I, I, V]
    lib.la_decode_step_ex.argtypes = [V, V, V, V, V, V, I, I, I, F, I, V]
    lib.la_forward_causal_state.argtypes = [V, V, V, V, V, V, I, I, I, I, F, I, V]
    VP = ctypes.POINTER(_Variant)
    lib.la_forward_variant.argtypes = [V, V, V, V, I, I, I, I, I, F, I, VP, V]
    lib.la_decode_step_variant.argtypes = [V, V, V, V, V, V, I, I, I, F, I, VP, V]
    lib.la_forward_gated.argtypes = [V, V, V, V, V, I, I, I, I, I, VP, V]
    lib.la_decode_step_gated.argtypes = [V, V, V, V, V, V, V, I, I, I, I, VP, V]
    lib.la_decode_step_delta.argtypes = [V, V, V, V, V, V, V, I, I, I, I, V]
    lib.la_forward_host.argtypes = [V, V, V, V, I, I, I, I, I, F, I, V,
                                    ctypes.c_size_t, V]
    lib.la_forward_host_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.la_forward_host_workspace_bytes.restype = ctypes.c_size_t
    lib.la_forward_delta.argtypes = [V, V, V, V, V, V, V, I, I, I, I, I, V]
    lib.la_qk_norm_rope.argtypes = [V, V, V, V, V, V, V, I, ctypes.c_float, V,
                                    I, I, I, I, I, I, I, V]
    lib.la_backward_qk_norm_rope.argtypes = [V, V, V, V, V, V, V, V, V, V, V, I,
                                             ctypes.c_float, V, I, I, I, I, I, I, I,
                                             V, ctypes.c_size_t, V]
    lib.la_backward_qk_norm_rope_workspace_bytes.argtypes = [I]
    lib.la_backward_qk_norm_rope_workspace_bytes.restype = ctypes.c_size_t
    lib.la_forward_recurrence.argtypes = [V, V, V, V, V, V, I, I, I, I, I, I, I,
                                          V, ctypes.c_size_t, V]
    lib.la_backward_recurrence.argtypes = [V, V, V, V, V, V, V, V, V, V,
                                           I, I, I, I, I, I, I, V, ctypes.c_size_t, V]
    lib.la_recurrence_workspace_bytes.argtypes = [I, I, I]
    lib.la_recurrence_workspace_bytes.restype = ctypes.c_size_t
    lib.la_decode_step_recurrence.argtypes = [V, V, V, V, V, V, I, I, I, I, I, I, V]
    lib.la_debug_inject_timeout.argtypes = [ctypes.c_longlong, I]
    lib.la_debug_fail_next_allocs.argtypes = [I]
    lib.la_check_device_status.argtypes = [V]
    lib.la_status_string.argtypes = [I]
    lib.la_status_string.restype = ctypes.c_char_p
    lib.la_last_error.argtypes = []
    lib.la_last_error.restype = ctypes.c_char_p
    lib.la_abi_version.argtypes = []
    lib.la_kernel_launch_count.argtypes = []
    lib.la_kernel_launch_count.restype = ctypes.c_ulonglong
    for n in ("la_forward", "la_forward_ex", "la_decode_step", "la_forward_host",
              "la_decode_step_ex", "la_forward_causal_state",
              "la_forward_variant", "la_decode_step_variant",
              "la_forward_gated", "la_decode_step_gated", "la_decode_step_delta",
              "la_debug_inject_timeout", "la_debug_fail_next_allocs",
              "la_forward_delta", "la_check_device_status", "la_abi_version",
              "la_qk_norm_rope", "la_backward_qk_norm_rope", "la_forward_recurrence",
              "la_backward_recurrence", "la_decode_step_recurrence"):
        getattr(lib, n).restype = I
    if path is None:
        _lib = lib
    return lib


def _raise_if(status: int):
    if status != 0:
        detail = load_library().la_last_error().decode(errors="replace")
        raise LinAttnError(status, detail)


def _torch():
    import torch
    return torch


_CODES = {}


def _codes():
    torch = _torch()
    _CODES.update({torch.float32: LA_F32, torch.bfloat16: LA_BF16,
                   torch.int32: 4, torch.int64: 8})  # positions: their bytes
    return _CODES


def _code(dtype) -> int:
    """LA_F32 or LA_BF16."""
    code = (_CODES or _codes()).get(dtype)
    if code != LA_F32 and code != LA_BF16:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return code


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _check_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _stream_ptr(stream, device):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _memory_of(stream, device):
    """Context in which new tensors come out of `stream`'s memory.  What another
    stream's allocator gives may still be read there by work that was enqueued
    before it was freed."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    return torch.cuda.stream(stream)


def _empty(stream, shape, dtype, device):
    """A new tensor in the memory of `stream` (None: of the current stream)."""
    if stream is None:
        return _torch().empty(shape, dtype=dtype, device=device)
    with _memory_of(stream, device):
        return _torch().empty(shape, dtype=dtype, device=device)


def _empty_like(stream, t):
    if stream is None:
        return _torch().empty_like(t)
    with _memory_of(stream, t.device):
        return _torch().empty_like(t)


def _enter(index, stream):
    """Makes CUDA device `index` the current one.  Returns the stream that the
    call goes to and the device to go back to (-1: it was current already)."""
    c = _torch()._C
    now, back = c._cuda_getDevice(), -1
    if now != index:
        _torch().cuda.set_device(index)
        back = now
    return (stream.cuda_stream if stream is not None else c._cuda_getCurrentRawStream(index)), back


def _leave(back):
    _torch().cuda.set_device(back)


def _decay_arg(decay, H):
    if decay is None:
        return None
    vals = [float(x) for x in (decay.tolist() if hasattr(decay, "tolist") else decay)]
    if len(vals) != H:
        raise ValueError(f"decay must have H={H} entries")
    return (ctypes.c_float * H)(*vals)


def forward(q, k, v, causal: bool = True, decay=None, out=None, *,
            path: int = 0, segment_chunks: int = 0, stream=None):
    """Linear attention over full sequences; q, k, v [B, H, N, d] on CUDA.

    causal=False: phi(Q)[phi(K)^T V] / phi(Q)[phi(K)^T 1].
    causal=True : running-state recurrence with optional per-head decay
    (`decay`: H floats in [0, 1]).  Returns `out` ([B, H, N, d], q's dtype).
    """
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(q, k, v, out)
    B, H, N, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_forward_ex(
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            B, H, N, d, int(bool(causal)), _decay_arg(decay, H),
            _dtype_code(q), int(path), int(segment_chunks),
            _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


def forward_variant(q, k, v, causal: bool = True, decay=None, out=None, *,
                    feature_map: str = "elu1", normalise: bool = True,
                    stream=None):
    """forward() with the feature map ("elu1" or "identity") and the
    normaliser selectable.  feature_map="identity", normalise=False with a
    decay is retention: o_i = sum_{j<=i} g^(i-j) (q_i . k_j) v_j."""
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(q, k, v, out)
    B, H, N, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_forward_variant(
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            B, H, N, d, int(bool(causal)), _decay_arg(decay, H), _dtype_code(q),
            _variant(feature_map, normalise), _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


def forward_gated(q, k, v, gates, out=None, *, feature_map: str = "elu1",
                  normalise: bool = True, stream=None):
    """Causal recurrence with a data-dependent scalar gate per token and
    head: gates [B, H, N] float32 on the GPU, values in [0, 1]
    (S_t = gates_t S_{t-1} + phi(k_t) v_t^T, z likewise)."""
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    B, H, N, d = q.shape
    if tuple(gates.shape) != (B, H, N) or gates.dtype != torch.float32:
        raise ValueError("gates must be float32 [B, H, N]")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(q, k, v, out, gates)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_forward_gated(
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            ctypes.c_void_p(gates.data_ptr()), B, H, N, d, _dtype_code(q),
            _variant(feature_map, normalise), _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


def decode_step_gated(S, z, q, k, v, gates, out=None, *, feature_map="elu1",
                      normalise=True, stream=None):
    """decode_step with this token's gate per head: gates [B, H] float32 on
    the GPU (S <- gates S + phi(k) v^T, z likewise)."""
    torch = _torch()
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, d] shape")
    B, H, d = q.shape
    if tuple(S.shape) != (B, H, d, d) or tuple(z.shape) != (B, H, d):
        raise ValueError("S must be [B, H, d, d] and z [B, H, d]")
    if tuple(gates.shape) != (B, H) or gates.dtype != torch.float32:
        raise ValueError("gates must be float32 [B, H]")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(S, z, q, k, v, out, gates)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_decode_step_gated(
            ctypes.c_void_p(S.data_ptr()), ctypes.c_void_p(z.data_ptr()),
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            ctypes.c_void_p(gates.data_ptr()), B, H, d, _dtype_code(q),
            _variant(feature_map, normalise), _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


def decode_step_delta(S, q, k, v, beta, alpha=None, out=None, *, stream=None):
    """One delta-rule step per head (Gated DeltaNet with `alpha`): S [B, H,
    d, d] fp32 (S[a][c], a key feature) updated in place; beta, alpha
    [B, H] fp32 on the GPU; returns o = S_t^T q [B, H, d]."""
    torch = _torch()
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, d] shape")
    B, H, d = q.shape
    if tuple(S.shape) != (B, H, d, d) or S.dtype != torch.float32:
        raise ValueError("S must be float32 [B, H, d, d]")
    for name, t in (("beta", beta), ("alpha", alpha)):
        if t is not None and (tuple(t.shape) != (B, H) or t.dtype != torch.float32):
            raise ValueError(f"{name} must be float32 [B, H]")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(S, q, k, v, out, beta, *([alpha] if alpha is not None else []))
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_decode_step_delta(
            ctypes.c_void_p(S.data_ptr()), ctypes.c_void_p(q.data_ptr()),
            ctypes.c_void_p(k.data_ptr()), ctypes.c_void_p(v.data_ptr()),
            ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(beta.data_ptr()),
            ctypes.c_void_p(alpha.data_ptr() if alpha is not None else None),
            B, H, d, _dtype_code(q), _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


def forward_delta(q, k, v, beta, alpha=None, out=None, S=None, *, stream=None):
    """The delta rule over sequences q, k, v [B, H, N, d] (DeltaNet; Gated
    DeltaNet with `alpha`): beta, alpha [B, H, N] fp32 on the GPU, one per
    token; S [B, H, d, d] fp32 (S[a][c], a key feature) the start state,
    updated in place to the state after the last token (None: start from
    zero).  Returns out [B, H, N, d] with o_t = S_t q_t."""
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    B, H, N, d = q.shape
    for name, t in (("beta", beta), ("alpha", alpha)):
        if t is not None and (tuple(t.shape) != (B, H, N) or t.dtype != torch.float32):
            raise ValueError(f"{name} must be float32 [B, H, N]")
    if S is not None and (tuple(S.shape) != (B, H, d, d) or S.dtype != torch.float32):
        raise ValueError("S must be float32 [B, H, d, d]")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(q, k, v, out, beta, *[t for t in (alpha, S) if t is not None])
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_forward_delta(
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            ctypes.c_void_p(beta.data_ptr()),
            ctypes.c_void_p(alpha.data_ptr() if alpha is not None else None),
            ctypes.c_void_p(S.data_ptr() if S is not None else None),
            B, H, N, d, _dtype_code(q), _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


def forward_causal_state(q, k, v, decay=None, out=None, S=None, z=None, *,
                         stream=None):
    """Causal forward that also returns the final state: (out, S, z) with
    S [B, H, d, d] and z [B, H, d] in fp32 -- the state after the last token,
    in the layout decode_step takes, so that a decode continues the
    sequence."""
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    B, H, N, d = q.shape
    if out is None:
        out = _empty_like(stream, q)
    if S is None:
        S = _empty(stream, (B, H, d, d), torch.float32, q.device)
    if z is None:
        z = _empty(stream, (B, H, d), torch.float32, q.device)
    if tuple(S.shape) != (B, H, d, d) or tuple(z.shape) != (B, H, d):
        raise ValueError("S must be [B, H, d, d] and z [B, H, d]")
    if S.dtype != torch.float32 or z.dtype != torch.float32:
        raise TypeError("S and z must be float32")
    _check_cuda(q, k, v, out, S, z)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_forward_causal_state(
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            ctypes.c_void_p(S.data_ptr()), ctypes.c_void_p(z.data_ptr()),
            B, H, N, d, _decay_arg(decay, H), _dtype_code(q),
            _stream_ptr(stream, q.device))
    _raise_if(st)
    return out, S, z


def decode_step(S, z, q, k, v, out=None, *, decay=None, feature_map="elu1",
                normalise=True, stream=None):
    """One decode step per head: S, z (fp32, [B, H, d, d] / [B, H, d]) are
    updated in place (S <- g S + phi(k) v^T, z <- g z + phi(k), with the
    per-head decay g from `decay`, H floats in [0, 1], or 1); q, k, v
    [B, H, d]; returns out [B, H, d].  feature_map / normalise as in
    forward_variant."""
    torch = _torch()
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, d] shape")
    B, H, d = q.shape
    if tuple(S.shape) != (B, H, d, d) or tuple(z.shape) != (B, H, d):
        raise ValueError("S must be [B, H, d, d] and z [B, H, d]")
    if S.dtype != torch.float32 or z.dtype != torch.float32:
        raise TypeError("S and z must be float32")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        out = _empty_like(stream, q)
    _check_cuda(S, z, q, k, v, out)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.la_decode_step_variant(
            ctypes.c_void_p(S.data_ptr()), ctypes.c_void_p(z.data_ptr()),
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            B, H, d, _decay_arg(decay, H), _dtype_code(q),
            _variant(feature_map, normalise), _stream_ptr(stream, q.device))
    _raise_if(st)
    return out


# ------------------------------------------------------------------ queries
# and keys out of a projection

def rope_frequencies(rotary_dim: int, base: float = 10000.0):
    """The usual rotation frequencies base^(-2i / rotary_dim), i < rotary_dim
    / 2, in radians per position, as qk_norm_rope takes them."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    return array.array("d", [float(base) ** (-2.0 * i / rotary_dim)
                             for i in range(rotary_dim // 2)])


# la_rope: frequencies, rotary_dim, interleaved, positions, position_bytes,
# position_stride_b, position_stride_n, offset
_ROPE = struct.Struct("@PiiPiqqq")


def _rope(frequencies, positions, offset, interleaved, shape, index):
    """The packed la_rope (None: no rotation) and what has to outlive the call;
    `shape`: q's, `index`: its device's."""
    if frequencies is None or len(frequencies) == 0:
        return None, None
    f = frequencies
    if not (isinstance(f, array.array) and f.typecode == "d"):
        f = array.array("d", [float(x) for x in f])
    if positions is None:
        return _ROPE.pack(f.buffer_info()[0], 2 * len(f), bool(interleaved), 0, 0, 0, 0, offset), f
    st, sb, sn = positions.stride(), 0, 0
    have, want = positions.shape, shape[:1] if len(shape) == 3 else (shape[0], shape[2])
    if have == want:
        sb, sn = (st[0], 0) if len(st) == 1 else st
    elif len(shape) == 4 and have == want[1:]:
        sn = st[0]
    else:
        raise ValueError(f"positions must have the shape {list(want)}"
                         + (f" or {list(want[1:])}" if len(shape) == 4 else ""))
    nbytes = (_CODES or _codes()).get(positions.dtype)
    if nbytes not in (4, 8):
        raise TypeError("positions must be int32 or int64")
    if positions.get_device() != index:
        raise ValueError("positions must be on q's CUDA device")
    return _ROPE.pack(f.buffer_info()[0], 2 * len(f), bool(interleaved), positions.data_ptr(),
                      nbytes, sb, sn, offset), f


_STRIDES = {n: struct.Struct(f"@{n}q") for n in (3, 6, 12, 18)}


def _check_rows(q, *ts):
    """Tensors of rows with q's dtype and CUDA device and a contiguous last
    dimension; returns the device's index and their packed la_strides."""
    index, dtype, v = q.get_device(), q.dtype, []
    if index < 0:
        raise ValueError("all tensors must be on a CUDA device")
    for t in ts:
        if t.get_device() != index:
            raise ValueError("all tensors must be on one CUDA device")
        if t.dtype is not dtype:
            raise TypeError("q, k, their outputs and gradients must share one dtype")
        s = t.stride()
        if s[-1] != 1 and t.shape[-1] > 1:
            raise ValueError("the last dimension must be contiguous")
        v += s[:3] if len(s) == 4 else (s[0], s[1], 0)
    return index, _STRIDES[len(v)].pack(*v)


def _weights(q_weight, k_weight, d, index):
    """(q_weight's and k_weight's pointers or None, their dtype code)."""
    pq = pk = dtype = None
    for w in (q_weight, k_weight):
        if w is None:
            continue
        if w.shape != (d,):
            raise ValueError(f"a weight must have the shape [{d}]")
        if w.get_device() != index:
            raise ValueError("the weights must be on q's CUDA device")
        if w.stride(0) != 1 and d > 1:
            raise ValueError("a weight must be contiguous")
        if dtype is not None and w.dtype is not dtype:
            raise TypeError("q_weight and k_weight must share one dtype")
        dtype = w.dtype
    if q_weight is not None:
        pq = q_weight.data_ptr()
    if k_weight is not None:
        pk = k_weight.data_ptr()
    return pq, pk, LA_F32 if dtype is None else _code(dtype)


def _check_qk(qs, ks):
    """B, Hq, Hk, N, d of q's and k's shapes."""
    n = len(qs)
    if n not in (3, 4) or len(ks) != n:
        raise ValueError("q and k must be [B, H, N, d], or [B, H, d] for one token")
    if ks[0] != qs[0] or ks[2:] != qs[2:]:
        raise ValueError("q and k may differ in the number of heads only")
    return qs[0], qs[1], ks[1], qs[2] if n == 4 else 1, qs[-1]


def qk_norm_rope(q, k, q_weight=None, k_weight=None, frequencies=None, positions=None, *,
                 offset: int = 0, norm: bool = True, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Queries and keys as forward() and decode_step() take them, in one pass:
    RMS norm over each head's d values, times a weight per feature, then the
    position rotation.  q [B, Hq, N, d] and k [B, Hk, N, d] (or [B, H, d]: one
    token each) may have any strides with a contiguous last dimension, such as
    views of a fused projection; the results are contiguous unless q_out and
    k_out say otherwise (q_out=q, k_out=k: in place).

    q_weight, k_weight [d]: float32 or bfloat16, or None.  frequencies:
    radians per position of each pair (rope_frequencies()), None for no
    rotation; features beyond 2 len(frequencies) are not rotated.  positions:
    int32 or int64 [B, N] or [N] ([B] for one token), or None for 0..N-1;
    `offset` is added.  interleaved: pairs (2i, 2i+1) instead of (i, i + R/2).
    Returns (q_out, k_out)."""
    qs, ks, device = q.shape, k.shape, q.device
    B, Hq, Hk, N, d = _check_qk(qs, ks)
    dtype = q.dtype
    if q_out is None:
        q_out = _empty(stream, qs, dtype, device)
    elif q_out.shape != qs:
        raise ValueError("q_out must have q's shape")
    if k_out is None:
        k_out = _empty(stream, ks, dtype, device)
    elif k_out.shape != ks:
        raise ValueError("k_out must have k's shape")
    index, strides = _check_rows(q, q, k, q_out, k_out)
    wq, wk, wcode = _weights(q_weight, k_weight, d, index)
    rope, keep = _rope(frequencies, positions, offset, interleaved, qs, index)
    code, lib = _code(dtype), load_library()
    to, back = _enter(index, stream)
    try:
        st = lib.la_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), strides, wq, wk,
            bool(norm), eps, rope, B, Hq, Hk, N, d, code, wcode, to)
    finally:
        if back >= 0:
            _leave(back)
    if st:
        _raise_if(st)
    return q_out, k_out


# workspace bytes of the backward per feature, by device
_BACK_WORKSPACE = {}


def backward_qk_norm_rope(dq_out, dk_out, q, k, q_weight=None, k_weight=None,
                          frequencies=None, positions=None, *, offset: int = 0,
                          norm: bool = True, eps: float = 1e-6, interleaved: bool = False,
                          dq=None, dk=None, stream=None):
    """Gradients of qk_norm_rope (same arguments as the forward call): returns
    (dq, dk, dq_weight, dk_weight), the weights' in float32 and None where
    there is no weight.  dq and dk take any strides, such as views of a fused
    projection's gradient (default: laid out like q and k)."""
    torch = _torch()
    qs, ks, device = q.shape, k.shape, q.device
    B, Hq, Hk, N, d = _check_qk(qs, ks)
    if dq_out.shape != qs or dk_out.shape != ks:
        raise ValueError("dq_out and dk_out must have the shapes of q and k")
    if dq is None:
        dq = _empty_like(stream, q)
    if dk is None:
        dk = _empty_like(stream, k)
    if dq.shape != qs or dk.shape != ks:
        raise ValueError("dq and dk must have the shapes of q and k")
    index, strides = _check_rows(q, dq_out, dk_out, q, k, dq, dk)
    wq, wk, wcode = _weights(q_weight, k_weight, d, index)
    rope, keep = _rope(frequencies, positions, offset, interleaved, qs, index)
    code, lib = _code(q.dtype), load_library()
    to, back = _enter(index, stream)
    try:
        dwq = dwk = ws = None
        ws_bytes = 0
        if wq is not None:
            dwq = _empty(stream, d, torch.float32, device)
        if wk is not None:
            dwk = _empty(stream, d, torch.float32, device)
        # on the current stream torch's allocator gives the workspace; the
        # library allocates on another one
        if stream is None and (wq is not None or wk is not None):
            per_feature = _BACK_WORKSPACE.get(index)
            if per_feature is None:
                per_feature = lib.la_backward_qk_norm_rope_workspace_bytes(1)
                _BACK_WORKSPACE[index] = per_feature
            ws_bytes = per_feature * d
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        st = lib.la_backward_qk_norm_rope(
            dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), _ptr(dwq), _ptr(dwk), strides, wq, wk, bool(norm), eps, rope, B, Hq,
            Hk, N, d, code, wcode, _ptr(ws), ws_bytes, to)
    finally:
        if back >= 0:
            _leave(back)
    if st:
        _raise_if(st)
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------ the
# recurrence with a gate per channel

def _gate(gate) -> int:
    code = GATES.get(gate)
    if code is None:
        raise ValueError(f"gate must be one of {sorted(GATES)}")
    return code


def _check_seq(x, gates, *ts):
    """[B, N, C] (or [B, C]) tensors of x's shape, dtype and device, and gates;
    returns the device's index."""
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    for t in ts:
        if t.shape != shape:
            raise ValueError("x, gates, out and the gradients must share one shape")
        if t.dtype is not dtype:
            raise TypeError("x, out and the gradients must share one dtype")
    if gates.shape != shape:
        raise ValueError("x, gates, out and the gradients must share one shape")
    if gates.dtype is not dtype and gates.dtype is not _torch().float32:
        raise TypeError("gates must be float32 or of x's dtype")
    for t in (x, gates, *ts):
        if index < 0 or t.get_device() != index:
            raise ValueError("all tensors must be on one CUDA device")
        if t.stride(-1) != 1 and shape[-1] > 1:
            raise ValueError("the last dimension must be contiguous")
    return index


def _check_state(B, C, index, *hs):
    float32 = _torch().float32
    for h in hs:
        if h is None:
            continue
        if h.shape != (B, C) or h.dtype is not float32:
            raise ValueError("a state must be float32 [B, C]")
        if h.get_device() != index:
            raise ValueError("all tensors must be on one CUDA device")
        if not h.is_contiguous():
            raise ValueError("a state must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _recurrence_workspace(lib, B, C, code, device, stream):
    """(workspace or None, bytes): on the current stream torch's allocator
    gives it; the library allocates on another one."""
    if stream is not None or B * C > 1024:  # more channels never need one
        return None, 0
    n = lib.la_recurrence_workspace_bytes(B, C, code)
    if n == 0:
        return None, 0
    torch = _torch()
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _seq_strides(*ts):
    v = []
    for t in ts:
        v += (0, 0) if t is None else t.stride()[:2]
    return _STRIDES[len(v)].pack(*v)


def forward_recurrence(x, gates, h0=None, out=None, *, h_last=None, gate: str = "value",
                       complement: bool = False, stream=None):
    """The gated linear recurrence with a gate per channel over sequences
    x, gates [B, N, C]: h_t = a_t h_{t-1} + x_t, or + (1 - a_t) x_t with
    `complement`.  gates (float32 or x's dtype) hold a_t ("value"), log a_t
    ("log") or its logit ("logit").  h0 [B, C] float32: the state before the
    first token (None: zero).  Any strides with contiguous channels.  Returns
    (out [B, N, C], h_last [B, C] float32); h_last=h0 updates in place, and
    decode_step_recurrence continues from it."""
    torch = _torch()
    if x.dim() != 3:
        raise ValueError("x must be [B, N, C]")
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    B, N, C = x.shape
    device = x.device
    if h_last is None:
        h_last = _empty(stream, (B, C), torch.float32, device)
    form = _gate(gate)
    index = _check_seq(x, gates, out)
    _check_state(B, C, index, h0, h_last)
    code, gcode, lib = _code(x.dtype), _code(gates.dtype), load_library()
    to, back = _enter(index, stream)
    try:
        ws, ws_bytes = _recurrence_workspace(lib, B, C, code, device, stream)
        st = lib.la_forward_recurrence(
            x.data_ptr(), gates.data_ptr(), _ptr(h0), out.data_ptr(), h_last.data_ptr(),
            _seq_strides(x, gates, out), B, N, C, form, bool(complement), code, gcode, _ptr(ws),
            ws_bytes, to)
    finally:
        if back >= 0:
            _leave(back)
    if st:
        _raise_if(st)
    return out, h_last


def backward_recurrence(dout, gates, out, x=None, h0=None, dh_last=None, *, dx=None,
                        dgates=None, dh0=None, gate: str = "value",
                        complement: bool = False, stream=None):
    """Gradients of forward_recurrence: dout and dh_last (None: zero) are those
    of its two results, `out` is what it returned; x is needed with
    `complement` only.  Returns (dx, dgates, dh0), dgates with respect to the
    gates as given (value, logarithm or logit)."""
    torch = _torch()
    if dout.dim() != 3:
        raise ValueError("dout must be [B, N, C]")
    if complement and x is None:
        raise ValueError("x is needed with complement")
    B, N, C = dout.shape
    device = dout.device
    if dx is None:
        dx = _empty(stream, dout.shape, dout.dtype, device)
    if dgates is None:
        dgates = _empty(stream, gates.shape, gates.dtype, device)
    if dh0 is None:
        dh0 = _empty(stream, (B, C), torch.float32, device)
    form = _gate(gate)
    if not complement:
        x = None
    index = _check_seq(dout, gates, out, dx, *([x] if x is not None else []))
    if dgates.dtype is not gates.dtype:
        raise TypeError("dgates must have the dtype of gates")
    _check_seq(dout, dgates)
    _check_state(B, C, index, h0, dh_last, dh0)
    code, gcode, lib = _code(dout.dtype), _code(gates.dtype), load_library()
    to, back = _enter(index, stream)
    try:
        ws, ws_bytes = _recurrence_workspace(lib, B, C, code, device, stream)
        st = lib.la_backward_recurrence(
            dout.data_ptr(), gates.data_ptr(), out.data_ptr(), _ptr(x), _ptr(h0),
            _ptr(dh_last), dx.data_ptr(), dgates.data_ptr(), dh0.data_ptr(),
            _seq_strides(dout, gates, out, x, dx, dgates), B, N, C, form, bool(complement),
            code, gcode, _ptr(ws), ws_bytes, to)
    finally:
        if back >= 0:
            _leave(back)
    if st:
        _raise_if(st)
    return dx, dgates, dh0


def decode_step_recurrence(h, x, gates, out=None, *, h_out=None, gate: str = "value",
                           complement: bool = False, stream=None):
    """One token of forward_recurrence: h [B, C] float32 is updated in place
    (or read, and the new state written to h_out); x, gates [B, C].  Returns
    out [B, C], the new state in x's dtype."""
    if x.dim() != 2:
        raise ValueError("x must be [B, C]")
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    if h_out is None:
        h_out = h
    B, C = x.shape
    form = _gate(gate)
    index = _check_seq(x, gates, out)
    _check_state(B, C, index, h, h_out)
    code, gcode, lib = _code(x.dtype), _code(gates.dtype), load_library()
    to, back = _enter(index, stream)
    try:
        st = lib.la_decode_step_recurrence(
            h.data_ptr(), h_out.data_ptr(), x.data_ptr(), gates.data_ptr(), out.data_ptr(),
            _STRIDES[3].pack(x.stride(0), gates.stride(0), out.stride(0)), B, C, form,
            bool(complement), code, gcode, to)
    finally:
        if back >= 0:
            _leave(back)
    if st:
        _raise_if(st)
    return out


def kernel_launch_count() -> int:
    """Kernels enqueued by the library in this process so far."""
    return int(load_library().la_kernel_launch_count())


def check_device_status(stream=None, device=None):
    """Synchronise the stream and raise if a kernel reported a device-side
    failure (a bounded wait that ran out)."""
    torch = _torch()
    dev = device if device is not None else torch.cuda.current_device()
    with torch.cuda.device(dev):
        st = load_library().la_check_device_status(_stream_ptr(stream, dev))
    _raise_if(st)


def host_workspace_bytes(shape, dtype) -> int:
    """Device workspace bytes that forward_host needs for [B, H, N, d]."""
    torch = _torch()
    code = LA_BF16 if dtype == torch.bfloat16 else LA_F32 if dtype == torch.float32 else -1
    if code < 0:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    B, H, N, d = (int(x) for x in shape)
    return int(load_library().la_forward_host_workspace_bytes(B, H, N, d, code))


def forward_host(q, k, v, causal: bool = True, decay=None, out=None, *,
                 workspace=None, device=None, stream=None):
    """forward() on HOST tensors q, k, v [B, H, N, d] (page-locked for full
    speed): the library copies them to the GPU, runs the forward and copies
    the result into `out` (a host tensor, allocated page-locked if None),
    pipelined over groups of heads.  `workspace` is a uint8 CUDA tensor of at
    least host_workspace_bytes(q.shape, q.dtype) bytes (allocated if None).
    The call is asynchronous: `out` is complete once `stream` (default: the
    current stream of `device`) has passed it, e.g. after
    torch.cuda.current_stream().synchronize()."""
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must share one [B, H, N, d] shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("forward_host takes contiguous host tensors")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if out.is_cuda or not out.is_contiguous() or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must be a contiguous host tensor like q")
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    need = host_workspace_bytes(q.shape, q.dtype)
    if workspace is None:
        workspace = _empty(stream, max(need, 1), torch.uint8, dev)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    B, H, N, d = q.shape
    lib = load_library()
    with torch.cuda.device(workspace.device):
        st = lib.la_forward_host(
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
            ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            B, H, N, d, int(bool(causal)), _decay_arg(decay, H),
            _dtype_code(q), ctypes.c_void_p(workspace.data_ptr()),
            ctypes.c_size_t(workspace.numel() * workspace.element_size()),
            _stream_ptr(stream, workspace.device))
    _raise_if(st)
    return out
