"""Python binding of the GB300 RMSNorm C ABI (``include/rmsnorm.h``).

Argument marshalling only: every function forwards to the entry point of the
same name in ``librmsnorm_gb300.so`` and raises :class:`RMSNormError` on a
non-OK status.  Pointers are device addresses (ints, or objects with a
``data_ptr()`` method such as torch tensors); ``stream`` is a raw
``cudaStream_t`` (int), an object with a ``cuda_stream`` attribute, or None
for the legacy default stream.  Importing works without the library; the
first call raises if it has not been built (``__graft_entry__.build()``) --
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = ["F32", "BF16", "OP_FWD", "OP_FUSED_ADD", "OP_BWD", "OP_FUSED_ADD_BWD", "RMSNormError",
           "OP_FWD_STRIDED", "OP_FWD_FP8", "OP_FUSED_ADD_FP8", "OP_FWD_NVFP4",
           "OP_FUSED_ADD_NVFP4", "rmsnorm_fwd_fp8", "rmsnorm_fwd_nvfp4", "OP_LAYERNORM_FWD",
           "OP_LAYERNORM_BWD", "layernorm_fwd", "layernorm_bwd_workspace_size", "layernorm_bwd",
           "library_path", "rmsnorm_fused_add_bwd", "rmsnorm_fwd_strided",
           "load_library", "rmsnorm_fwd", "rmsnorm_fused_add_fwd", "rmsnorm_bwd",
           "rmsnorm_bwd_workspace_size", "rmsnorm_status_string", "rmsnorm_describe_plan",
           "rmsnorm_bwd_noalloc", "NOALLOC_SCRATCH_BYTES", "rmsnorm_check_device",
           "rmsnorm_last_error", "rmsnorm_reload_debug_env", "EXPORTED_SYMBOLS", "Heads", "Rope",
           "rmsnorm_rope_fwd", "rmsnorm_rope_bwd_workspace_size", "rmsnorm_rope_bwd",
           "rmsnorm_token_logprob_fwd", "rmsnorm_token_logprob_bwd", "rmsnorm_policy_loss_fwd",
           "rmsnorm_preference_loss_fwd"]

F32 = 0
BF16 = 1
OP_FWD, OP_FUSED_ADD, OP_BWD, OP_FUSED_ADD_BWD = 0, 1, 2, 3
OP_FWD_STRIDED, OP_FWD_FP8, OP_FUSED_ADD_FP8, OP_FWD_NVFP4, OP_FUSED_ADD_NVFP4 = 4, 5, 6, 7, 8
OP_LAYERNORM_FWD, OP_LAYERNORM_BWD = 9, 10
_DT_NAMES = {"f32": F32, "bf16": BF16}

EXPORTED_SYMBOLS = ("rmsnorm_fwd", "rmsnorm_fused_add_fwd", "rmsnorm_bwd_workspace_size",
                    "rmsnorm_bwd", "rmsnorm_status_string", "rmsnorm_describe_plan",
                    "rmsnorm_bwd_noalloc", "rmsnorm_check_device", "rmsnorm_last_error",
                    "rmsnorm_fused_add_bwd", "rmsnorm_fwd_strided", "rmsnorm_fwd_fp8",
                    "rmsnorm_fwd_nvfp4", "layernorm_fwd", "layernorm_bwd_workspace_size",
                    "layernorm_bwd", "rmsnorm_reload_debug_env", "rmsnorm_rope_fwd",
                    "rmsnorm_rope_bwd_workspace_size", "rmsnorm_rope_bwd",
                    "rmsnorm_token_logprob_fwd", "rmsnorm_token_logprob_bwd",
                    "rmsnorm_policy_loss_fwd", "rmsnorm_preference_loss_fwd")

# Size of the library-owned scratch of rmsnorm_bwd_noalloc (16 MiB).
NOALLOC_SCRATCH_BYTES = 16 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "librmsnorm_gb300.so")
_lock = threading.Lock()
_lib = None


class RMSNormError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = f" [{rmsnorm_last_error()}]" if status == 5 else ""
        super().__init__(f"{where}: {rmsnorm_status_string(status)} (status {status}){detail}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load the shared library (raises if it is missing: no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                                  "(nvcc, sm_103a) first")
            lib = ctypes.CDLL(_LIB_PATH)
            P, I64, I, F, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                ctypes.c_size_t)
            lib.rmsnorm_fwd.argtypes = [P, P, P, P, I64, I64, F, I, I, P]
            lib.rmsnorm_fwd.restype = I
            lib.rmsnorm_fused_add_fwd.argtypes = [P, P, P, P, P, I64, I64, F, I, I, P]
            lib.rmsnorm_fused_add_fwd.restype = I
            lib.rmsnorm_bwd_workspace_size.argtypes = [I64, I64, I, I, I, ctypes.POINTER(SZ)]
            lib.rmsnorm_bwd_workspace_size.restype = I
            lib.rmsnorm_bwd.argtypes = [P, P, P, P, P, P, P, SZ, I64, I64, F, I, I, P]
            lib.rmsnorm_bwd.restype = I
            lib.rmsnorm_status_string.argtypes = [I]
            lib.rmsnorm_status_string.restype = ctypes.c_char_p
            lib.rmsnorm_describe_plan.argtypes = [I, I64, I64, I, I, I, I, ctypes.c_char_p, SZ]
            lib.rmsnorm_describe_plan.restype = I
            lib.rmsnorm_bwd_noalloc.argtypes = [P, P, P, P, P, P, I64, I64, F, I, I, P]
            lib.rmsnorm_bwd_noalloc.restype = I
            lib.rmsnorm_check_device.argtypes = [P]
            lib.rmsnorm_check_device.restype = I
            lib.rmsnorm_fused_add_bwd.argtypes = [P, P, P, P, P, P, I, P, SZ, I64, I64, F, I, I, P]
            lib.rmsnorm_fused_add_bwd.restype = I
            lib.rmsnorm_fwd_strided.argtypes = [P, I64, I64, P, P, I64, I64, P, I64, I64, I64, F,
                                                I, I, P]
            lib.rmsnorm_fwd_strided.restype = I
            lib.layernorm_fwd.argtypes = [P, P, P, P, P, P, I64, I64, F, I, I, P]
            lib.layernorm_fwd.restype = I
            lib.layernorm_bwd_workspace_size.argtypes = [I64, I64, I, I, I, ctypes.POINTER(SZ)]
            lib.layernorm_bwd_workspace_size.restype = I
            lib.layernorm_bwd.argtypes = [P, P, P, P, P, P, P, P, P, SZ, I64, I64, F, I, I, P]
            lib.layernorm_bwd.restype = I
            lib.rmsnorm_fwd_fp8.argtypes = [P, P, P, P, P, P, I64, I64, F, I, I, P]
            lib.rmsnorm_fwd_fp8.restype = I
            lib.rmsnorm_fwd_nvfp4.argtypes = [P, P, P, F, P, P, P, I64, I64, F, I, I, P]
            lib.rmsnorm_fwd_nvfp4.restype = I
            lib.rmsnorm_rope_fwd.argtypes = [P, P, P, P, P, P, P, I64, I64, F, I, I, P]
            lib.rmsnorm_rope_fwd.restype = I
            lib.rmsnorm_rope_bwd_workspace_size.argtypes = [I64, I64, I64, I64, I, I, I,
                                                            ctypes.POINTER(SZ)]
            lib.rmsnorm_rope_bwd_workspace_size.restype = I
            lib.rmsnorm_rope_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, SZ, P, I64, I64, F,
                                             I, I, P]
            lib.rmsnorm_rope_bwd.restype = I
            DBL = ctypes.c_double
            lib.rmsnorm_token_logprob_fwd.argtypes = [P, I64, P, DBL, P, P, I64, I64, I, P]
            lib.rmsnorm_token_logprob_fwd.restype = I
            lib.rmsnorm_token_logprob_bwd.argtypes = [P, I64, P, DBL, P, P, P, P, I64, I64, I64, I,
                                                      P]
            lib.rmsnorm_token_logprob_bwd.restype = I
            lib.rmsnorm_policy_loss_fwd.argtypes = [P, I64, P, DBL, P, P, P, P, F, F, F, P, P, P, P,
                                                    P, P, I64, I64, I64, I, P]
            lib.rmsnorm_policy_loss_fwd.restype = I
            lib.rmsnorm_preference_loss_fwd.argtypes = [P, I64, P, DBL, P, P, I64, F, F, P, P, P, P,
                                                        P, I64, I64, I, P]
            lib.rmsnorm_preference_loss_fwd.restype = I
            lib.rmsnorm_last_error.argtypes = []
            lib.rmsnorm_last_error.restype = ctypes.c_char_p
            lib.rmsnorm_reload_debug_env.argtypes = []
            lib.rmsnorm_reload_debug_env.restype = None
            _lib = lib
    return _lib


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return int(a.data_ptr())


class Heads(ctypes.Structure):
    """A [T, H, D] view of q or k (rmsnorm_heads_t): the device address of its first
    element, the element strides of tokens and heads, and H.  `Heads.of(t)` takes
    them from a torch tensor of that shape whose last dimension is contiguous."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_token", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("heads", ctypes.c_int64)]

    def __init__(self, data, stride_token, stride_head, heads):
        super().__init__(_ptr(data), stride_token, stride_head, heads)
        self._keep = data

    @classmethod
    def of(cls, t):
        if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
            raise ValueError("a [T, H, D] tensor with a contiguous last dimension is wanted")
        return cls(t, t.stride(0), t.stride(1), t.shape[1])


class Rope(ctypes.Structure):
    """Rotary positions (rmsnorm_rope_t).  positions: int64 [axes, T] (or [T] for one
    axis); inv_freq: float32 [rotary_dim / 2]; sections: frequencies per axis; pairs:
    "halves" or "adjacent"; order: "blocks" or "interleaved".  Device tensors (kept
    alive by this object), or raw addresses with positions_stride given."""
    _fields_ = [("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_int64),
                ("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int64),
                ("axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("pairs", ctypes.c_int32), ("order", ctypes.c_int32)]
    _PAIRS = {"halves": 0, "adjacent": 1}
    _ORDERS = {"blocks": 0, "interleaved": 1}

    def __init__(self, positions, inv_freq, sections, rotary_dim, pairs="halves",
                 order="blocks", positions_stride=None):
        sections = tuple(sections)
        if not 1 <= len(sections) <= 4:
            raise ValueError("one to four axes are supported")
        if positions_stride is None:
            if positions.dim() == 2 and positions.shape[0] != len(sections):
                raise ValueError(f"positions must have a row for each of the {len(sections)} axes")
            if positions.dim() not in (1, 2) or (positions.dim() == 1 and len(sections) > 1):
                raise ValueError("positions must be [axes, T], or [T] for one axis")
            if positions.stride(-1) != 1 and positions.shape[-1] > 1:
                raise ValueError("positions must be contiguous along the tokens")
            positions_stride = positions.stride(0) if positions.dim() == 2 else 0
        if hasattr(positions, "dtype") and str(positions.dtype) != "torch.int64":
            raise TypeError(f"positions must be int64, got {positions.dtype}")
        if hasattr(inv_freq, "dtype"):
            if str(inv_freq.dtype) != "torch.float32" or not inv_freq.is_contiguous():
                raise TypeError("inv_freq must be a contiguous float32 tensor")
            if 2 * inv_freq.numel() < rotary_dim:
                raise ValueError(f"inv_freq must hold {rotary_dim // 2} frequencies")
        super().__init__(_ptr(positions), positions_stride, _ptr(inv_freq), rotary_dim,
                         len(sections), (ctypes.c_int32 * 4)(*sections), self._PAIRS[pairs],
                         self._ORDERS[order])
        self._keep = (positions, inv_freq)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _dt(d) -> int:
    """dtype name ("f32", "bf16") or raw code (passed through unchanged)."""
    return _DT_NAMES[d] if isinstance(d, str) else int(d)


def _check(status: int, where: str):
    if status != 0:
        raise RMSNormError(status, where)


def rmsnorm_fwd(x, gamma, y, rstd, M, N, eps, x_dtype, w_dtype, stream=None):
    _check(load_library().rmsnorm_fwd(_ptr(x), _ptr(gamma), _ptr(y), _ptr(rstd), M, N, eps,
                                      _dt(x_dtype), _dt(w_dtype), _stream(stream)),
           "rmsnorm_fwd")


def rmsnorm_fused_add_fwd(x, residual, gamma, y, rstd, M, N, eps, x_dtype, w_dtype,
                          stream=None):
    _check(load_library().rmsnorm_fused_add_fwd(_ptr(x), _ptr(residual), _ptr(gamma), _ptr(y),
                                                _ptr(rstd), M, N, eps, _dt(x_dtype),
                                                _dt(w_dtype), _stream(stream)),
           "rmsnorm_fused_add_fwd")


def rmsnorm_bwd_workspace_size(M, N, x_dtype, w_dtype, device=-1) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().rmsnorm_bwd_workspace_size(M, N, _dt(x_dtype), _dt(w_dtype), device,
                                                     ctypes.byref(out)),
           "rmsnorm_bwd_workspace_size")
    return int(out.value)


def rmsnorm_bwd(dy, x, rstd, gamma, dx, dgamma, workspace, workspace_bytes, M, N, eps, x_dtype,
                w_dtype, stream=None):
    _check(load_library().rmsnorm_bwd(_ptr(dy), _ptr(x), _ptr(rstd), _ptr(gamma), _ptr(dx),
                                      _ptr(dgamma), _ptr(workspace), workspace_bytes, M, N, eps,
                                      _dt(x_dtype), _dt(w_dtype), _stream(stream)),
           "rmsnorm_bwd")


def rmsnorm_fwd_strided(x, x_stride_token, x_stride_head, gamma, y, y_stride_token,
                        y_stride_head, rstd, T, H, D, eps, x_dtype, w_dtype, stream=None):
    _check(load_library().rmsnorm_fwd_strided(_ptr(x), x_stride_token, x_stride_head,
                                              _ptr(gamma), _ptr(y), y_stride_token,
                                              y_stride_head, _ptr(rstd), T, H, D, eps,
                                              _dt(x_dtype), _dt(w_dtype), _stream(stream)),
           "rmsnorm_fwd_strided")


def layernorm_fwd(x, gamma, beta, y, mean, rstd, M, N, eps, x_dtype, w_dtype, stream=None):
    _check(load_library().layernorm_fwd(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean),
                                        _ptr(rstd), M, N, eps, _dt(x_dtype), _dt(w_dtype),
                                        _stream(stream)),
           "layernorm_fwd")


def layernorm_bwd_workspace_size(M, N, x_dtype, w_dtype, device=-1):
    n = ctypes.c_size_t(0)
    _check(load_library().layernorm_bwd_workspace_size(M, N, _dt(x_dtype), _dt(w_dtype), device,
                                                       ctypes.byref(n)),
           "layernorm_bwd_workspace_size")
    return int(n.value)


def layernorm_bwd(dy, x, mean, rstd, gamma, dx, dgamma, dbeta, workspace, workspace_bytes, M, N,
                  eps, x_dtype, w_dtype, stream=None):
    _check(load_library().layernorm_bwd(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(gamma),
                                        _ptr(dx), _ptr(dgamma), _ptr(dbeta), _ptr(workspace),
                                        workspace_bytes, M, N, eps, _dt(x_dtype), _dt(w_dtype),
                                        _stream(stream)),
           "layernorm_bwd")


def rmsnorm_fwd_fp8(x, residual, gamma, q, scale, rstd, M, N, eps, x_dtype, w_dtype,
                    stream=None):
    _check(load_library().rmsnorm_fwd_fp8(_ptr(x), _ptr(residual), _ptr(gamma), _ptr(q),
                                          _ptr(scale), _ptr(rstd), M, N, eps, _dt(x_dtype),
                                          _dt(w_dtype), _stream(stream)),
           "rmsnorm_fwd_fp8")


def rmsnorm_fwd_nvfp4(x, residual, gamma, global_scale, q, block_scale, rstd, M, N, eps,
                      x_dtype, w_dtype, stream=None):
    _check(load_library().rmsnorm_fwd_nvfp4(_ptr(x), _ptr(residual), _ptr(gamma),
                                            float(global_scale), _ptr(q), _ptr(block_scale),
                                            _ptr(rstd), M, N, eps, _dt(x_dtype), _dt(w_dtype),
                                            _stream(stream)),
           "rmsnorm_fwd_nvfp4")


def rmsnorm_fused_add_bwd(dy, h, rstd, gamma, dres, dgamma, dgamma_dtype, workspace,
                          workspace_bytes, M, N, eps, x_dtype, w_dtype, stream=None):
    _check(load_library().rmsnorm_fused_add_bwd(_ptr(dy), _ptr(h), _ptr(rstd), _ptr(gamma),
                                                _ptr(dres), _ptr(dgamma), _dt(dgamma_dtype),
                                                _ptr(workspace), workspace_bytes, M, N, eps,
                                                _dt(x_dtype), _dt(w_dtype), _stream(stream)),
           "rmsnorm_fused_add_bwd")


def rmsnorm_bwd_noalloc(dy, x, rstd, gamma, dx, dgamma, M, N, eps, x_dtype, w_dtype,
                        stream=None):
    """rmsnorm_bwd without a workspace argument: for callers that cannot
    allocate, the dgamma partials use a scratch array owned by the library
    (see include/rmsnorm.h for its limit and sharing rules)."""
    _check(load_library().rmsnorm_bwd_noalloc(_ptr(dy), _ptr(x), _ptr(rstd), _ptr(gamma),
                                              _ptr(dx), _ptr(dgamma), M, N, eps, _dt(x_dtype),
                                              _dt(w_dtype), _stream(stream)),
           "rmsnorm_bwd_noalloc")


def rmsnorm_rope_fwd(q, k, q_gamma, k_gamma, q_out, k_out, rope, T, D, eps, x_dtype, w_dtype,
                     stream=None):
    """Rotary positions over q and k ([T, H, D] views as Heads; k may be None),
    behind the per-head RMSNorm unless both gammas are None."""
    _check(load_library().rmsnorm_rope_fwd(_ref(q), _ref(k), _ptr(q_gamma), _ptr(k_gamma),
                                           _ref(q_out), _ref(k_out), _ref(rope), T, D, eps,
                                           _dt(x_dtype), _dt(w_dtype), _stream(stream)),
           "rmsnorm_rope_fwd")


def rmsnorm_rope_bwd_workspace_size(T, q_heads, k_heads, D, x_dtype, w_dtype, device=-1) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().rmsnorm_rope_bwd_workspace_size(T, q_heads, k_heads, D, _dt(x_dtype),
                                                          _dt(w_dtype), device,
                                                          ctypes.byref(out)),
           "rmsnorm_rope_bwd_workspace_size")
    return int(out.value)


def rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_gamma, k_gamma, dq, dk, dq_gamma, dk_gamma,
                     workspace, workspace_bytes, rope, T, D, eps, x_dtype, w_dtype, stream=None):
    _check(load_library().rmsnorm_rope_bwd(_ref(dq_out), _ref(dk_out), _ref(q), _ref(k),
                                           _ptr(q_gamma), _ptr(k_gamma), _ref(dq), _ref(dk),
                                           _ptr(dq_gamma), _ptr(dk_gamma), _ptr(workspace),
                                           workspace_bytes, _ref(rope), T, D, eps, _dt(x_dtype),
                                           _dt(w_dtype), _stream(stream)),
           "rmsnorm_rope_bwd")


def rmsnorm_token_logprob_fwd(logits, ld, targets, inv_temperature, logp, rel_lse, M, V, x_dtype,
                              stream=None):
    """logp, and rel_lse for the backward, of each row's target token (rows of V logits,
    row stride ld)."""
    _check(load_library().rmsnorm_token_logprob_fwd(_ptr(logits), ld, _ptr(targets),
                                                    inv_temperature, _ptr(logp), _ptr(rel_lse),
                                                    M, V, _dt(x_dtype), _stream(stream)),
           "rmsnorm_token_logprob_fwd")


def rmsnorm_token_logprob_bwd(logits, ld, targets, inv_temperature, rel_lse, dlogp, scale, dlogits,
                              ld_out, M, V, x_dtype, stream=None):
    """The logits' gradient from dlogp (times the device scalar `scale`, None for 1)."""
    _check(load_library().rmsnorm_token_logprob_bwd(_ptr(logits), ld, _ptr(targets),
                                                    inv_temperature, _ptr(rel_lse), _ptr(dlogp),
                                                    _ptr(scale), _ptr(dlogits), ld_out, M, V,
                                                    _dt(x_dtype), _stream(stream)),
           "rmsnorm_token_logprob_bwd")


def rmsnorm_policy_loss_fwd(logits, ld, targets, inv_temperature, old_logp, ref_logp, advantages,
                            weights, clip_low, clip_high, kl_coef, loss, token_loss, logp, rel_lse,
                            dlogp, dlogits, ld_out, M, V, x_dtype, stream=None):
    """Clipped policy loss; dlogits (None to skip) takes its gradient in the same pass."""
    _check(load_library().rmsnorm_policy_loss_fwd(
        _ptr(logits), ld, _ptr(targets), inv_temperature, _ptr(old_logp), _ptr(ref_logp),
        _ptr(advantages), _ptr(weights), clip_low, clip_high, kl_coef, _ptr(loss),
        _ptr(token_loss), _ptr(logp), _ptr(rel_lse), _ptr(dlogp), _ptr(dlogits), ld_out, M, V,
        _dt(x_dtype), _stream(stream)), "rmsnorm_policy_loss_fwd")


def rmsnorm_preference_loss_fwd(logits, ld, targets, inv_temperature, ref_logp, cu_seqlens, pairs,
                                beta, label_smoothing, loss, margins, logp, rel_lse, dlogp, M, V,
                                x_dtype, stream=None):
    """Preference loss over pairs of sequences (chosen first, then rejected)."""
    _check(load_library().rmsnorm_preference_loss_fwd(
        _ptr(logits), ld, _ptr(targets), inv_temperature, _ptr(ref_logp), _ptr(cu_seqlens), pairs,
        beta, label_smoothing, _ptr(loss), _ptr(margins), _ptr(logp), _ptr(rel_lse), _ptr(dlogp), M,
        V, _dt(x_dtype), _stream(stream)), "rmsnorm_preference_loss_fwd")


def rmsnorm_check_device(stream=None):
    """Wait for `stream`, then raise RMSNormError(RMSNORM_ERR_TIMEOUT) if a
    kernel on the current device gave up a bounded wait (clears the flag)."""
    _check(load_library().rmsnorm_check_device(_stream(stream)), "rmsnorm_check_device")


def rmsnorm_reload_debug_env():
    """Re-read RMSNORM_FORCE_VARIANT, RMSNORM_WAIT_LIMIT_CYCLES and
    RMSNORM_NO_PDL from the environment (the library reads them once at load;
    call this after changing them, with no other thread inside the library)."""
    load_library().rmsnorm_reload_debug_env()


def rmsnorm_last_error() -> str:
    """The failing CUDA call behind this thread's last RMSNORM_ERR_CUDA."""
    try:
        return load_library().rmsnorm_last_error().decode()
    except ImportError:
        return ""


def rmsnorm_status_string(status: int) -> str:
    try:
        return load_library().rmsnorm_status_string(status).decode()
    except ImportError:
        return f"status {status}"


def rmsnorm_describe_plan(op, M, N, x_dtype, w_dtype, aligned16=True, device=-1) -> str:
    """aligned16: True / False, or "mixed" (ops 0-3: outputs on 16 bytes, x and
    dy off them)."""
    buf = ctypes.create_string_buffer(256)
    a = 2 if aligned16 == "mixed" else (1 if aligned16 else 0)
    _check(load_library().rmsnorm_describe_plan(op, M, N, _dt(x_dtype), _dt(w_dtype),
                                                a, device, buf, 256),
           "rmsnorm_describe_plan")
    return buf.value.decode()
