"""Thin ctypes binding of libdeltanet.so (argument marshalling only).

Every step of the computation runs in the library's HIP kernels; this module
checks tensors (device, dtype, contiguity, shape), allocates outputs and the
workspace through PyTorch's caching allocator (on the launch stream, and
recorded on the current one when that is another), and passes raw device
pointers and the HIP stream (the current one unless ``stream=`` names another)
to the C ABI.  If the library is missing it raises: there is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdeltanet.so")

DN_OK = 0
DN_F32 = 0
DN_BF16 = 1
STATUS_NAMES = {0: "DN_OK", 1: "DN_ERR_NULL_ARG", 2: "DN_ERR_BAD_SHAPE", 3: "DN_ERR_UNSUPPORTED",
                4: "DN_ERR_MISALIGNED", 5: "DN_ERR_ALIASING", 6: "DN_ERR_WORKSPACE",
                7: "DN_ERR_HIP"}
# Every symbol include/deltanet.h declares.
EXPORTS = ("deltanet_chunk_fwd", "deltanet_chunk_fwd_workspace_bytes", "deltanet_decode_step",
           "deltanet_gated_chunk_fwd", "deltanet_gated_chunk_fwd_workspace_bytes",
           "deltanet_gated_decode_step", "deltanet_feature_prep", "deltanet_chunk_fwd_features",
           "deltanet_chunk_fwd_features_workspace_bytes", "deltanet_decode_step_features",
           "deltanet_kda_chunk_fwd", "deltanet_kda_chunk_fwd_workspace_bytes",
           "deltanet_kda_decode_step", "deltanet_chunk_bwd", "deltanet_chunk_bwd_workspace_bytes",
           "deltanet_status_string", "deltanet_last_hip_error", "deltanet_version",
           "deltanet_profile_start", "deltanet_profile_stop", "deltanet_chunk_fwd_noalloc",
           "deltanet_linear_chunk_fwd", "deltanet_linear_chunk_fwd_workspace_bytes",
           "deltanet_linear_chunk_bwd", "deltanet_linear_chunk_bwd_workspace_bytes",
           "deltanet_linear_decode_step", "deltanet_qk_norm_rope", "deltanet_qk_norm_rope_bwd",
           "deltanet_qk_norm_rope_bwd_workspace_bytes")
PROFILE_SLOTS = ("chunk_prep", "chunk_scan", "decode", "features", "bwd_prep", "bwd_fwd_scan",
                 "bwd_scan", "bwd_cc", "bwd_qk", "linear_state", "linear_out", "linear_bwd",
                 "linear_decode", "qk_norm_rope", "qk_norm_rope_bwd")

_lib = None


class DeltaNetError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({detail})")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once and declare its C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m deltanet_delta_rule_chunk_amd.build`"
            " (there is no non-HIP fallback)")
    lib = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.deltanet_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, sz, vp]
    lib.deltanet_chunk_fwd.restype = i
    lib.deltanet_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                               vp]
    lib.deltanet_chunk_fwd_noalloc.restype = i
    lib.deltanet_chunk_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.deltanet_chunk_fwd_workspace_bytes.restype = sz
    lib.deltanet_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.deltanet_decode_step.restype = i
    lib.deltanet_gated_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                             vp, sz, vp]
    lib.deltanet_gated_chunk_fwd.restype = i
    lib.deltanet_gated_chunk_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.deltanet_gated_chunk_fwd_workspace_bytes.restype = sz
    lib.deltanet_gated_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.deltanet_gated_decode_step.restype = i
    lib.deltanet_feature_prep.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.deltanet_feature_prep.restype = i
    lib.deltanet_chunk_fwd_features.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                                i, i, vp, sz, vp]
    lib.deltanet_chunk_fwd_features.restype = i
    lib.deltanet_chunk_fwd_features_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.deltanet_chunk_fwd_features_workspace_bytes.restype = sz
    lib.deltanet_decode_step_features.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.deltanet_decode_step_features.restype = i
    lib.deltanet_kda_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                           vp, sz, vp]
    lib.deltanet_kda_chunk_fwd.restype = i
    lib.deltanet_kda_chunk_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.deltanet_kda_chunk_fwd_workspace_bytes.restype = sz
    lib.deltanet_kda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
    lib.deltanet_kda_decode_step.restype = i
    lib.deltanet_chunk_bwd.argtypes = [vp] * 12 + [i] * 7 + [vp, sz, vp]
    lib.deltanet_chunk_bwd.restype = i
    lib.deltanet_chunk_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.deltanet_chunk_bwd_workspace_bytes.restype = sz
    f = ctypes.c_float
    lib.deltanet_linear_chunk_fwd.argtypes = [vp] * 7 + [i] * 8 + [vp, sz, vp]
    lib.deltanet_linear_chunk_fwd.restype = i
    lib.deltanet_linear_chunk_bwd.argtypes = [vp] * 12 + [i] * 7 + [vp, sz, vp]
    lib.deltanet_linear_chunk_bwd.restype = i
    lib.deltanet_linear_decode_step.argtypes = [vp] * 6 + [i] * 7 + [vp]
    lib.deltanet_linear_decode_step.restype = i
    lib.deltanet_qk_norm_rope.argtypes = [vp] * 9 + [i] + [vp] * 2 + [i] * 8 + [f, i, vp]
    lib.deltanet_qk_norm_rope.restype = i
    lib.deltanet_qk_norm_rope_bwd.argtypes = ([vp] * 9 + [i] + [vp] * 8 + [i] * 8
                                              + [f, i, vp, sz, vp])
    lib.deltanet_qk_norm_rope_bwd.restype = i
    for name in ("linear_chunk_fwd", "linear_chunk_bwd"):
        fn = getattr(lib, f"deltanet_{name}_workspace_bytes")
        fn.argtypes, fn.restype = [i] * 7, sz
    lib.deltanet_qk_norm_rope_bwd_workspace_bytes.argtypes = [i] * 6
    lib.deltanet_qk_norm_rope_bwd_workspace_bytes.restype = sz
    lib.deltanet_status_string.argtypes = [i]
    lib.deltanet_status_string.restype = ctypes.c_char_p
    lib.deltanet_last_hip_error.argtypes = []
    lib.deltanet_last_hip_error.restype = i
    lib.deltanet_version.argtypes = []
    lib.deltanet_version.restype = i
    lib.deltanet_profile_start.argtypes = []
    lib.deltanet_profile_start.restype = i
    lib.deltanet_profile_stop.argtypes = [ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(ctypes.c_int), i]
    lib.deltanet_profile_stop.restype = i
    _lib = lib
    return lib


_CODES = {torch.float32: DN_F32, torch.bfloat16: DN_BF16}


def _code(dt: torch.dtype) -> int:
    code = _CODES.get(dt)
    if code is not None:
        return code
    raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, shape, dtype=None, device=None):
    # One look for tensors that are right; the reasons only for those that are not.
    if (type(t) is torch.Tensor and t.shape == shape and t.device == device
            and (dtype is None or t.dtype is dtype) and t.is_contiguous() and t.is_cuda):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raise(lib, status: int, what: str):
    detail = lib.deltanet_status_string(status).decode()
    if status == 7:
        detail += f"; hipError {lib.deltanet_last_hip_error()}"
    raise DeltaNetError(status, what, detail)


# The current stream's handle without a Stream object around it (1.7 us less
# per call), where this PyTorch has it.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None and device.index is not None:
        return _current_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _alloc(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """A new tensor from PyTorch's caching allocator, of the stream that the
    kernels run on: a block of the current stream may still be in use there by
    work that the other one does not wait for.  It is recorded on the current
    stream as well, where the caller may read it last, so that it is not handed
    out again before that."""
    if stream is None or stream == torch.cuda.current_stream(device):
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def workspace_bytes(B: int, H: int, L: int, d_k: int, d_v: int, C: int,
                    in_dtype: torch.dtype = torch.bfloat16, gated: bool = False,
                    features: bool = False) -> int:
    lib = load()
    if features:
        return int(lib.deltanet_chunk_fwd_features_workspace_bytes(B, H, L, d_k, d_v, C,
                                                                    _code(in_dtype), int(gated)))
    fn = lib.deltanet_gated_chunk_fwd_workspace_bytes if gated else lib.deltanet_chunk_fwd_workspace_bytes
    return int(fn(B, H, L, d_k, d_v, C, _code(in_dtype)))


def bwd_workspace_bytes(B: int, H: int, L: int, d_k: int, d_v: int, C: int = 64,
                        in_dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().deltanet_chunk_bwd_workspace_bytes(B, H, L, d_k, d_v, C, _code(in_dtype)))


def chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
              S0: Optional[torch.Tensor], dO: torch.Tensor, dS_final: Optional[torch.Tensor] = None,
              C: int = 64, *, want_dS0: bool = True, workspace: Optional[torch.Tensor] = None,
              stream=None):
    """Gradient of the chunked forward (``deltanet_chunk_bwd``).  q,k ``[B,H,L,d_k]``,
    v ``[B,H,L,d_v]`` (fp32 or bf16), beta ``[B,H,L]``, S0 ``[B,H,d_k,d_v]`` or None,
    dO ``[B,H,L,d_v]`` fp32, dS_final ``[B,H,d_k,d_v]`` fp32 or None.  Returns fp32
    ``(dq, dk, dv, dbeta, dS0)`` (dS0 None when ``want_dS0`` is False)."""
    lib = load()
    B, H, L, d_k = q.shape
    d_v = v.shape[-1]
    dev = q.device
    _check(q, "q", (B, H, L, d_k), device=dev)
    _check(k, "k", (B, H, L, d_k), q.dtype, dev)
    _check(v, "v", (B, H, L, d_v), q.dtype, dev)
    _check(beta, "beta", (B, H, L), torch.float32, dev)
    _check(dO, "dO", (B, H, L, d_v), torch.float32, dev)
    for t, n in ((S0, "S0"), (dS_final, "dS_final")):
        if t is not None:
            _check(t, n, (B, H, d_k, d_v), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev, stream=stream)
    dq, dk = _alloc((B, H, L, d_k), **f32), _alloc((B, H, L, d_k), **f32)
    dv, db = _alloc((B, H, L, d_v), **f32), _alloc((B, H, L), **f32)
    dS0 = _alloc((B, H, d_k, d_v), **f32) if want_dS0 else None
    need = bwd_workspace_bytes(B, H, L, d_k, d_v, C, q.dtype)
    if workspace is None and need > 0:
        workspace = _alloc(need, torch.uint8, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.deltanet_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(dO),
                                _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(db), _ptr(dS0),
                                B, H, L, d_k, d_v, C, _code(q.dtype), _ptr(workspace), ws_bytes,
                                _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_chunk_bwd")
    return dq, dk, dv, db, dS0


class _DeltaRule(torch.autograd.Function):
    """``chunk_fwd`` (fp32 o) with its gradient from ``chunk_bwd``.  Only the
    inputs are kept for the backward, which recomputes the forward inside the
    library.  The gradients come back in fp32; autograd casts them to the
    inputs' dtype."""

    @staticmethod
    def forward(ctx, q, k, v, beta, S0, C):
        o, S_final = chunk_fwd(q, k, v, beta, S0, C)
        ctx.save_for_backward(q, k, v, beta, S0)
        ctx.C = C
        return o, S_final

    @staticmethod
    def backward(ctx, dO, dS_final):
        q, k, v, beta, S0 = ctx.saved_tensors
        want_dS0 = S0 is not None and ctx.needs_input_grad[4]
        dq, dk, dv, db, dS0 = chunk_bwd(q, k, v, beta, S0, dO.contiguous(), dS_final.contiguous(),
                                        ctx.C, want_dS0=want_dS0)
        return dq, dk, dv, db, dS0, None


def delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
               S0: Optional[torch.Tensor] = None, C: int = 64
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable chunked delta-rule forward for training: ``(o, S_final)``
    as ``chunk_fwd`` returns them (o in fp32), with gradients for q, k, v,
    beta and S0 from ``deltanet_chunk_bwd``."""
    return _DeltaRule.apply(q, k, v, beta, S0, C)


def kda_workspace_bytes(B: int, H: int, L: int, d_k: int, d_v: int, C: int = 64,
                        in_dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load().deltanet_kda_chunk_fwd_workspace_bytes(B, H, L, d_k, d_v, C,
                                                             _code(in_dtype)))


def kda_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                  beta: torch.Tensor, S0: Optional[torch.Tensor] = None, C: int = 64, *,
                  out_dtype: torch.dtype = torch.float32, o: Optional[torch.Tensor] = None,
                  S_final: Optional[torch.Tensor] = None, want_state: bool = True,
                  workspace: Optional[torch.Tensor] = None, stream=None
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked forward with per-dimension decay (``deltanet_kda_chunk_fwd``):
    ``chunk_fwd``'s arguments with alpha ``[B,H,L,d_k]`` fp32."""
    lib = load()
    B, H, L, d_k = q.shape
    d_v = v.shape[-1]
    dev = q.device
    _check(q, "q", (B, H, L, d_k), device=dev)
    _check(k, "k", (B, H, L, d_k), q.dtype, dev)
    _check(v, "v", (B, H, L, d_v), q.dtype, dev)
    _check(alpha, "alpha", (B, H, L, d_k), torch.float32, dev)
    _check(beta, "beta", (B, H, L), torch.float32, dev)
    if S0 is not None:
        _check(S0, "S0", (B, H, d_k, d_v), torch.float32, dev)
    if o is None:
        o = _alloc((B, H, L, d_v), out_dtype, dev, stream)
    _check(o, "o", (B, H, L, d_v), out_dtype, dev)
    if S_final is None and want_state:
        S_final = _alloc((B, H, d_k, d_v), torch.float32, dev, stream)
    if S_final is not None:
        _check(S_final, "S_final", (B, H, d_k, d_v), torch.float32, dev)
    need = kda_workspace_bytes(B, H, L, d_k, d_v, C, q.dtype)
    if workspace is None and need > 0:
        workspace = _alloc(need, torch.uint8, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.deltanet_kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                                    _ptr(o), _ptr(S_final), B, H, L, d_k, d_v, C, _code(q.dtype),
                                    _code(out_dtype), _ptr(workspace), ws_bytes,
                                    _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_kda_chunk_fwd")
    return o, S_final


def kda_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                    beta: torch.Tensor, S: torch.Tensor, *, out_dtype: torch.dtype = torch.float32,
                    o: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode step with per-dimension decay (``deltanet_kda_decode_step``):
    alpha ``[B,H,d_k]`` fp32; S updated in place; returns o = q S_new."""
    lib = load()
    B, H, d_k = q.shape
    d_v = v.shape[-1]
    dev = q.device
    _check(q, "q", (B, H, d_k), device=dev)
    _check(k, "k", (B, H, d_k), q.dtype, dev)
    _check(v, "v", (B, H, d_v), q.dtype, dev)
    _check(alpha, "alpha", (B, H, d_k), torch.float32, dev)
    _check(beta, "beta", (B, H), torch.float32, dev)
    _check(S, "S", (B, H, d_k, d_v), torch.float32, dev)
    if o is None:
        o = _alloc((B, H, d_v), out_dtype, dev, stream)
    _check(o, "o", (B, H, d_v), out_dtype, dev)
    st = lib.deltanet_kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S),
                                      _ptr(o), B, H, d_k, d_v, _code(q.dtype), _code(out_dtype),
                                      _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_kda_decode_step")
    return o


def feature_prep(q_raw: torch.Tensor, k_raw: torch.Tensor, beta_logit: torch.Tensor, *,
                 in_place: bool = False, stream=None
                 ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The layer's feature maps: ``normalise(silu(q_raw))``, ``normalise(silu(k_raw))``
    (``[B,H,L,d_k]``, same dtype as the inputs) and ``sigmoid(beta_logit)``
    (``[B,H,L]`` fp32), by ``deltanet_feature_prep``.  ``in_place`` writes the
    results over the inputs."""
    lib = load()
    B, H, L, d_k = q_raw.shape
    dev = q_raw.device
    _check(q_raw, "q_raw", (B, H, L, d_k), device=dev)
    _check(k_raw, "k_raw", (B, H, L, d_k), q_raw.dtype, dev)
    _check(beta_logit, "beta_logit", (B, H, L), torch.float32, dev)
    if in_place:
        qh, kh, b = q_raw, k_raw, beta_logit
    else:
        qh = _alloc(q_raw.shape, q_raw.dtype, dev, stream)
        kh = _alloc(k_raw.shape, k_raw.dtype, dev, stream)
        b = _alloc(beta_logit.shape, beta_logit.dtype, dev, stream)
    st = lib.deltanet_feature_prep(_ptr(q_raw), _ptr(k_raw), _ptr(beta_logit), _ptr(qh), _ptr(kh),
                                   _ptr(b), B, H, L, d_k, _code(q_raw.dtype), _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_feature_prep")
    return qh, kh, b


def chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
              S0: Optional[torch.Tensor] = None, C: int = 64, *,
              out_dtype: torch.dtype = torch.float32, o: Optional[torch.Tensor] = None,
              S_final: Optional[torch.Tensor] = None, want_state: bool = True,
              workspace: Optional[torch.Tensor] = None, stream=None,
              alpha: Optional[torch.Tensor] = None, features: bool = False
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked delta-rule forward.  q,k ``[B,H,L,d_k]``, v ``[B,H,L,d_v]`` (fp32 or
    bf16, same dtype), beta ``[B,H,L]`` fp32, S0 ``[B,H,d_k,d_v]`` fp32 or None.
    With ``alpha`` (``[B,H,L]`` fp32) the gated form runs
    (``deltanet_gated_chunk_fwd``).  With ``features`` q, k are the raw
    projections and beta the logits, mapped by the layer's feature maps first
    (``deltanet_chunk_fwd_features``).  Returns ``(o, S_final)``; S_final is
    None when ``want_state`` is False."""
    lib = load()
    B, H, L, d_k = q.shape
    d_v = v.shape[-1]
    dev = q.device
    _check(q, "q", (B, H, L, d_k), device=dev)
    _check(k, "k", (B, H, L, d_k), q.dtype, dev)
    _check(v, "v", (B, H, L, d_v), q.dtype, dev)
    _check(beta, "beta", (B, H, L), torch.float32, dev)
    if alpha is not None:
        _check(alpha, "alpha", (B, H, L), torch.float32, dev)
    if S0 is not None:
        _check(S0, "S0", (B, H, d_k, d_v), torch.float32, dev)
    if o is None:
        o = _alloc((B, H, L, d_v), out_dtype, dev, stream)
    _check(o, "o", (B, H, L, d_v), out_dtype, dev)
    if S_final is None and want_state:
        S_final = _alloc((B, H, d_k, d_v), torch.float32, dev, stream)
    if S_final is not None:
        _check(S_final, "S_final", (B, H, d_k, d_v), torch.float32, dev)
    in_code = _code(q.dtype)
    need = workspace_bytes(B, H, L, d_k, d_v, C, q.dtype, gated=alpha is not None,
                           features=features)
    if workspace is None and need > 0:
        workspace = _alloc(need, torch.uint8, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if features:
        st = lib.deltanet_chunk_fwd_features(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                             _ptr(S0), _ptr(o), _ptr(S_final), B, H, L, d_k, d_v,
                                             C, in_code, _code(out_dtype), _ptr(workspace),
                                             ws_bytes, _stream(dev, stream))
        if st != DN_OK:
            _raise(lib, st, "deltanet_chunk_fwd_features")
    elif alpha is None:
        st = lib.deltanet_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(o),
                                    _ptr(S_final), B, H, L, d_k, d_v, C, in_code,
                                    _code(out_dtype), _ptr(workspace), ws_bytes,
                                    _stream(dev, stream))
        if st != DN_OK:
            _raise(lib, st, "deltanet_chunk_fwd")
    else:
        st = lib.deltanet_gated_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                          _ptr(S0), _ptr(o), _ptr(S_final), B, H, L, d_k, d_v, C,
                                          in_code, _code(out_dtype), _ptr(workspace), ws_bytes,
                                          _stream(dev, stream))
        if st != DN_OK:
            _raise(lib, st, "deltanet_gated_chunk_fwd")
    return o, S_final


def gated_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                    beta: torch.Tensor, S0: Optional[torch.Tensor] = None, C: int = 64, **kw
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated (Gated DeltaNet) chunked forward: ``chunk_fwd`` with a per-token
    decay alpha ``[B,H,L]`` fp32 applied to the state before each write."""
    return chunk_fwd(q, k, v, beta, S0, C, alpha=alpha, **kw)


def decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                S: torch.Tensor, *, out_dtype: torch.dtype = torch.float32,
                o: Optional[torch.Tensor] = None, stream=None,
                alpha: Optional[torch.Tensor] = None, features: bool = False) -> torch.Tensor:
    """One decode step; updates S ``[B,H,d_k,d_v]`` in place and returns o
    ``[B,H,d_v]`` = q S_new.  With ``alpha`` (``[B,H]`` fp32) the gated step
    runs (``deltanet_gated_decode_step``).  With ``features`` q, k are the raw
    projections and beta the logits, mapped inside the step's kernel
    (``deltanet_decode_step_features``)."""
    lib = load()
    B, H, d_k = q.shape
    d_v = v.shape[-1]
    dev = q.device
    _check(q, "q", (B, H, d_k), device=dev)
    _check(k, "k", (B, H, d_k), q.dtype, dev)
    _check(v, "v", (B, H, d_v), q.dtype, dev)
    _check(beta, "beta", (B, H), torch.float32, dev)
    _check(S, "S", (B, H, d_k, d_v), torch.float32, dev)
    if o is None:
        o = _alloc((B, H, d_v), out_dtype, dev, stream)
    _check(o, "o", (B, H, d_v), out_dtype, dev)
    if alpha is not None:
        _check(alpha, "alpha", (B, H), torch.float32, dev)
    if features:
        st = lib.deltanet_decode_step_features(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                               _ptr(S), _ptr(o), B, H, d_k, d_v, _code(q.dtype),
                                               _code(out_dtype), _stream(dev, stream))
        if st != DN_OK:
            _raise(lib, st, "deltanet_decode_step_features")
    elif alpha is None:
        st = lib.deltanet_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S), _ptr(o),
                                      B, H, d_k, d_v, _code(q.dtype), _code(out_dtype),
                                      _stream(dev, stream))
        if st != DN_OK:
            _raise(lib, st, "deltanet_decode_step")
    else:
        st = lib.deltanet_gated_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                            _ptr(S), _ptr(o), B, H, d_k, d_v, _code(q.dtype),
                                            _code(out_dtype), _stream(dev, stream))
        if st != DN_OK:
            _raise(lib, st, "deltanet_gated_decode_step")
    return o


def gated_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                      beta: torch.Tensor, S: torch.Tensor, **kw) -> torch.Tensor:
    """Gated decode step: ``decode_step`` with the per-(b, h) decay alpha."""
    return decode_step(q, k, v, beta, S, alpha=alpha, **kw)


def _elsewhere(device: torch.device) -> bool:
    """Whether the device is not the current one (a null stream names the
    current device's, so a call on its tensors has to make it current)."""
    return device.type == "cuda" and device.index != torch.cuda.current_device()


@functools.lru_cache(maxsize=1024)
def linear_workspace_bytes(B: int, H: int, L: int, d_k: int, d_v: int,
                           in_dtype: torch.dtype = torch.bfloat16, H_qk: Optional[int] = None,
                           backward: bool = False) -> int:
    """Workspace of ``linear_chunk_fwd`` (``linear_chunk_bwd``) for these sizes."""
    lib = load()
    fn = (lib.deltanet_linear_chunk_bwd_workspace_bytes if backward
          else lib.deltanet_linear_chunk_fwd_workspace_bytes)
    return int(fn(B, H, H if H_qk is None else H_qk, L, d_k, d_v, _code(in_dtype)))


def _workspace(given: Optional[torch.Tensor], need: int, device: torch.device, stream):
    """(tensor or None, pointer, bytes) of the caller's workspace or a new one."""
    if given is None:
        if need == 0:
            return None, None, 0
        given = _alloc(need, torch.uint8, device, stream)
    elif given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return given, given.data_ptr(), given.numel() * given.element_size()


def _check_linear(q, k, v, log_decay, states, dims):
    """Shapes of the gated linear recurrence's inputs, ``[B, H, L, d]`` or (one
    token, ``dims`` = 3) ``[B, H, d]``; ``states`` are (tensor or None, name)
    pairs.  Returns (B, H, H_qk, d_k, d_v)."""
    qs, vs = q.shape, v.shape
    if len(qs) != dims or len(vs) != dims:
        raise ValueError(f"q and v must have {dims} dimensions (got {tuple(qs)}, {tuple(vs)})")
    dev, dt = q.device, q.dtype
    B, H_qk, H, d_k, d_v = qs[0], qs[1], vs[1], qs[-1], vs[-1]
    state = (B, H, d_k, d_v)
    # One look at everything; the reasons only where something is wrong.
    good = (q.is_cuda and k.shape == qs and k.dtype is dt and v.dtype is dt and vs[0] == B
            and vs[2:-1] == qs[2:-1] and k.device == dev and v.device == dev
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
            and (log_decay is None or (log_decay.shape == vs[:-1] and log_decay.device == dev
                                       and log_decay.dtype is torch.float32
                                       and log_decay.is_contiguous())))
    if good:
        for t, _ in states:
            if t is not None and not (t.shape == state and t.dtype is torch.float32
                                      and t.device == dev and t.is_contiguous()):
                good = False
    if not good:
        tok = tuple(qs[2:-1])
        _check(q, "q", (B, H_qk, *tok, d_k), device=dev)
        _check(k, "k", (B, H_qk, *tok, d_k), dt, dev)
        _check(v, "v", (B, H, *tok, d_v), dt, dev)
        if log_decay is not None:
            _check(log_decay, "log_decay", (B, H, *tok), torch.float32, dev)
        for t, n in states:
            if t is not None:
                _check(t, n, state, torch.float32, dev)
    return B, H, H_qk, d_k, d_v


def linear_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     log_decay: Optional[torch.Tensor] = None, S0: Optional[torch.Tensor] = None,
                     *, out_dtype: torch.dtype = torch.float32, o: Optional[torch.Tensor] = None,
                     S_final: Optional[torch.Tensor] = None, want_state: bool = True,
                     workspace: Optional[torch.Tensor] = None, stream=None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence over a sequence (``deltanet_linear_chunk_fwd``):
    ``S = e^g S + k^T v``, ``o = q S``.  q,k ``[B,H_qk,L,d_k]``, v ``[B,H,L,d_v]``
    (fp32 or bf16, same dtype; H a multiple of H_qk, head h reads q and k of
    head ``h // (H // H_qk)``), log_decay ``[B,H,L]`` fp32 (``-inf`` wipes the
    state exactly) or None, S0 ``[B,H,d_k,d_v]`` fp32 or None.  Returns
    ``(o, S_final)``; S_final is None when ``want_state`` is False."""
    lib = _lib or load()
    B, H, H_qk, d_k, d_v = _check_linear(q, k, v, log_decay, ((S0, "S0"), (S_final, "S_final")), 4)
    dev, L = q.device, q.shape[2]
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return linear_chunk_fwd(q, k, v, log_decay, S0, out_dtype=out_dtype, o=o,
                                    S_final=S_final, want_state=want_state, workspace=workspace,
                                    stream=stream)
    if o is None:
        o = _alloc((B, H, L, d_v), out_dtype, dev, stream)
    else:
        _check(o, "o", (B, H, L, d_v), out_dtype, dev)
    if S_final is None and want_state:
        S_final = _alloc((B, H, d_k, d_v), torch.float32, dev, stream)
    need = linear_workspace_bytes(B, H, L, d_k, d_v, q.dtype, H_qk)
    keep, ws, ws_bytes = _workspace(workspace, need, dev, stream)
    st = lib.deltanet_linear_chunk_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(log_decay),
                                       _ptr(S0), o.data_ptr(), _ptr(S_final), B, H, H_qk, L, d_k,
                                       d_v, _code(q.dtype), _code(out_dtype), ws, ws_bytes,
                                       _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_linear_chunk_fwd")
    return o, S_final


def linear_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     log_decay: Optional[torch.Tensor], S0: Optional[torch.Tensor],
                     dO: torch.Tensor, dS_final: Optional[torch.Tensor] = None, *,
                     want_dS0: bool = True, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of ``linear_chunk_fwd`` (``deltanet_linear_chunk_bwd``) from dO
    ``[B,H,L,d_v]`` (the inputs' dtype) and dS_final ``[B,H,d_k,d_v]`` fp32 or
    None.  Returns ``(dq, dk, dv, dlog_decay, dS0)``: dq, dk, dv in the inputs'
    dtype, dlog_decay (None without log_decay) and dS0 (None when ``want_dS0``
    is False) in fp32."""
    lib = _lib or load()
    B, H, H_qk, d_k, d_v = _check_linear(q, k, v, log_decay,
                                         ((S0, "S0"), (dS_final, "dS_final")), 4)
    dev, dt, L = q.device, q.dtype, q.shape[2]
    _check(dO, "dO", (B, H, L, d_v), dt, dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return linear_chunk_bwd(q, k, v, log_decay, S0, dO, dS_final, want_dS0=want_dS0,
                                    workspace=workspace, stream=stream)
    dq, dk = _alloc(q.shape, dt, dev, stream), _alloc(q.shape, dt, dev, stream)
    dv = _alloc(v.shape, dt, dev, stream)
    dg = None if log_decay is None else _alloc(log_decay.shape, torch.float32, dev, stream)
    dS0 = _alloc((B, H, d_k, d_v), torch.float32, dev, stream) if want_dS0 else None
    need = linear_workspace_bytes(B, H, L, d_k, d_v, dt, H_qk, True)
    keep, ws, ws_bytes = _workspace(workspace, need, dev, stream)
    st = lib.deltanet_linear_chunk_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(log_decay),
                                       _ptr(S0), dO.data_ptr(), _ptr(dS_final), dq.data_ptr(),
                                       dk.data_ptr(), dv.data_ptr(), _ptr(dg), _ptr(dS0), B, H,
                                       H_qk, L, d_k, d_v, _code(dt), ws, ws_bytes,
                                       _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_linear_chunk_bwd")
    return dq, dk, dv, dg, dS0


class _LinearRule(torch.autograd.Function):
    """``linear_chunk_fwd`` (o in the inputs' dtype) with its gradient from
    ``linear_chunk_bwd``, which needs only the inputs."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, S0):
        o, S_final = linear_chunk_fwd(q, k, v, log_decay, S0, out_dtype=v.dtype)
        ctx.save_for_backward(q, k, v, log_decay, S0)
        return o, S_final

    @staticmethod
    @once_differentiable
    def backward(ctx, dO, dS_final):
        q, k, v, log_decay, S0 = ctx.saved_tensors
        want_dS0 = S0 is not None and ctx.needs_input_grad[4]
        return linear_chunk_bwd(q, k, v, log_decay, S0, dO.contiguous(), dS_final.contiguous(),
                                want_dS0=want_dS0)


def linear_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                log_decay: Optional[torch.Tensor] = None, S0: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable gated linear recurrence for training: ``(o, S_final)`` as
    ``linear_chunk_fwd`` returns them (o in the inputs' dtype), with gradients
    for every input from ``deltanet_linear_chunk_bwd``."""
    return _LinearRule.apply(q, k, v, log_decay, S0)


def linear_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       log_decay: Optional[torch.Tensor], S: torch.Tensor, *,
                       out_dtype: torch.dtype = torch.float32, o: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """One token of the gated linear recurrence (``deltanet_linear_decode_step``):
    updates S ``[B,H,d_k,d_v]`` in place and returns o ``[B,H,d_v]`` = q S_new.
    q,k ``[B,H_qk,d_k]``, v ``[B,H,d_v]``, log_decay ``[B,H]`` fp32 or None."""
    lib = _lib or load()
    B, H, H_qk, d_k, d_v = _check_linear(q, k, v, log_decay, ((S, "S"),), 3)
    dev = q.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return linear_decode_step(q, k, v, log_decay, S, out_dtype=out_dtype, o=o,
                                      stream=stream)
    if o is None:
        o = _alloc((B, H, d_v), out_dtype, dev, stream)
    else:
        _check(o, "o", (B, H, d_v), out_dtype, dev)
    st = lib.deltanet_linear_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                         _ptr(log_decay), S.data_ptr(), o.data_ptr(), B, H, H_qk,
                                         d_k, d_v, _code(q.dtype), _code(out_dtype),
                                         _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_linear_decode_step")
    return o


def _check_rows(t: torch.Tensor, name: str, shape, dtype, device):
    """A tensor of rows at any strides over its other dimensions."""
    if (type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.device == device
            and t.is_cuda and t.stride(-1) == 1):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


@functools.lru_cache(maxsize=1024)
def _strides(s):
    """The C array of a row tensor's strides (of all but the last dimension)."""
    return (ctypes.c_longlong * 3)(*s[:3])


@functools.lru_cache(maxsize=256)
def _int_array(*x):
    return (ctypes.c_int * len(x))(*x)


def _qk_setup(q_raw, k_raw, positions, inv_freq, q_weight, k_weight, sections):
    """Checks shared by both directions; (sizes, leading arguments)."""
    qs, ks = q_raw.shape, k_raw.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q_raw and k_raw must be [B, H, L, d]")
    dev, dt, (B, H_q, L, d), H_k = q_raw.device, q_raw.dtype, qs, ks[1]
    qst, kst = q_raw.stride(), k_raw.stride()
    if not (q_raw.is_cuda and ks[0] == B and ks[2:] == qs[2:] and k_raw.dtype is dt
            and k_raw.device == dev and qst[3] == 1 and kst[3] == 1):
        _check_rows(q_raw, "q_raw", (B, H_q, L, d), dt, dev)
        _check_rows(k_raw, "k_raw", (B, H_k, L, d), dt, dev)
    if q_weight is not None:
        _check(q_weight, "q_weight", (d,), torch.float32, dev)
    if k_weight is not None:
        _check(k_weight, "k_weight", (d,), torch.float32, dev)
    d_rot, axes, counts, pos, inv = 0, 1, None, None, None
    if inv_freq is not None:
        n = inv_freq.numel()
        d_rot = 2 * n
        _check(inv_freq, "inv_freq", (n,), torch.float32, dev)
        if positions is None:
            raise ValueError("positions are required with inv_freq")
        several = positions.dim() == 3
        axes = positions.shape[0] if several else 1
        _check(positions, "positions", (axes, B, L) if several else (B, L), torch.int32, dev)
        if sections is not None:
            if len(sections) != axes:
                raise ValueError(f"{len(sections)} sections for {axes} position axes")
            counts = _int_array(*sections)
        elif axes > 1:
            raise ValueError("several position axes need sections")
        if d_rot:
            pos, inv = positions.data_ptr(), inv_freq.data_ptr()
    lead = (q_raw.data_ptr(), _strides(qst), k_raw.data_ptr(), _strides(kst),
            _ptr(q_weight), _ptr(k_weight), pos, inv, counts, axes)
    return (B, H_q, H_k, L, d, d_rot), lead


def qk_norm_rope(q_raw: torch.Tensor, k_raw: torch.Tensor, positions: Optional[torch.Tensor],
                 inv_freq: Optional[torch.Tensor], *, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, sections=None, eps: float = 1e-6,
                 norm: bool = True, interleaved: bool = False, stream=None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-head RMS norm of q and k and rotation by position in one pass
    (``deltanet_qk_norm_rope``).  q_raw ``[B,H_q,L,d]``, k_raw ``[B,H_k,L,d]``
    (fp32 or bf16) at any strides with contiguous rows, so views of a fused
    projection are read in place; weights ``[d]`` fp32 or None; positions
    ``[B,L]`` or ``[axes,B,L]`` int32; inv_freq ``[d_rot/2]`` fp32 (None: no
    rotation); ``sections``: rotated pairs per position axis.  Returns dense
    ``(q_hat, k_hat)`` in the inputs' dtype."""
    lib = _lib or load()
    (B, H_q, H_k, L, d, d_rot), lead = _qk_setup(q_raw, k_raw, positions, inv_freq, q_weight,
                                                 k_weight, sections)
    dev, dt = q_raw.device, q_raw.dtype
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return qk_norm_rope(q_raw, k_raw, positions, inv_freq, q_weight=q_weight,
                                k_weight=k_weight, sections=sections, eps=eps, norm=norm,
                                interleaved=interleaved, stream=stream)
    qh, kh = _alloc((B, H_q, L, d), dt, dev, stream), _alloc((B, H_k, L, d), dt, dev, stream)
    st = lib.deltanet_qk_norm_rope(*lead, qh.data_ptr(), kh.data_ptr(), B, H_q, H_k, L, d, d_rot,
                                   int(norm), int(interleaved), eps, _code(dt),
                                   _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_qk_norm_rope")
    return qh, kh


@functools.lru_cache(maxsize=1024)
def _qk_bwd_workspace_bytes(*sizes) -> int:
    return int(load().deltanet_qk_norm_rope_bwd_workspace_bytes(*sizes))


def _like_rows(t: torch.Tensor, stream) -> torch.Tensor:
    """A new tensor of t's shape: token rows ([B, L, H, d] in memory) if t's
    heads lie inside its token rows, dense otherwise."""
    B, H, L, d = t.shape
    if t.stride(1) < t.stride(2):
        return _alloc((B, L, H, d), t.dtype, t.device, stream).transpose(1, 2)
    return _alloc((B, H, L, d), t.dtype, t.device, stream)


def qk_norm_rope_bwd(q_raw: torch.Tensor, k_raw: torch.Tensor, positions: Optional[torch.Tensor],
                     inv_freq: Optional[torch.Tensor], dq_hat: torch.Tensor, dk_hat: torch.Tensor,
                     *, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, sections=None, eps: float = 1e-6,
                     norm: bool = True, interleaved: bool = False,
                     dq_raw: Optional[torch.Tensor] = None, dk_raw: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of ``qk_norm_rope`` (``deltanet_qk_norm_rope_bwd``).  dq_hat,
    dk_hat are dense, in the inputs' dtype.  Returns ``(dq_raw, dk_raw,
    dq_weight, dk_weight)``; the weights' gradients (fp32) are None where the
    weight is.  ``dq_raw``, ``dk_raw`` may be given, at any strides (the parts
    of a fused projection's gradient)."""
    lib = _lib or load()
    (B, H_q, H_k, L, d, d_rot), lead = _qk_setup(q_raw, k_raw, positions, inv_freq, q_weight,
                                                 k_weight, sections)
    dev, t = q_raw.device, q_raw.dtype
    _check(dq_hat, "dq_hat", (B, H_q, L, d), t, dev)
    _check(dk_hat, "dk_hat", (B, H_k, L, d), t, dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return qk_norm_rope_bwd(q_raw, k_raw, positions, inv_freq, dq_hat, dk_hat,
                                    q_weight=q_weight, k_weight=k_weight, sections=sections,
                                    eps=eps, norm=norm, interleaved=interleaved, dq_raw=dq_raw,
                                    dk_raw=dk_raw, workspace=workspace, stream=stream)
    if dq_raw is None:
        dq_raw = _like_rows(q_raw, stream)
    else:
        _check_rows(dq_raw, "dq_raw", (B, H_q, L, d), t, dev)
    if dk_raw is None:
        dk_raw = _like_rows(k_raw, stream)
    else:
        _check_rows(dk_raw, "dk_raw", (B, H_k, L, d), t, dev)
    dqw = None if q_weight is None else _alloc((d,), torch.float32, dev, stream)
    dkw = None if k_weight is None else _alloc((d,), torch.float32, dev, stream)
    need = _qk_bwd_workspace_bytes(B, H_q, H_k, L, d, _code(t))
    keep, ws, ws_bytes = _workspace(workspace, need, dev, stream)
    st = lib.deltanet_qk_norm_rope_bwd(*lead, dq_hat.data_ptr(), dk_hat.data_ptr(),
                                       dq_raw.data_ptr(), _strides(dq_raw.stride()), dk_raw.data_ptr(),
                                       _strides(dk_raw.stride()), _ptr(dqw), _ptr(dkw), B, H_q, H_k, L, d,
                                       d_rot, int(norm), int(interleaved), eps, _code(t), ws,
                                       ws_bytes, _stream(dev, stream))
    if st != DN_OK:
        _raise(lib, st, "deltanet_qk_norm_rope_bwd")
    return dq_raw, dk_raw, dqw, dkw


class _RotaryQK(torch.autograd.Function):
    """``qk_norm_rope`` with its gradient from ``qk_norm_rope_bwd``."""

    @staticmethod
    def forward(ctx, q_raw, k_raw, q_weight, k_weight, positions, inv_freq, how):
        ctx.save_for_backward(q_raw, k_raw, q_weight, k_weight, positions, inv_freq)
        ctx.how = how
        return qk_norm_rope(q_raw, k_raw, positions, inv_freq, q_weight=q_weight,
                            k_weight=k_weight, **how)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_hat, dk_hat):
        q_raw, k_raw, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
        return (*qk_norm_rope_bwd(q_raw, k_raw, positions, inv_freq, dq_hat.contiguous(),
                                  dk_hat.contiguous(), q_weight=q_weight, k_weight=k_weight,
                                  **ctx.how), None, None, None)


def rotary_qk(q_raw: torch.Tensor, k_raw: torch.Tensor, positions: Optional[torch.Tensor],
              inv_freq: Optional[torch.Tensor], *, q_weight: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None, sections=None, eps: float = 1e-6,
              norm: bool = True, interleaved: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable ``qk_norm_rope`` for training, with gradients for q_raw,
    k_raw and the weights from ``deltanet_qk_norm_rope_bwd``.  There is none for
    inv_freq, which may not ask for it."""
    if inv_freq is not None and inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq has no gradient here (pass it detached)")
    # (A copy: the backward uses the sections of this call whatever becomes of the list.)
    sections = None if sections is None else tuple(sections)
    return _RotaryQK.apply(q_raw, k_raw, q_weight, k_weight, positions, inv_freq,
                           dict(sections=sections, eps=eps, norm=norm, interleaved=interleaved))


def profile_start() -> None:
    """Start bracketing this thread's kernel launches with HIP events."""
    st = load().deltanet_profile_start()
    if st != DN_OK:
        _raise(load(), st, "deltanet_profile_start")


def profile_stop() -> dict:
    """Stop, wait for the recorded events and return
    ``{slot: (total_ms, launches)}`` for the slots that launched."""
    lib = load()
    n = len(PROFILE_SLOTS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    st = lib.deltanet_profile_stop(ms, cnt, n)
    if st != DN_OK:
        _raise(lib, st, "deltanet_profile_stop")
    return {PROFILE_SLOTS[i]: (ms[i], cnt[i]) for i in range(n) if cnt[i]}
