"""delta_rule_linear_amd -- MI355X (gfx950) delta-rule linear-attention forward.

Thin Python binding over the C ABI in include/deltarule.h, with the same names.
It only marshals arguments (shape checks, output and workspace allocation with
PyTorch, the current HIP stream); every step of the computation runs in the
HIP kernels of libdeltarule.so.  If the library is missing the binding raises:
there is no fallback path.

    o, S = dr_chunk_fwd(q, k, v, log_alpha, beta, S0, gate="scalar", beta_mode="scalar")
    o = dr_decode_step(S, q, k, v, log_alpha, beta, gate="scalar", beta_mode="scalar")

With separate channel-wise erase and write strengths (FG2-GDN+):

    o, S = dr_chunk_fwd_kv(q, k, v, log_alpha, beta_k, beta_v, S0, gate="channel")
    o = dr_decode_step_kv(S, q, k, v, log_alpha, beta_k, beta_v, gate="channel")

With a diagonal preconditioner on the gradient step (write-side key scales):

    o, S = dr_chunk_fwd_precond(q, k, v, log_alpha, beta, key_scale, S0, gate="scalar",
                                beta_mode="scalar")

Gradients of the chunked forward (any gate and beta mode):

    g = dr_chunk_bwd(q, k, v, log_alpha, beta, S0, dO, dS_final, gate="scalar")
    g["dq"], g["dk"], g["dv"], g["dlog_alpha"], g["dbeta"], g["dS0"]

Linear attention with a decay per head (no erase term), its gradients and one token:

    o, S = dr_linear_attn_fwd(q, k, v, log_alpha, S0, decay="token")
    g = dr_linear_attn_bwd(q, k, v, log_alpha, S0, dO, dS_final, decay="token")
    o = dr_linear_attn_step(S, q, k, v, log_alpha, decay="head")

Layer norm of rows, such as those outputs, and its gradients:

    y, mean, rstd = dr_layernorm_fwd(o, weight, bias)
    g = dr_layernorm_bwd(o, weight, mean, rstd, dy)

RMS norm with the residual's addition (also to 8 bits with scales), the short causal
convolution and the gated linear recurrence of a layer:

    y, rstd, total = dr_rmsnorm_fwd(x, weight, residual)
    y8, scale, rstd, total = dr_rmsnorm_fwd_e4m3(x, weight, residual)
    y, state = dr_short_conv_fwd(x, weight, bias, state)
    h, h_final = dr_gated_scan_fwd(x, gate, h0, decay="logit", inputs="unit")
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdeltarule.so")

DR_ABI_VERSION = 12
DR_OK, DR_ERR_NULL, DR_ERR_SHAPE, DR_ERR_UNSUPPORTED, DR_ERR_ALIGN, DR_ERR_WORKSPACE, DR_ERR_HIP = range(7)
DR_F32, DR_BF16 = 0, 1
GATES = {"none": 0, "scalar": 1, "channel": 2}
BETAS = {"scalar": 0, "channel": 1}
DECAYS = {"none": 0, "head": 1, "token": 2}
SCAN_DECAYS = {"log": 0, "logit": 1}
SCAN_INPUTS = {"plain": 0, "blend": 1, "unit": 2}
ACTIVATIONS = {"none": 0, "silu": 1}
DR_IN_QK_L2NORM, DR_IN_BETA_LOGIT = 1, 2
EXPORTS = ("dr_chunk_fwd_workspace_bytes", "dr_chunk_fwd", "dr_chunk_fwd_kv", "dr_decode_step",
           "dr_decode_step_kv", "dr_chunk_fwd_precond_workspace_bytes", "dr_chunk_fwd_precond",
           "dr_decode_step_precond", "dr_status_str", "dr_last_error", "dr_abi_version",
           "dr_profile_begin", "dr_profile_end", "dr_chunk_bwd_workspace_bytes", "dr_chunk_bwd",
           "dr_chunk_bwd_kv", "dr_chunk_fwd_noalloc", "dr_chunk_fwd_kv_workspace_bytes",
           "dr_chunk_bwd_kv_workspace_bytes", "dr_chunk_bwd_precond_workspace_bytes", "dr_chunk_bwd_precond",
           "dr_chunk_bwd_workspace_bytes_min", "dr_linear_attn_fwd_workspace_bytes", "dr_linear_attn_fwd",
           "dr_linear_attn_bwd_workspace_bytes", "dr_linear_attn_bwd", "dr_linear_attn_step", "dr_layernorm_fwd",
           "dr_layernorm_bwd_workspace_bytes", "dr_layernorm_bwd", "dr_rmsnorm_fwd", "dr_rmsnorm_fwd_e4m3",
           "dr_rmsnorm_bwd_workspace_bytes", "dr_rmsnorm_bwd", "dr_short_conv_fwd",
           "dr_short_conv_bwd_workspace_bytes", "dr_short_conv_bwd", "dr_short_conv_step",
           "dr_gated_scan_fwd_workspace_bytes", "dr_gated_scan_fwd", "dr_gated_scan_bwd_workspace_bytes",
           "dr_gated_scan_bwd", "dr_gated_scan_step")
DR_NOALLOC_SCRATCH_BYTES = 256 << 20


class DeltaRuleError(RuntimeError):
    """A dr_* call returned an error status."""

    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{dr_status_str(status)} ({detail})")


class ChunkDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int), ("Dk", ctypes.c_int),
                ("Dv", ctypes.c_int), ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("gate", ctypes.c_int), ("beta", ctypes.c_int), ("input_flags", ctypes.c_uint)]


class ProfileReport(ctypes.Structure):
    _fields_ = [("chunk_calls", ctypes.c_int), ("decode_calls", ctypes.c_int), ("prep_ms", ctypes.c_double),
                ("scan_ms", ctypes.c_double), ("decode_ms", ctypes.c_double), ("bwd_calls", ctypes.c_int),
                ("bwd_prep_ms", ctypes.c_double), ("bwd_fscan_ms", ctypes.c_double),
                ("bwd_rscan_ms", ctypes.c_double), ("bwd_post_ms", ctypes.c_double),
                ("linear_attn_fwd_ms", ctypes.c_double), ("linear_attn_bwd_ms", ctypes.c_double),
                ("linear_attn_step_ms", ctypes.c_double), ("layernorm_fwd_ms", ctypes.c_double),
                ("layernorm_bwd_ms", ctypes.c_double), ("rmsnorm_fwd_ms", ctypes.c_double),
                ("rmsnorm_bwd_ms", ctypes.c_double), ("short_conv_fwd_ms", ctypes.c_double),
                ("short_conv_bwd_ms", ctypes.c_double), ("short_conv_step_ms", ctypes.c_double),
                ("gated_scan_fwd_ms", ctypes.c_double), ("gated_scan_bwd_ms", ctypes.c_double),
                ("gated_scan_step_ms", ctypes.c_double)]


class DecodeDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("H", ctypes.c_int), ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("gate", ctypes.c_int),
                ("beta", ctypes.c_int), ("input_flags", ctypes.c_uint)]


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("t", ctypes.c_longlong)]


class LinAttnDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("L", ctypes.c_int),
                ("Dk", ctypes.c_int), ("Dv", ctypes.c_int), ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("decay", ctypes.c_int), ("q", Strides), ("k", Strides), ("v", Strides), ("o", Strides),
                ("dq", Strides), ("dk", Strides), ("dv", Strides)]


class LinAttnStepDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("Dk", ctypes.c_int),
                ("Dv", ctypes.c_int), ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("decay", ctypes.c_int)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int), ("D", ctypes.c_int),
                ("per_head", ctypes.c_int), ("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int),
                ("dy_dtype", ctypes.c_int), ("eps", ctypes.c_float), ("x", Strides), ("y", Strides),
                ("dy", Strides)]


class RMSNormDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int), ("D", ctypes.c_int),
                ("per_head", ctypes.c_int), ("x_dtype", ctypes.c_int), ("res_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("dy_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("block", ctypes.c_int), ("x", Strides), ("res", Strides), ("y", Strides), ("total", Strides),
                ("dy", Strides)]


class ShortConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("L", ctypes.c_int), ("C", ctypes.c_int), ("W", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int), ("dy_dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("x", Strides), ("y", Strides), ("dy", Strides)]


class GatedScanDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("L", ctypes.c_int), ("C", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("h_dtype", ctypes.c_int), ("dh_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("decay", ctypes.c_int), ("inputs", ctypes.c_int), ("x", Strides),
                ("gate", Strides), ("h", Strides), ("dh", Strides), ("dx", Strides), ("dgate", Strides)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m delta_rule_linear_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        L.dr_chunk_fwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
        L.dr_chunk_fwd.argtypes = [ctypes.POINTER(ChunkDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   ctypes.c_size_t, vp]
        L.dr_chunk_fwd.restype = ctypes.c_int
        L.dr_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.dr_chunk_fwd_noalloc.restype = ctypes.c_int
        L.dr_chunk_fwd_kv.argtypes = [ctypes.POINTER(ChunkDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                      vp, ctypes.c_size_t, vp]
        L.dr_chunk_fwd_kv.restype = ctypes.c_int
        L.dr_decode_step.argtypes = [ctypes.POINTER(DecodeDesc), vp, vp, vp, vp, vp, vp, vp, vp]
        L.dr_decode_step.restype = ctypes.c_int
        L.dr_decode_step_kv.argtypes = [ctypes.POINTER(DecodeDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.dr_decode_step_kv.restype = ctypes.c_int
        L.dr_chunk_fwd_precond_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_fwd_precond_workspace_bytes.restype = ctypes.c_size_t
        L.dr_chunk_fwd_precond.argtypes = [ctypes.POINTER(ChunkDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                           vp, ctypes.c_size_t, vp]
        L.dr_chunk_fwd_precond.restype = ctypes.c_int
        L.dr_decode_step_precond.argtypes = [ctypes.POINTER(DecodeDesc), vp, vp, vp, vp, vp, vp, vp, vp,
                                             vp]
        L.dr_decode_step_precond.restype = ctypes.c_int
        L.dr_chunk_bwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.dr_chunk_bwd_workspace_bytes_min.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_bwd_workspace_bytes_min.restype = ctypes.c_size_t
        L.dr_chunk_fwd_kv_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_fwd_kv_workspace_bytes.restype = ctypes.c_size_t
        L.dr_chunk_bwd_kv_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_bwd_kv_workspace_bytes.restype = ctypes.c_size_t
        L.dr_chunk_bwd.argtypes = [ctypes.POINTER(ChunkDesc)] + [vp] * 15 + [ctypes.c_size_t, vp]
        L.dr_chunk_bwd.restype = ctypes.c_int
        L.dr_chunk_bwd_kv.argtypes = [ctypes.POINTER(ChunkDesc)] + [vp] * 17 + [ctypes.c_size_t, vp]
        L.dr_chunk_bwd_kv.restype = ctypes.c_int
        L.dr_chunk_bwd_precond_workspace_bytes.argtypes = [ctypes.POINTER(ChunkDesc)]
        L.dr_chunk_bwd_precond_workspace_bytes.restype = ctypes.c_size_t
        L.dr_chunk_bwd_precond.argtypes = [ctypes.POINTER(ChunkDesc)] + [vp] * 17 + [ctypes.c_size_t, vp]
        L.dr_chunk_bwd_precond.restype = ctypes.c_int
        for name, desc, nptr in (("dr_linear_attn_fwd", LinAttnDesc, 7), ("dr_linear_attn_bwd", LinAttnDesc, 12)):
            getattr(L, name).argtypes = [ctypes.POINTER(desc)] + [vp] * (nptr + 1) + [ctypes.c_size_t, vp]
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name + "_workspace_bytes").argtypes = [ctypes.POINTER(desc)]
            getattr(L, name + "_workspace_bytes").restype = ctypes.c_size_t
        L.dr_linear_attn_step.argtypes = [ctypes.POINTER(LinAttnStepDesc)] + [vp] * 7
        L.dr_linear_attn_step.restype = ctypes.c_int
        L.dr_layernorm_fwd.argtypes = [ctypes.POINTER(LayerNormDesc)] + [vp] * 7
        L.dr_layernorm_fwd.restype = ctypes.c_int
        L.dr_layernorm_bwd_workspace_bytes.argtypes = [ctypes.POINTER(LayerNormDesc)]
        L.dr_layernorm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.dr_layernorm_bwd.argtypes = [ctypes.POINTER(LayerNormDesc)] + [vp] * 9 + [ctypes.c_size_t, vp]
        L.dr_layernorm_bwd.restype = ctypes.c_int
        # pointers behind the descriptor; then, where there is one, the workspace and its size
        for name, desc, nptr, ws in (("dr_rmsnorm_fwd", RMSNormDesc, 6, None), ("dr_rmsnorm_fwd_e4m3", RMSNormDesc, 7, None),
                                     ("dr_rmsnorm_bwd", RMSNormDesc, 7, "_workspace_bytes"),
                                     ("dr_short_conv_fwd", ShortConvDesc, 6, None),
                                     ("dr_short_conv_bwd", ShortConvDesc, 10, "_workspace_bytes"),
                                     ("dr_short_conv_step", ShortConvDesc, 5, None),
                                     ("dr_gated_scan_fwd", GatedScanDesc, 5, "_workspace_bytes"),
                                     ("dr_gated_scan_bwd", GatedScanDesc, 9, "_workspace_bytes"),
                                     ("dr_gated_scan_step", GatedScanDesc, 4, None)):
            getattr(L, name).argtypes = ([ctypes.POINTER(desc)] + [vp] * nptr +
                                         ([vp, ctypes.c_size_t] if ws else []) + [vp])
            getattr(L, name).restype = ctypes.c_int
            if ws:
                getattr(L, name + ws).argtypes = [ctypes.POINTER(desc)]
                getattr(L, name + ws).restype = ctypes.c_size_t
        L.dr_status_str.argtypes = [ctypes.c_int]
        L.dr_status_str.restype = ctypes.c_char_p
        L.dr_last_error.argtypes = []
        L.dr_last_error.restype = ctypes.c_char_p
        L.dr_abi_version.argtypes = []
        L.dr_abi_version.restype = ctypes.c_int
        L.dr_profile_begin.argtypes = []
        L.dr_profile_begin.restype = ctypes.c_int
        L.dr_profile_end.argtypes = [ctypes.POINTER(ProfileReport)]
        L.dr_profile_end.restype = ctypes.c_int
        if L.dr_abi_version() != DR_ABI_VERSION:
            raise ImportError(f"{LIB_PATH} has ABI {L.dr_abi_version()}, binding expects {DR_ABI_VERSION}")
        _lib = L
    return _lib


def dr_abi_version() -> int:
    return int(lib().dr_abi_version())


def dr_status_str(status: int) -> str:
    return lib().dr_status_str(int(status)).decode()


def dr_last_error() -> str:
    return lib().dr_last_error().decode()


def _check(status: int):
    if status != DR_OK:
        raise DeltaRuleError(status, dr_last_error())


def dr_profile_begin() -> None:
    """Start recording per-kernel HIP events in later calls."""
    _check(lib().dr_profile_begin())


def dr_profile_end() -> dict:
    """Stop recording; wait for the events and return the summed kernel times (ms)."""
    rep = ProfileReport()
    _check(lib().dr_profile_end(ctypes.byref(rep)))
    return {f: getattr(rep, f) for f, _ in ProfileReport._fields_}


# ---------------------------------------------------------------------------
# torch-facing wrappers (argument marshalling only)
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.bfloat16:
        return DR_BF16
    if dt == torch.float32:
        return DR_F32
    raise TypeError(f"unsupported dtype {dt}: use torch.bfloat16 or torch.float32")


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _need(t, name, dtype=None, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def input_flags(qk_l2norm: bool = False, beta_logit: bool = False) -> int:
    return (DR_IN_QK_L2NORM if qk_l2norm else 0) | (DR_IN_BETA_LOGIT if beta_logit else 0)


def chunk_desc(B, H, L, Dk, Dv, in_dtype, out_dtype, gate: str, beta_mode: str,
               flags: int = 0) -> ChunkDesc:
    return ChunkDesc(B, H, L, Dk, Dv, in_dtype, out_dtype, GATES[gate], BETAS[beta_mode], flags)


def dr_chunk_fwd_workspace_bytes(desc: ChunkDesc) -> int:
    return int(lib().dr_chunk_fwd_workspace_bytes(ctypes.byref(desc)))


def dr_chunk_fwd_precond_workspace_bytes(desc: ChunkDesc) -> int:
    return int(lib().dr_chunk_fwd_precond_workspace_bytes(ctypes.byref(desc)))


def dr_chunk_fwd(q, k, v, log_alpha, beta, S0=None, *, gate: str, beta_mode: str,
                 out_dtype=None, o=None, S_final=None, want_state: bool = True,
                 workspace=None, stream=None, qk_l2norm: bool = False, beta_logit: bool = False):
    """Chunked forward over [B, H, L, D] device tensors; returns (o, S_final).

    q, k: [B,H,L,Dk]; v: [B,H,L,Dv] (bf16 or fp32, same dtype); log_alpha:
    [B,H,L] / [B,H,L,Dk] fp32 or None for gate "none"; beta: [B,H,L] /
    [B,H,L,Dk] fp32; S0: [B,H,Dk,Dv] fp32 or None.  S_final may be passed in
    (it may be S0 itself for an in-place carry); with want_state=False no
    final state is written and None is returned for it.  qk_l2norm and
    beta_logit switch on the input preparation (DR_IN_QK_L2NORM,
    DR_IN_BETA_LOGIT).
    """
    return _chunk(q, k, v, log_alpha, beta, None, S0, gate, beta_mode, out_dtype, o, S_final,
                  want_state, workspace, stream, input_flags(qk_l2norm, beta_logit))


def dr_chunk_fwd_precond(q, k, v, log_alpha, beta, key_scale, S0=None, *, gate: str, beta_mode: str,
                         out_dtype=None, o=None, S_final=None, want_state: bool = True, workspace=None,
                         stream=None, qk_l2norm: bool = False, beta_logit: bool = False):
    """dr_chunk_fwd with write-side key scales key_scale [B,H,L,Dk] fp32 (the
    diagonal preconditioner of the gradient step)."""
    if key_scale is None:
        raise ValueError("key_scale is required")
    return _chunk(q, k, v, log_alpha, beta, None, S0, gate, beta_mode, out_dtype, o, S_final,
                  want_state, workspace, stream, input_flags(qk_l2norm, beta_logit), key_scale)


def dr_chunk_fwd_kv(q, k, v, log_alpha, beta_k, beta_v, S0=None, *, gate: str, beta_mode: str = "channel",
                    out_dtype=None, o=None, S_final=None, want_state: bool = True, workspace=None, stream=None,
                    qk_l2norm: bool = False, beta_logit: bool = False):
    """dr_chunk_fwd with separate erase (beta_k) and write (beta_v)
    strengths, both [B,H,L,Dk] (beta_mode "channel") or both [B,H,L]
    (beta_mode "scalar") fp32; Dv == Dk."""
    if beta_v is None:
        raise ValueError("beta_v is required")
    return _chunk(q, k, v, log_alpha, beta_k, beta_v, S0, gate, beta_mode, out_dtype, o, S_final,
                  want_state, workspace, stream, input_flags(qk_l2norm, beta_logit))


def dr_chunk_fwd_kv_workspace_bytes(desc: ChunkDesc) -> int:
    return int(lib().dr_chunk_fwd_kv_workspace_bytes(ctypes.byref(desc)))


def dr_chunk_bwd_workspace_bytes_min(desc: ChunkDesc) -> int:
    """The least workspace dr_chunk_bwd accepts (segments of chunks below
    dr_chunk_bwd_workspace_bytes; equal to it where segments do not apply)."""
    return int(lib().dr_chunk_bwd_workspace_bytes_min(ctypes.byref(desc)))


def dr_chunk_bwd_kv_workspace_bytes(desc: ChunkDesc) -> int:
    return int(lib().dr_chunk_bwd_kv_workspace_bytes(ctypes.byref(desc)))


def dr_chunk_fwd_noalloc(q, k, v, log_alpha, beta, S0=None, *, gate: str, beta_mode: str, o, S_final=None,
                         stream=None, qk_l2norm: bool = False, beta_logit: bool = False):
    """dr_chunk_fwd without a workspace: the library's per-GPU scratch array
    (DR_NOALLOC_SCRATCH_BYTES) takes its place, for callers that cannot
    allocate.  o (and S_final, or None to skip it) are the caller's tensors;
    nothing is allocated here or in the library.  Calls that overlap in time
    on one GPU race on the scratch array.  Returns (o, S_final)."""
    return _chunk(q, k, v, log_alpha, beta, None, S0, gate, beta_mode, o.dtype, o, S_final,
                  False, None, stream, input_flags(qk_l2norm, beta_logit), noalloc=True)


def _chunk(q, k, v, log_alpha, beta, beta_v, S0, gate, beta_mode, out_dtype, o, S_final, want_state,
           workspace, stream, flags, key_scale=None, noalloc=False):
    torch = _torch()
    B, H, L, Dk = q.shape
    Dv = v.shape[-1]
    _need(q, "q")
    _need(k, "k", q.dtype, (B, H, L, Dk))
    _need(v, "v", q.dtype, (B, H, L, Dv))
    gshape = {"none": None, "scalar": (B, H, L), "channel": (B, H, L, Dk)}[gate]
    if gshape is None:
        if log_alpha is not None:
            raise ValueError("gate 'none' takes no log_alpha")
    else:
        _need(log_alpha, "log_alpha", torch.float32, gshape)
    bshape = (B, H, L) if beta_mode == "scalar" else (B, H, L, Dk)
    _need(beta, "beta", torch.float32, bshape)
    if beta_v is not None:
        _need(beta_v, "beta_v", torch.float32, bshape)
    if key_scale is not None:
        _need(key_scale, "key_scale", torch.float32, (B, H, L, Dk))
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, Dk, Dv))
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty((B, H, L, Dv), dtype=out_dtype, device=q.device)
    else:
        _need(o, "o", out_dtype, (B, H, L, Dv))
    if want_state and S_final is None:
        S_final = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    elif S_final is not None:
        _need(S_final, "S_final", torch.float32, (B, H, Dk, Dv))
    desc = chunk_desc(B, H, L, Dk, Dv, _dtype_code(q.dtype), _dtype_code(out_dtype), gate, beta_mode,
                      flags)
    if noalloc:
        _check(lib().dr_chunk_fwd_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                          _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_final), _stream(stream)))
        return o, S_final
    nbytes = (dr_chunk_fwd_precond_workspace_bytes(desc) if key_scale is not None
              else dr_chunk_fwd_kv_workspace_bytes(desc) if beta_v is not None
              else dr_chunk_fwd_workspace_bytes(desc))
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if key_scale is not None:
        _check(lib().dr_chunk_fwd_precond(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                          _ptr(beta), _ptr(key_scale), _ptr(S0), _ptr(o), _ptr(S_final),
                                          _ptr(workspace), wbytes, _stream(stream)))
    elif beta_v is None:
        _check(lib().dr_chunk_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                  _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_final), _ptr(workspace),
                                  wbytes, _stream(stream)))
    else:
        _check(lib().dr_chunk_fwd_kv(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                     _ptr(beta), _ptr(beta_v), _ptr(S0), _ptr(o), _ptr(S_final),
                                     _ptr(workspace), wbytes, _stream(stream)))
    return o, S_final


def dr_chunk_bwd_workspace_bytes(desc: ChunkDesc) -> int:
    return int(lib().dr_chunk_bwd_workspace_bytes(ctypes.byref(desc)))


def dr_chunk_bwd_kv(q, k, v, log_alpha, beta_k, beta_v, S0, dO, dS_final=None, *, gate: str,
                    beta_mode: str = "channel", want_dS0: bool = True, workspace=None, stream=None,
                    qk_l2norm: bool = False, beta_logit: bool = False):
    """Gradients of dr_chunk_fwd_kv (separate erase and write strengths, both
    [B,H,L,Dk] or both [B,H,L] fp32): as dr_chunk_bwd, with dbeta the erase
    strength's gradient and dbeta_v the write strength's."""
    if beta_v is None:
        raise ValueError("beta_v is required")
    return dr_chunk_bwd(q, k, v, log_alpha, beta_k, S0, dO, dS_final, gate=gate, beta_mode=beta_mode,
                        want_dS0=want_dS0, workspace=workspace, stream=stream, qk_l2norm=qk_l2norm,
                        beta_logit=beta_logit, _beta_v=beta_v)


def dr_chunk_bwd_precond_workspace_bytes(desc: ChunkDesc) -> int:
    return int(lib().dr_chunk_bwd_precond_workspace_bytes(ctypes.byref(desc)))


def dr_chunk_bwd_precond(q, k, v, log_alpha, beta, key_scale, S0, dO, dS_final=None, *, gate: str,
                         beta_mode: str = "scalar", want_dS0: bool = True, workspace=None, stream=None,
                         qk_l2norm: bool = False, beta_logit: bool = False):
    """Gradients of dr_chunk_fwd_precond (write-side key scales key_scale,
    [B,H,L,Dk] fp32): as dr_chunk_bwd, with dkey_scale the scales' gradient."""
    if key_scale is None:
        raise ValueError("key_scale is required")
    return dr_chunk_bwd(q, k, v, log_alpha, beta, S0, dO, dS_final, gate=gate, beta_mode=beta_mode,
                        want_dS0=want_dS0, workspace=workspace, stream=stream, qk_l2norm=qk_l2norm,
                        beta_logit=beta_logit, _key_scale=key_scale)


def dr_chunk_bwd(q, k, v, log_alpha, beta, S0, dO, dS_final=None, *, gate: str, beta_mode: str = "scalar",
                 want_dS0: bool = True, workspace=None, stream=None, qk_l2norm: bool = False,
                 beta_logit: bool = False, _beta_v=None, _key_scale=None):
    """Gradients of dr_chunk_fwd (any gate and beta mode) for the
    loss whose gradients with respect to o and S_final are dO [B,H,L,Dv] and
    dS_final [B,H,Dk,Dv] (fp32; dS_final None means zero).  q, k, v and the
    other inputs are as for dr_chunk_fwd, with the same input preparation
    (qk_l2norm, beta_logit): the gradients are those of the raw inputs.
    Returns a dict of fp32 device tensors dq, dk, dv, dlog_alpha (None for
    gate "none"), dbeta and dS0 (None with want_dS0=False).  workspace: a
    device uint8 tensor (None: one of dr_chunk_bwd_workspace_bytes bytes is
    allocated); one smaller than that, down to dr_chunk_bwd_workspace_bytes_min,
    makes the library run the backward in segments of chunks."""
    torch = _torch()
    B, H, L, Dk = q.shape
    Dv = v.shape[-1]
    _need(q, "q")
    _need(k, "k", q.dtype, (B, H, L, Dk))
    _need(v, "v", q.dtype, (B, H, L, Dv))
    gshape = {"none": None, "scalar": (B, H, L), "channel": (B, H, L, Dk)}[gate]
    if gshape is None:
        if log_alpha is not None:
            raise ValueError("gate 'none' takes no log_alpha")
    else:
        _need(log_alpha, "log_alpha", torch.float32, gshape)
    bshape = (B, H, L) if beta_mode == "scalar" else (B, H, L, Dk)
    _need(beta, "beta", torch.float32, bshape)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, Dk, Dv))
    if _beta_v is not None:
        _need(_beta_v, "beta_v", torch.float32, bshape)
    if _key_scale is not None:
        _need(_key_scale, "key_scale", torch.float32, (B, H, L, Dk))
    _need(dO, "dO", torch.float32, (B, H, L, Dv))
    if dS_final is not None:
        _need(dS_final, "dS_final", torch.float32, (B, H, Dk, Dv))
    f32 = dict(dtype=torch.float32, device=q.device)
    out = {"dq": torch.empty((B, H, L, Dk), **f32), "dk": torch.empty((B, H, L, Dk), **f32),
           "dv": torch.empty((B, H, L, Dv), **f32),
           "dlog_alpha": torch.empty(gshape, **f32) if gshape is not None else None,
           "dbeta": torch.empty(bshape, **f32),
           "dS0": torch.empty((B, H, Dk, Dv), **f32) if want_dS0 else None}
    desc = chunk_desc(B, H, L, Dk, Dv, _dtype_code(q.dtype), DR_F32, gate, beta_mode,
                      input_flags(qk_l2norm, beta_logit))
    if _key_scale is not None:
        nbytes = dr_chunk_bwd_precond_workspace_bytes(desc)
    elif _beta_v is not None:
        nbytes = dr_chunk_bwd_kv_workspace_bytes(desc)
    else:
        nbytes = dr_chunk_bwd_workspace_bytes(desc)
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if _key_scale is not None:
        out["dkey_scale"] = torch.empty((B, H, L, Dk), **f32)
        _check(lib().dr_chunk_bwd_precond(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                          _ptr(beta), _ptr(_key_scale), _ptr(S0), _ptr(dO), _ptr(dS_final),
                                          _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                          _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]), _ptr(out["dkey_scale"]),
                                          _ptr(out["dS0"]), _ptr(workspace), wbytes, _stream(stream)))
    elif _beta_v is None:
        _check(lib().dr_chunk_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                  _ptr(S0), _ptr(dO), _ptr(dS_final), _ptr(out["dq"]), _ptr(out["dk"]),
                                  _ptr(out["dv"]), _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]), _ptr(out["dS0"]),
                                  _ptr(workspace), wbytes, _stream(stream)))
    else:
        out["dbeta_v"] = torch.empty(bshape, **f32)
        _check(lib().dr_chunk_bwd_kv(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                     _ptr(_beta_v), _ptr(S0), _ptr(dO), _ptr(dS_final), _ptr(out["dq"]),
                                     _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]),
                                     _ptr(out["dbeta_v"]), _ptr(out["dS0"]), _ptr(workspace), wbytes,
                                     _stream(stream)))
    return out


def dr_decode_step(S, q, k, v, log_alpha, beta, *, gate: str, beta_mode: str, out_dtype=None,
                   o=None, stream=None, qk_l2norm: bool = False, beta_logit: bool = False):
    """One decode step for N x H states (updated in place); returns o [N,H,Dv].

    S: [N,H,Dk,Dv] fp32; q, k: [N,H,Dk]; v: [N,H,Dv]; log_alpha: [N,H] /
    [N,H,Dk] or None; beta: [N,H] / [N,H,Dk].
    """
    return _decode(S, q, k, v, log_alpha, beta, None, gate, beta_mode, out_dtype, o, stream,
                   input_flags(qk_l2norm, beta_logit))


def dr_decode_step_precond(S, q, k, v, log_alpha, beta, key_scale, *, gate: str, beta_mode: str,
                           out_dtype=None, o=None, stream=None, qk_l2norm: bool = False,
                           beta_logit: bool = False):
    """dr_decode_step with write-side key scales key_scale [N,H,Dk] fp32."""
    if key_scale is None:
        raise ValueError("key_scale is required")
    return _decode(S, q, k, v, log_alpha, beta, None, gate, beta_mode, out_dtype, o, stream,
                   input_flags(qk_l2norm, beta_logit), key_scale)


def dr_decode_step_kv(S, q, k, v, log_alpha, beta_k, beta_v, *, gate: str, beta_mode: str = "channel",
                      out_dtype=None, o=None, stream=None, qk_l2norm: bool = False, beta_logit: bool = False):
    """dr_decode_step with separate erase (beta_k) and write (beta_v)
    strengths, both [N,H,Dk] (beta_mode "channel", Dv == Dk) or both [N,H]
    (beta_mode "scalar") fp32."""
    if beta_v is None:
        raise ValueError("beta_v is required")
    return _decode(S, q, k, v, log_alpha, beta_k, beta_v, gate, beta_mode, out_dtype, o, stream,
                   input_flags(qk_l2norm, beta_logit))


def _decode(S, q, k, v, log_alpha, beta, beta_v, gate, beta_mode, out_dtype, o, stream, flags,
            key_scale=None):
    torch = _torch()
    N, H, Dk, Dv = S.shape
    _need(S, "S", torch.float32)
    _need(q, "q", None, (N, H, Dk))
    _need(k, "k", q.dtype, (N, H, Dk))
    _need(v, "v", q.dtype, (N, H, Dv))
    gshape = {"none": None, "scalar": (N, H), "channel": (N, H, Dk)}[gate]
    if gshape is None:
        if log_alpha is not None:
            raise ValueError("gate 'none' takes no log_alpha")
    else:
        _need(log_alpha, "log_alpha", torch.float32, gshape)
    bshape = (N, H) if beta_mode == "scalar" else (N, H, Dk)
    _need(beta, "beta", torch.float32, bshape)
    if beta_v is not None:
        _need(beta_v, "beta_v", torch.float32, bshape)
    if key_scale is not None:
        _need(key_scale, "key_scale", torch.float32, (N, H, Dk))
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty((N, H, Dv), dtype=out_dtype, device=S.device)
    else:
        _need(o, "o", out_dtype, (N, H, Dv))
    desc = DecodeDesc(N, H, Dk, Dv, _dtype_code(q.dtype), _dtype_code(out_dtype), GATES[gate],
                      BETAS[beta_mode], flags)
    if key_scale is not None:
        _check(lib().dr_decode_step_precond(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                            _ptr(beta), _ptr(key_scale), _ptr(S), _ptr(o), _stream(stream)))
    elif beta_v is None:
        _check(lib().dr_decode_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                    _ptr(beta), _ptr(S), _ptr(o), _stream(stream)))
    else:
        _check(lib().dr_decode_step_kv(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                       _ptr(beta), _ptr(beta_v), _ptr(S), _ptr(o), _stream(stream)))
    return o


# ---------------------------------------------------------------------------
# linear attention with a decay per head; layer norm
# ---------------------------------------------------------------------------

def _strides(t):
    """The strides of a [B,H,L,D] view in elements (0 where a dimension is 1)."""
    n, s = t.shape, t.stride()
    return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)


def _need_rows(t, name, device, dtype=None, shape=None):
    """A device tensor whose last dimension is contiguous; other strides are free."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_on(t, name, device, dtype, shape):
    torch = _torch()
    if (isinstance(t, torch.Tensor) and t.device == device and t.shape == shape and t.is_contiguous() and
            (dtype is None or t.dtype == dtype)):
        return
    _need(t, name, dtype, shape)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


class _on:
    """Runs on `device`, on `stream` (default: the device's current stream), so
    that what is allocated inside belongs to that stream; gives the raw stream."""

    __slots__ = ("ctx", "stream")

    def __init__(self, device, stream):
        cuda = _torch().cuda
        if stream is None:
            self.ctx = None if cuda.current_device() == device.index else cuda.device(device)
            self.stream = _raw_stream(device)
        else:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.ctx, self.stream = cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.stream

    def __exit__(self, *exc):
        return None if self.ctx is None else self.ctx.__exit__(*exc)


def _raw_stream(device) -> int:
    """The device's current stream, without building a Stream object where
    PyTorch offers that."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(device).cuda_stream if raw is None else raw(device.index)


def _workspace(workspace, nbytes, device):
    torch = _torch()
    if workspace is None:
        return (torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes) if nbytes else (None, 0)
    _need(workspace, "workspace")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _decay_arg(log_alpha, decay, H, token_shape, device):
    torch = _torch()
    if decay not in DECAYS:
        raise ValueError(f"decay must be one of {sorted(DECAYS)}, got {decay!r}")
    if decay == "none":
        if log_alpha is not None:
            raise ValueError("decay 'none' takes no log_alpha")
    else:
        _need_on(log_alpha, "log_alpha", device, torch.float32, (H,) if decay == "head" else token_shape)


def _fit_int(sizes):
    """A descriptor's sizes are C ints: ctypes would keep the low 32 bits of a
    larger one, and the call would treat that many rows as all of them."""
    for n in sizes:
        if n > 2 ** 31 - 1 or n < -2 ** 31:
            raise ValueError(f"a dimension of {n}: at most 2^31 - 1 is supported")


def linattn_desc(B, H, Hk, L, Dk, Dv, in_dtype, out_dtype, decay: str) -> LinAttnDesc:
    """A descriptor for dense tensors; the strides can be set afterwards."""
    _fit_int((B, H, Hk, L, Dk, Dv))
    qk, vo = Strides(Hk * L * Dk, L * Dk, Dk), Strides(H * L * Dv, L * Dv, Dv)
    return LinAttnDesc(B, H, Hk, L, Dk, Dv, in_dtype, out_dtype, DECAYS[decay], qk, qk, vo, vo, qk, qk, vo)


# Descriptors and workspace sizes of the shapes in use (they depend on sizes,
# types and strides alone).
@functools.lru_cache(maxsize=512)
def _linattn_plan(bwd: bool, sizes, *strides):
    _fit_int(sizes)
    desc = LinAttnDesc(*sizes, *(Strides(*s) for s in strides))
    fn = lib().dr_linear_attn_bwd_workspace_bytes if bwd else lib().dr_linear_attn_fwd_workspace_bytes
    return desc, ctypes.byref(desc), int(fn(ctypes.byref(desc)))


@functools.lru_cache(maxsize=512)
def _linattn_step_plan(*sizes):
    _fit_int(sizes)
    desc = LinAttnStepDesc(*sizes)
    return desc, ctypes.byref(desc)


@functools.lru_cache(maxsize=512)
def _layernorm_plan(sizes, *strides):
    _fit_int(sizes[:4])   # B, H, L, D
    desc = LayerNormDesc(*sizes, *(Strides(*s) for s in strides))
    return desc, ctypes.byref(desc), int(lib().dr_layernorm_bwd_workspace_bytes(ctypes.byref(desc)))


def dr_linear_attn_fwd_workspace_bytes(desc: LinAttnDesc) -> int:
    return int(lib().dr_linear_attn_fwd_workspace_bytes(ctypes.byref(desc)))


def dr_linear_attn_bwd_workspace_bytes(desc: LinAttnDesc) -> int:
    return int(lib().dr_linear_attn_bwd_workspace_bytes(ctypes.byref(desc)))


def _linattn_inputs(q, k, v, log_alpha, S0, decay):
    torch = _torch()
    if not (isinstance(q, torch.Tensor) and isinstance(v, torch.Tensor)) or q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B, heads, L, channels] tensors")
    B, Hk, L, Dk = q.shape
    H, Dv = v.shape[1], v.shape[-1]
    _need_rows(q, "q", None)
    _need_rows(k, "k", q.device, q.dtype, (B, Hk, L, Dk))
    _need_rows(v, "v", q.device, q.dtype, (B, H, L, Dv))
    _decay_arg(log_alpha, decay, H, (B, H, L), q.device)
    if S0 is not None:
        _need_on(S0, "S0", q.device, torch.float32, (B, H, Dk, Dv))
    return B, H, Hk, L, Dk, Dv


def _state(like, shape, device):
    """A new fp32 state, like another if there is one (less work than by sizes)."""
    torch = _torch()
    return torch.empty(shape, dtype=torch.float32, device=device) if like is None else torch.empty_like(like)


def dr_linear_attn_fwd(q, k, v, log_alpha=None, S0=None, *, decay: str, out_dtype=None, o=None, S_final=None,
                       want_state: bool = True, workspace=None, stream=None):
    """Linear attention with a decay per head, S_t = alpha_t S_{t-1} + k_t v_t^T,
    o_t = S_t^T q_t, over [B, heads, L, D] device tensors; returns (o, S_final).

    q, k: [B,Hk,L,Dk]; v: [B,H,L,Dv] (bf16 or fp32, same dtype), H a multiple of
    Hk; any strides whose channels are contiguous and whose rows start at
    multiples of 16 bytes (views of [B,L,H,D] projections).  decay "head":
    log_alpha [H] fp32, one constant per head; "token": [B,H,L] fp32; "none".
    S0: [B,H,Dk,Dv] fp32 or None.  o defaults to out_dtype (fp32) in v's order
    of dimensions; S_final may be S0 itself; with want_state=False and no
    S_final none is written and None is returned for it.
    """
    torch = _torch()
    B, H, Hk, L, Dk, Dv = _linattn_inputs(q, k, v, log_alpha, S0, decay)
    dev = q.device
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty_like(v, dtype=torch.float32 if out_dtype is None else out_dtype)
        else:
            _need_rows(o, "o", dev, out_dtype, (B, H, L, Dv))
        if S_final is not None:
            _need_on(S_final, "S_final", dev, torch.float32, (B, H, Dk, Dv))
        elif want_state:
            S_final = _state(S0, (B, H, Dk, Dv), dev)
        _, desc, nbytes = _linattn_plan(
            False, (B, H, Hk, L, Dk, Dv, _dtype_code(q.dtype), _dtype_code(o.dtype), DECAYS[decay]),
            _strides(q), _strides(k), _strides(v), _strides(o))
        workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_linear_attn_fwd(desc, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(S0),
                                        _ptr(o), _ptr(S_final), _ptr(workspace), wbytes, st))
    return o, S_final


def dr_linear_attn_bwd(q, k, v, log_alpha, S0, dO, dS_final=None, *, decay: str, grad_dtype=None,
                       want_dS0: bool = True, workspace=None, stream=None):
    """Gradients of dr_linear_attn_fwd for the loss whose gradients with respect
    to o and S_final are dO [B,H,L,Dv] (q's dtype) and dS_final [B,H,Dk,Dv]
    (fp32; None: zero).  Returns a dict of device tensors: dq, dk, dv in
    grad_dtype (fp32) and in the order of their inputs' dimensions, dlog_alpha
    (log_alpha's shape, fp32; None for decay "none") and dS0 (fp32; None with
    want_dS0=False)."""
    torch = _torch()
    B, H, Hk, L, Dk, Dv = _linattn_inputs(q, k, v, log_alpha, S0, decay)
    dev = q.device
    _need_rows(dO, "dO", dev, q.dtype, (B, H, L, Dv))
    if dS_final is not None:
        _need_on(dS_final, "dS_final", dev, torch.float32, (B, H, Dk, Dv))
    to = torch.float32 if grad_dtype is None else grad_dtype
    with _on(dev, stream) as st:
        out = {"dq": torch.empty_like(q, dtype=to), "dk": torch.empty_like(k, dtype=to),
               "dv": torch.empty_like(v, dtype=to),
               "dlog_alpha": None if log_alpha is None else torch.empty_like(log_alpha),
               "dS0": _state(S0, (B, H, Dk, Dv), dev) if want_dS0 else None}
        _, desc, nbytes = _linattn_plan(
            True, (B, H, Hk, L, Dk, Dv, _dtype_code(q.dtype), _dtype_code(to), DECAYS[decay]),
            _strides(q), _strides(k), _strides(v), _strides(dO), _strides(out["dq"]), _strides(out["dk"]),
            _strides(out["dv"]))
        workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_linear_attn_bwd(desc, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(S0),
                                        _ptr(dO), _ptr(dS_final), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                        _ptr(out["dlog_alpha"]), _ptr(out["dS0"]), _ptr(workspace), wbytes, st))
    return out


def dr_linear_attn_step(S, q, k, v, log_alpha=None, *, decay: str, out_dtype=None, o=None, stream=None):
    """One token of the linear attention for N x H states (updated in place);
    returns o [N,H,Dv].

    S: [N,H,Dk,Dv] fp32; q, k: [N,Hk,Dk]; v: [N,H,Dv]; log_alpha: [H] (decay
    "head"), [N,H] ("token") or None ("none").
    """
    torch = _torch()
    N, H, Dk, Dv = S.shape
    _need(S, "S", torch.float32)
    dev, Hk = S.device, q.shape[1]
    _need_on(q, "q", dev, None, (N, Hk, Dk))
    _need_on(k, "k", dev, q.dtype, (N, Hk, Dk))
    _need_on(v, "v", dev, q.dtype, (N, H, Dv))
    _decay_arg(log_alpha, decay, H, (N, H), dev)
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty_like(v, dtype=torch.float32 if out_dtype is None else out_dtype)
        else:
            _need_on(o, "o", dev, out_dtype, (N, H, Dv))
        _, desc = _linattn_step_plan(N, H, Hk, Dk, Dv, _dtype_code(q.dtype), _dtype_code(o.dtype), DECAYS[decay])
        _check(lib().dr_linear_attn_step(desc, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(S),
                                         _ptr(o), st))
    return o


def _norm_dims(t, per_head: bool):
    """Sizes and strides of x as [B, H, L, D] rows: [N, D], and with a weight for
    each head [N, H, D] or [B, H, L, D]; with one weight also [B, L, D] and
    [B, H, L, D]."""
    n, s = t.shape, t.stride()
    if len(n) == 4:
        dims, steps = (n[0], n[1], n[2], n[3]), (s[0], s[1], s[2])
    elif len(n) == 3:
        dims, steps = ((n[0], n[1], 1, n[2]), (s[0], s[1], 0)) if per_head else ((n[0], 1, n[1], n[2]), (s[0], 0, s[1]))
    elif len(n) == 2 and not per_head:
        dims, steps = (1, 1, n[0], n[1]), (0, 0, s[0])
    else:
        raise ValueError("x must be [N, D], [B, L, D], [N, H, D] or [B, H, L, D], with a weight [D] or [H, D]")
    return dims, tuple(st if k > 1 else 0 for k, st in zip(dims, steps))


def _norm_args(x, per_head, weight, bias):
    """The sizes and strides of x's rows and whether the weights are one per head."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if weight is not None and bias is not None and weight.dim() != bias.dim():
        raise ValueError("weight and bias must have the same shape")
    if per_head is None:
        first = bias if weight is None else weight
        per_head = first is not None and first.dim() == 2
    dims, steps = _norm_dims(x, per_head)
    _need_rows(x, "x", None)
    shape = (dims[1], dims[3]) if per_head else (dims[3],)
    if weight is not None:
        _need_on(weight, "weight", x.device, torch.float32, shape)
    if bias is not None:
        _need_on(bias, "bias", x.device, torch.float32, shape)
    return dims, steps, per_head, shape


def dr_layernorm_fwd(x, weight=None, bias=None, *, eps: float = 1e-5, out_dtype=None, y=None, mean=None, rstd=None,
                     stream=None):
    """Layer norm over the last dimension of x: (x - mean) rstd weight + bias;
    returns (y, mean, rstd).

    x: [N,D], [B,L,D] or [B,H,L,D] (bf16 or fp32) with weight and bias [D] fp32;
    or, with one weight per head [H,D], [N,H,D] or [B,H,L,D].  Channels are
    contiguous, other strides free; tensors start at multiples of 16 bytes where
    D and the strides are multiples of 8, else anywhere.  y defaults to out_dtype (x's dtype) in x's
    order of dimensions; mean and rstd are fp32, contiguous, of x's leading shape.
    """
    torch = _torch()
    dims, steps, per_head, _ = _norm_args(x, None, weight, bias)
    dev, lead = x.device, x.shape[:-1]
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype)
        else:
            _need_rows(y, "y", dev, out_dtype, x.shape)
        ysteps = steps if y.stride() == x.stride() else _norm_dims(y, per_head)[1]
        if mean is None:
            mean = torch.empty(lead, dtype=torch.float32, device=dev)
        else:
            _need_on(mean, "mean", dev, torch.float32, lead)
        if rstd is None:
            rstd = torch.empty_like(mean)   # a like tensor takes half the time of one by its sizes
        else:
            _need_on(rstd, "rstd", dev, torch.float32, lead)
        _, desc, _ = _layernorm_plan(dims + (int(per_head), _dtype_code(x.dtype), _dtype_code(y.dtype), DR_F32,
                                             float(eps)), steps, ysteps)
        _check(lib().dr_layernorm_fwd(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), st))
    return y, mean, rstd


def dr_layernorm_bwd_workspace_bytes(desc: LayerNormDesc) -> int:
    return int(lib().dr_layernorm_bwd_workspace_bytes(ctypes.byref(desc)))


def dr_layernorm_bwd(x, weight, mean, rstd, dy, *, per_head=None, grad_dtype=None, dx=None, want_sums: bool = True,
                     workspace=None, stream=None):
    """Gradients of dr_layernorm_fwd: dx in grad_dtype (x's dtype) and in x's
    order of dimensions, dweight and dbias fp32 (None with want_sums=False), in
    a dict.  x, weight, mean and rstd are the forward's; dy (bf16 or fp32) has
    x's shape.  Without a weight, per_head=True makes the sums one per head."""
    torch = _torch()
    if weight is not None and per_head is not None and per_head != (weight.dim() == 2):
        raise ValueError("per_head does not fit the weight's shape")
    dims, steps, per_head, wshape = _norm_args(x, per_head, weight, None)
    dev, lead = x.device, x.shape[:-1]
    _need_on(mean, "mean", dev, torch.float32, lead)
    _need_on(rstd, "rstd", dev, torch.float32, lead)
    _need_rows(dy, "dy", dev, None, x.shape)
    with _on(dev, stream) as st:
        if dx is None:
            dx = torch.empty_like(x, dtype=grad_dtype)
        else:
            _need_rows(dx, "dx", dev, grad_dtype, x.shape)
        _, desc, nbytes = _layernorm_plan(dims + (int(per_head), _dtype_code(x.dtype), _dtype_code(dx.dtype),
                                                  _dtype_code(dy.dtype), 0.0), steps,
                                          *(steps if t.stride() == x.stride() else _norm_dims(t, per_head)[1]
                                            for t in (dx, dy)))
        out = {"dx": dx, "dweight": None, "dbias": None}
        wbytes = 0
        if want_sums:
            out["dweight"] = (torch.empty(wshape, dtype=torch.float32, device=dev) if weight is None else
                              torch.empty_like(weight))
            out["dbias"] = torch.empty_like(out["dweight"])
            workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_layernorm_bwd(desc, _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy),
                                      _ptr(dx), _ptr(out["dweight"]), _ptr(out["dbias"]), _ptr(workspace), wbytes,
                                      st))
    return out


# ---------------------------------------------------------------------------
# RMS norm with the residual's addition
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=512)
def _rmsnorm_plan(sizes, *strides):
    _fit_int(sizes[:4])   # B, H, L, D
    desc = RMSNormDesc(*sizes, *(Strides(*s) for s in strides))
    return desc, ctypes.byref(desc), int(lib().dr_rmsnorm_bwd_workspace_bytes(ctypes.byref(desc)))


def _new_f32(like, shape, device):
    """A new fp32 tensor, from another one if there is one (less work than by a device)."""
    return _torch().empty(shape, dtype=_torch().float32, device=device) if like is None else like.new_empty(shape)


def _rmsnorm_fwd(x, weight, residual, eps, out_dtype, block, y, scale, rstd, total, stream):
    torch = _torch()
    e4m3 = block is not None
    dims, steps, per_head, _ = _norm_args(x, None, weight, None)
    dev, lead = x.device, x.shape[:-1]
    if residual is not None:
        _need_rows(residual, "residual", dev, None, x.shape)
    elif total is not None:
        raise ValueError("total is the sum with the residual: there is none")
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x, dtype=torch.float8_e4m3fn if e4m3 else out_dtype)
        else:
            _need_rows(y, "y", dev, torch.float8_e4m3fn if e4m3 else out_dtype, x.shape)
        if rstd is None:
            rstd = _new_f32(weight, lead, dev)
        else:
            _need_on(rstd, "rstd", dev, torch.float32, lead)
        if e4m3:
            if block not in (0, 128):
                raise ValueError(f"block must be 128 (columns of a scale) or 0 (a row), got {block!r}")
            shape = lead + ((x.shape[-1] + 127) // 128 if block else 1,)
            if scale is None:
                scale = _new_f32(weight, shape, dev)
            else:
                _need_on(scale, "scale", dev, torch.float32, shape)
        if residual is not None:
            if total is None:
                total = torch.empty_like(residual)
            else:
                _need_rows(total, "total", dev, residual.dtype, x.shape)
        none = (0, 0, 0)
        more = [none if t is None else steps if t.stride() == x.stride() else _norm_dims(t, per_head)[1]
                for t in (residual, y, total)]
        _, desc, _ = _rmsnorm_plan(dims + (int(per_head), _dtype_code(x.dtype),
                                           _dtype_code(x.dtype if residual is None else residual.dtype),
                                           DR_F32 if e4m3 else _dtype_code(y.dtype), DR_F32, float(eps), block or 0),
                                   steps, *more, none)
        if e4m3:
            _check(lib().dr_rmsnorm_fwd_e4m3(desc, _ptr(x), _ptr(residual), _ptr(weight), _ptr(y), _ptr(scale),
                                             _ptr(total), _ptr(rstd), st))
        else:
            _check(lib().dr_rmsnorm_fwd(desc, _ptr(x), _ptr(residual), _ptr(weight), _ptr(y), _ptr(total),
                                        _ptr(rstd), st))
    return y, scale, rstd, total


def dr_rmsnorm_fwd(x, weight=None, residual=None, *, eps: float = 1e-5, out_dtype=None, y=None, rstd=None, total=None,
                   stream=None):
    """RMS norm over the last dimension of s = x + residual: y = s rstd weight,
    rstd = 1 / sqrt(mean(s^2) + eps); returns (y, rstd, total).

    x: [N,D], [B,L,D] or [B,H,L,D] (bf16 or fp32) with a weight [D] fp32 (None:
    ones); or, with one weight per head [H,D], [N,H,D] or [B,H,L,D].  residual: x's
    shape, of x's dtype or fp32; total is the sum in its dtype (None without one), and
    may be the residual itself.
    y and rstd come from the sum before that rounding.  Channels are contiguous,
    other strides free, rows start at any element.  y defaults to out_dtype (x's
    dtype) in x's order of dimensions; rstd is fp32, of x's leading shape.
    """
    y, _, rstd, total = _rmsnorm_fwd(x, weight, residual, eps, out_dtype, None, y, None, rstd, total, stream)
    return y, rstd, total


def dr_rmsnorm_fwd_e4m3(x, weight=None, residual=None, *, eps: float = 1e-5, block: int = 128, y=None, scale=None,
                        rstd=None, total=None, stream=None):
    """dr_rmsnorm_fwd with y in 8 bits (torch.float8_e4m3fn) and scales: y is near
    scale * code.  block 128: a scale for each 128 columns, [..., ceil(D/128)]; 0: one
    for a row, [..., 1].  Returns (y, scale, rstd, total)."""
    if block is None:
        raise ValueError("block must be 128 (columns of a scale) or 0 (a row), got None")
    return _rmsnorm_fwd(x, weight, residual, eps, None, block, y, scale, rstd, total, stream)


def dr_rmsnorm_bwd_workspace_bytes(desc: RMSNormDesc) -> int:
    return int(lib().dr_rmsnorm_bwd_workspace_bytes(ctypes.byref(desc)))


def dr_rmsnorm_bwd(x, weight, rstd, dy, ds=None, *, per_head=None, grad_dtype=None, dx=None, want_sums: bool = True,
                   workspace=None, stream=None):
    """Gradients of dr_rmsnorm_fwd: dx, of x and of the residual, in grad_dtype (x's
    dtype) and in x's order of dimensions, and dweight fp32 (None with
    want_sums=False), in a dict.  x is the forward's total (its x without a
    residual) and rstd its rstd; dy (bf16 or fp32) has x's shape, and so has ds, the
    gradient that reaches the total besides (None: none).  Without a weight,
    per_head=True makes dweight one per head."""
    torch = _torch()
    if weight is not None and per_head is not None and per_head != (weight.dim() == 2):
        raise ValueError("per_head does not fit the weight's shape")
    dims, steps, per_head, wshape = _norm_args(x, per_head, weight, None)
    dev, lead = x.device, x.shape[:-1]
    _need_on(rstd, "rstd", dev, torch.float32, lead)
    _need_rows(dy, "dy", dev, None, x.shape)
    if ds is not None:
        _need_rows(ds, "ds", dev, None, x.shape)
    with _on(dev, stream) as st:
        if dx is None:
            dx = torch.empty_like(x, dtype=grad_dtype)
        else:
            _need_rows(dx, "dx", dev, grad_dtype, x.shape)
        none = (0, 0, 0)
        sds, sdx, sdy = (none if t is None else steps if t.stride() == x.stride() else _norm_dims(t, per_head)[1]
                         for t in (ds, dx, dy))
        _, desc, nbytes = _rmsnorm_plan(dims + (int(per_head), _dtype_code(x.dtype),
                                                _dtype_code(x.dtype if ds is None else ds.dtype),
                                                _dtype_code(dx.dtype), _dtype_code(dy.dtype), 0.0, 0),
                                        steps, sds, sdx, none, sdy)
        out = {"dx": dx, "dweight": None}
        wbytes = 0
        if want_sums:
            out["dweight"] = (torch.empty(wshape, dtype=torch.float32, device=dev) if weight is None else
                              torch.empty_like(weight))
            workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_rmsnorm_bwd(desc, _ptr(x), _ptr(weight), _ptr(rstd), _ptr(dy), _ptr(ds), _ptr(dx),
                                    _ptr(out["dweight"]), _ptr(workspace), wbytes, st))
    return out


# ---------------------------------------------------------------------------
# short causal convolution; gated linear recurrence
# ---------------------------------------------------------------------------

def _seq_strides(t):
    """The strides of a [B,L,C] view in elements (0 where a dimension is 1)."""
    n, s = t.shape, t.stride()
    return (s[0] if n[0] > 1 else 0, 0, s[1] if n[1] > 1 else 0)


def _need_seq(t, name, device=None, dtype=None, shape=None, dims=3):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a [B, L, C] tensor" if dims == 3 else f"{name} must be a [B, C] tensor")
    _need_rows(t, name, device, dtype, shape)


def _mode(value, modes, name):
    if value not in modes:
        raise ValueError(f"{name} must be one of {sorted(modes)}, got {value!r}")
    return modes[value]


@functools.lru_cache(maxsize=512)
def _short_conv_plan(sizes, *strides):
    _fit_int(sizes[:4])   # B, L, C, W
    desc = ShortConvDesc(*sizes, *(Strides(*s) for s in strides))
    return desc, ctypes.byref(desc), int(lib().dr_short_conv_bwd_workspace_bytes(ctypes.byref(desc)))


def _conv_args(C, weight, bias, dev):
    torch = _torch()
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [C, W] tensor")
    W = weight.shape[1]
    _need_on(weight, "weight", dev, torch.float32, (C, W))
    if bias is not None:
        _need_on(bias, "bias", dev, torch.float32, (C,))
    return W


def dr_short_conv_fwd(x, weight, bias=None, state=None, *, activation: str = "silu", out_dtype=None, y=None,
                      state_out=None, want_state: bool = True, stream=None):
    """Causal convolution of each channel over W tokens, z_t = bias + sum_j weight_j
    x_{t-W+1+j}, and y = z sigmoid(z) ("silu") or z ("none"); returns (y, state_out).

    x: [B,L,C] bf16 or fp32, channels contiguous, other strides free (a slice of a
    fused projection); weight [C,W] fp32, W in 2..8; bias [C] fp32 or None; state
    [B,W-1,C] in x's dtype, the inputs before the first, oldest first (None: zeros).
    state_out are the last W-1 inputs; it may be state itself; with
    want_state=False and no state_out none is written and None is returned.  y
    defaults to out_dtype (x's dtype) in x's order of dimensions.
    """
    torch = _torch()
    act = _mode(activation, ACTIVATIONS, "activation")
    _need_seq(x, "x")
    dev = x.device
    B, L, C = x.shape
    W = _conv_args(C, weight, bias, dev)
    if state is not None:
        _need_on(state, "state", dev, x.dtype, (B, W - 1, C))
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype)
        else:
            _need_seq(y, "y", dev, out_dtype, x.shape)
        if state_out is not None:
            _need_on(state_out, "state_out", dev, x.dtype, (B, W - 1, C))
        elif want_state:
            state_out = torch.empty((B, max(W - 1, 0), C), dtype=x.dtype, device=dev) if state is None else torch.empty_like(state)
        _, desc, _ = _short_conv_plan((B, L, C, W, _dtype_code(x.dtype), _dtype_code(y.dtype), DR_F32, act),
                                      _seq_strides(x), _seq_strides(y), (0, 0, 0))
        _check(lib().dr_short_conv_fwd(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), _ptr(state_out), st))
    return y, state_out


def dr_short_conv_bwd_workspace_bytes(desc: ShortConvDesc) -> int:
    return int(lib().dr_short_conv_bwd_workspace_bytes(ctypes.byref(desc)))


def dr_short_conv_bwd(x, weight, bias, state, dy, dstate_out=None, *, activation: str = "silu", grad_dtype=None,
                      want_sums: bool = True, want_dstate: bool = True, workspace=None, stream=None):
    """Gradients of dr_short_conv_fwd for the loss whose gradients with respect to y
    and state_out are dy [B,L,C] (bf16 or fp32) and dstate_out [B,W-1,C] (fp32; None:
    zero).  Returns a dict: dx in grad_dtype (x's dtype) and in x's order of
    dimensions; dweight, dbias fp32 (None with want_sums=False); dstate, of the
    initial state, fp32 (None with want_dstate=False)."""
    torch = _torch()
    act = _mode(activation, ACTIVATIONS, "activation")
    _need_seq(x, "x")
    dev = x.device
    B, L, C = x.shape
    W = _conv_args(C, weight, bias, dev)
    if state is not None:
        _need_on(state, "state", dev, x.dtype, (B, W - 1, C))
    _need_seq(dy, "dy", dev, None, x.shape)
    if dstate_out is not None:
        _need_on(dstate_out, "dstate_out", dev, torch.float32, (B, W - 1, C))
    with _on(dev, stream) as st:
        out = {"dx": torch.empty_like(x, dtype=grad_dtype), "dweight": None, "dbias": None,
               "dstate": _state(dstate_out, (B, max(W - 1, 0), C), dev) if want_dstate else None}
        _, desc, nbytes = _short_conv_plan((B, L, C, W, _dtype_code(x.dtype), _dtype_code(out["dx"].dtype),
                                            _dtype_code(dy.dtype), act),
                                           _seq_strides(x), _seq_strides(out["dx"]), _seq_strides(dy))
        wbytes = 0
        if want_sums:
            out["dweight"] = torch.empty_like(weight)
            out["dbias"] = torch.empty((C,), dtype=torch.float32, device=dev) if bias is None else torch.empty_like(bias)
            workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_short_conv_bwd(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(dy), _ptr(dstate_out),
                                       _ptr(out["dx"]), _ptr(out["dweight"]), _ptr(out["dbias"]), _ptr(out["dstate"]),
                                       _ptr(workspace), wbytes, st))
    return out


def dr_short_conv_step(state, x, weight, bias=None, *, activation: str = "silu", out_dtype=None, y=None, stream=None):
    """One token of the short convolution for N states [N,W-1,C] (x's dtype, updated
    in place); x: [N,C]; returns y [N,C]."""
    torch = _torch()
    act = _mode(activation, ACTIVATIONS, "activation")
    _need(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a [N, C] tensor")
    dev = x.device
    N, C = x.shape
    W = _conv_args(C, weight, bias, dev)
    _need_on(state, "state", dev, x.dtype, (N, W - 1, C))
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype)
        else:
            _need_on(y, "y", dev, out_dtype, (N, C))
        none = (0, 0, 0)
        _, desc, _ = _short_conv_plan((N, 1, C, W, _dtype_code(x.dtype), _dtype_code(y.dtype), DR_F32, act),
                                      none, none, none)
        _check(lib().dr_short_conv_step(desc, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), st))
    return y


@functools.lru_cache(maxsize=512)
def _gated_scan_plan(bwd: bool, sizes, *strides):
    _fit_int(sizes[:3])   # B, L, C
    desc = GatedScanDesc(*sizes, *(Strides(*s) for s in strides))
    fn = lib().dr_gated_scan_bwd_workspace_bytes if bwd else lib().dr_gated_scan_fwd_workspace_bytes
    return desc, ctypes.byref(desc), int(fn(ctypes.byref(desc)))


def dr_gated_scan_fwd_workspace_bytes(desc: GatedScanDesc) -> int:
    return int(lib().dr_gated_scan_fwd_workspace_bytes(ctypes.byref(desc)))


def dr_gated_scan_bwd_workspace_bytes(desc: GatedScanDesc) -> int:
    return int(lib().dr_gated_scan_bwd_workspace_bytes(ctypes.byref(desc)))


def dr_gated_scan_fwd(x, gate, h0=None, *, decay: str, inputs: str = "plain", out_dtype=None, h=None, h_final=None,
                      want_state: bool = True, workspace=None, stream=None):
    """Gated linear recurrence of each channel, h_t = a_t h_{t-1} + c(a_t) x_t over
    [B,L,C] device tensors; returns (h, h_final).

    x: bf16 or fp32; gate: x's dtype or fp32; channels contiguous, other strides
    free.  decay "log": a = e^gate (-inf starts anew); "logit": a = sigmoid(gate).
    inputs "plain": c = 1; "blend": 1 - a; "unit": sqrt(1 - a^2).  h0: [B,C] fp32 or
    None.  h defaults to out_dtype (fp32) in x's order of dimensions; h_final may be
    h0 itself; with want_state=False and no h_final none is written and None is
    returned for it.
    """
    torch = _torch()
    modes = _mode(decay, SCAN_DECAYS, "decay"), _mode(inputs, SCAN_INPUTS, "inputs")
    _need_seq(x, "x")
    dev = x.device
    B, L, C = x.shape
    _need_seq(gate, "gate", dev, None, x.shape)
    if h0 is not None:
        _need_on(h0, "h0", dev, torch.float32, (B, C))
    with _on(dev, stream) as st:
        if h is None:
            h = torch.empty_like(x, dtype=torch.float32 if out_dtype is None else out_dtype)
        else:
            _need_seq(h, "h", dev, out_dtype, x.shape)
        if h_final is not None:
            _need_on(h_final, "h_final", dev, torch.float32, (B, C))
        elif want_state:
            h_final = _state(h0, (B, C), dev)
        none = (0, 0, 0)
        _, desc, nbytes = _gated_scan_plan(
            False, (B, L, C, _dtype_code(x.dtype), _dtype_code(gate.dtype), _dtype_code(h.dtype), DR_F32, DR_F32) + modes,
            _seq_strides(x), _seq_strides(gate), _seq_strides(h), none, none, none)
        workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_gated_scan_fwd(desc, _ptr(x), _ptr(gate), _ptr(h0), _ptr(h), _ptr(h_final), _ptr(workspace),
                                       wbytes, st))
    return h, h_final


def dr_gated_scan_bwd(x, gate, h0, h, dh, dh_final=None, *, decay: str, inputs: str = "plain", grad_dtype=None,
                      want_dh0: bool = True, workspace=None, stream=None):
    """Gradients of dr_gated_scan_fwd for the loss whose gradients with respect to h
    and h_final are dh [B,L,C] (bf16 or fp32) and dh_final [B,C] (fp32; None: zero);
    h is what the forward returned.  Returns a dict: dx and dgate in grad_dtype
    (fp32) and in their inputs' order of dimensions, dh0 [B,C] fp32 (None with
    want_dh0=False)."""
    torch = _torch()
    modes = _mode(decay, SCAN_DECAYS, "decay"), _mode(inputs, SCAN_INPUTS, "inputs")
    _need_seq(x, "x")
    dev = x.device
    B, L, C = x.shape
    _need_seq(gate, "gate", dev, None, x.shape)
    _need_seq(h, "h", dev, None, x.shape)
    _need_seq(dh, "dh", dev, None, x.shape)
    if h0 is not None:
        _need_on(h0, "h0", dev, torch.float32, (B, C))
    if dh_final is not None:
        _need_on(dh_final, "dh_final", dev, torch.float32, (B, C))
    to = torch.float32 if grad_dtype is None else grad_dtype
    with _on(dev, stream) as st:
        out = {"dx": torch.empty_like(x, dtype=to), "dgate": torch.empty_like(gate, dtype=to),
               "dh0": _state(h0, (B, C), dev) if want_dh0 else None}
        _, desc, nbytes = _gated_scan_plan(
            True, (B, L, C, _dtype_code(x.dtype), _dtype_code(gate.dtype), _dtype_code(h.dtype), _dtype_code(dh.dtype),
                   _dtype_code(to)) + modes,
            *(_seq_strides(t) for t in (x, gate, h, dh, out["dx"], out["dgate"])))
        workspace, wbytes = _workspace(workspace, nbytes, dev)
        _check(lib().dr_gated_scan_bwd(desc, _ptr(x), _ptr(gate), _ptr(h0), _ptr(h), _ptr(dh), _ptr(dh_final),
                                       _ptr(out["dx"]), _ptr(out["dgate"]), _ptr(out["dh0"]), _ptr(workspace), wbytes, st))
    return out


def dr_gated_scan_step(state, x, gate, *, decay: str, inputs: str = "plain", out_dtype=None, h=None, stream=None):
    """One token of the gated recurrence for N states [N,C] (fp32, updated in place);
    x and gate: [N,C]; returns h [N,C], the new state in out_dtype (fp32)."""
    torch = _torch()
    modes = _mode(decay, SCAN_DECAYS, "decay"), _mode(inputs, SCAN_INPUTS, "inputs")
    _need(state, "state", torch.float32)
    if state.dim() != 2:
        raise ValueError("state must be a [N, C] tensor")
    dev, (N, C) = state.device, state.shape
    _need_on(x, "x", dev, None, (N, C))
    _need_on(gate, "gate", dev, None, (N, C))
    with _on(dev, stream) as st:
        if h is None:
            h = torch.empty_like(x, dtype=torch.float32 if out_dtype is None else out_dtype)
        else:
            _need_on(h, "h", dev, out_dtype, (N, C))
        none = (0, 0, 0)
        _, desc, _ = _gated_scan_plan(False, (N, 1, C, _dtype_code(x.dtype), _dtype_code(gate.dtype),
                                              _dtype_code(h.dtype), DR_F32, DR_F32) + modes, *(none,) * 6)
        _check(lib().dr_gated_scan_step(desc, _ptr(x), _ptr(gate), _ptr(state), _ptr(h), st))
    return h
