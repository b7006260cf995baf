"""ctypes binding of the C ABI in include/gdn.h.

Argument marshalling only: each function takes torch tensors that already
live on the GPU (or None), passes their device pointers, row strides and the
current stream to the entry point of the same name, and raises GDNError on a
non-OK status.  Every step of the mixer runs in the library's CUDA kernels;
if the compiled library is missing, loading it raises -- there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

from . import build_lib

GDN_BF16, GDN_FP32 = 0, 1
GDN_FLAG_L2NORM_QK = 1
DEVERR_CU_SEQLENS, DEVERR_SLOT, DEVERR_TIMEOUT, DEVERR_PAGE = 1, 2, 4, 8
STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED",
          3: "GDN_ERR_WORKSPACE", 4: "GDN_ERR_CUDA", 5: "GDN_ERR_DEVICE"}


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, STATUS.get(status, str(status))))


class Config(ctypes.Structure):
    _fields_ = [("hk", ctypes.c_int32), ("hv", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("chunk", ctypes.c_int32), ("act", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("q_scale", ctypes.c_float),
                ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float)]


class MixerIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64),
                ("z", ctypes.c_void_p), ("ld_z", ctypes.c_int64),
                ("u", ctypes.c_void_p), ("b_logit", ctypes.c_void_p), ("ld_ub", ctypes.c_int64),
                ("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("norm_w", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("T", ctypes.c_int64),
                ("state_idx", ctypes.c_void_p), ("state_in", ctypes.c_void_p),
                ("state_out", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int32)]


class SSMConfig(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("heads", ctypes.c_int32), ("d_state", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("act", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class SSMIO(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld_x", ctypes.c_int64), ("b", ctypes.c_void_p),
                ("c", ctypes.c_void_p), ("ld_bc", ctypes.c_int64), ("dt", ctypes.c_void_p),
                ("ld_dt", ctypes.c_int64), ("z", ctypes.c_void_p), ("ld_z", ctypes.c_int64),
                ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("conv_w", ctypes.c_void_p), ("conv_bias", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("T", ctypes.c_int64),
                ("state_idx", ctypes.c_void_p), ("state_in", ctypes.c_void_p),
                ("state_out", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("y", ctypes.c_void_p)]


class BlockNormIO(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("act", ctypes.c_int32),
                ("res", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("res_scale", ctypes.c_float),
                ("block", ctypes.c_void_p), ("ld_block", ctypes.c_int64),
                ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64), ("gate_cols", ctypes.c_int32),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
                ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
                ("res_out", ctypes.c_void_p), ("ld_res_out", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("ld_h", ctypes.c_int64),
                ("rstd_post", ctypes.c_void_p), ("rstd_pre", ctypes.c_void_p),
                ("dh", ctypes.c_void_p), ("ld_dh", ctypes.c_int64),
                ("d_res_out", ctypes.c_void_p), ("ld_d_res_out", ctypes.c_int64),
                ("d_residual", ctypes.c_void_p), ("ld_d_residual", ctypes.c_int64),
                ("d_block", ctypes.c_void_p), ("ld_d_block", ctypes.c_int64),
                ("d_gate", ctypes.c_void_p), ("ld_d_gate", ctypes.c_int64),
                ("dw_post", ctypes.c_void_p), ("dw_pre", ctypes.c_void_p)]


class AttnConfig(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("act", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("n_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class AttnPrepIO(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("ld_q", ctypes.c_int64), ("hs_q", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("ld_k", ctypes.c_int64), ("hs_k", ctypes.c_int64),
                ("v", ctypes.c_void_p), ("ld_v", ctypes.c_int64), ("hs_v", ctypes.c_int64),
                ("T", ctypes.c_int64), ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
                ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("n_seqs", ctypes.c_int32),
                ("rows", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
                ("dq_out", ctypes.c_void_p), ("dk_out", ctypes.c_void_p),
                ("dq", ctypes.c_void_p), ("ld_dq", ctypes.c_int64), ("hs_dq", ctypes.c_int64),
                ("dk", ctypes.c_void_p), ("ld_dk", ctypes.c_int64), ("hs_dk", ctypes.c_int64),
                ("dw_q", ctypes.c_void_p), ("dw_k", ctypes.c_void_p)]


class AttnDecodeIO(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("ld_q", ctypes.c_int64), ("hs_q", ctypes.c_int64),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("tokens", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()
LIB_PATH = build_lib.LIB


def header_entry_points():
    """Names of the functions declared in include/gdn.h."""
    txt = open(os.path.join(build_lib.INCLUDE, "gdn.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", txt)))


def load(path: str | None = None):
    """Load the compiled library (building it first if sources are newer)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if path is None and build_lib.needs_build():
            build_lib.build()
        if not os.path.exists(p):
            raise RuntimeError("GDN CUDA library not found at %s; run build()" % p)
        lib = ctypes.CDLL(p)
        V, P, I32, I64, U32, SZ = (ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                   ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t)
        CP = ctypes.POINTER(Config)
        sig = {
            "gdn_workspace_size": ([CP, I64, I32], SZ),
            "gdn_gate_prep": ([CP, P, P, I64, I64, P, P, P, P, V], I32),
            "gdn_conv1d_prefill": ([CP, P, I64, P, I32, I64, P, P, P, P, I32, V], I32),
            "gdn_conv1d_step": ([CP, P, I64, I32, P, P, P, P, I32, V], I32),
            "gdn_chunk_prefill": ([CP, P, P, I64, P, I64, I32, P, P, P, I32, I64, P, P, P, P, I32,
                                   U32, P, SZ, V], I32),
            "gdn_recurrent_decode": ([CP, P, P, I64, P, I64, I32, P, P, I32, P, P, P, I32, U32, V],
                                     I32),
            "gdn_gated_rmsnorm": ([CP, P, I32, P, I64, P, I64, P, I32, V], I32),
            "gdn_mixer_prefill": ([CP, ctypes.POINTER(MixerIO), P, SZ, V], I32),
            "gdn_mixer_decode": ([CP, ctypes.POINTER(MixerIO), P, SZ, V], I32),
            "gdn_mixer_prefill_static": ([CP, ctypes.POINTER(MixerIO), V], I32),
            "gdn_state_copy": ([CP, P, P, I32, P, P, I32, P, P, I32, V], I32),
            "gdn_mixer_verify": ([CP, ctypes.POINTER(MixerIO), I32, P, P, SZ, V], I32),
            "gdn_backward_workspace_size": ([CP, I64, I32], SZ),
            "gdn_state_to_q8": ([CP, P, P, P, P, U32, V], I32),
            "gdn_state_from_q8": ([CP, P, P, P, V], I32),
            "gdn_mixer_decode_q8": ([CP, ctypes.POINTER(MixerIO), P, P, P, U32, P, SZ, V], I32),
            "gdn_chunk_states": ([CP, P, I64, P, I64, I32, P, P, P, I32, I64, P, P, P, P, P, SZ, V], I32),
            "gdn_chunk_backward": ([CP, P, P, I64, P, I64, I32, P, P, P, I32, I64, P, P, P, P, P, P, P,
                                    I64, P, P, P, P, P, SZ, V], I32),
            "gdn_ssm_workspace_size": ([ctypes.POINTER(SSMConfig), I64, I32], SZ),
            "gdn_ssm_conv_prefill": ([ctypes.POINTER(SSMConfig), P, I64, P, I32, I64, P, P, P, P, P, V],
                                     I32),
            "gdn_ssm_prefill": ([ctypes.POINTER(SSMConfig), ctypes.POINTER(SSMIO), P, SZ, V], I32),
            "gdn_ssm_decode": ([ctypes.POINTER(SSMConfig), ctypes.POINTER(SSMIO), P, SZ, V], I32),
            "gdn_block_norm": ([ctypes.POINTER(BlockNormIO), V], I32),
            "gdn_block_norm_workspace_size": ([I64, I32], SZ),
            "gdn_block_norm_backward": ([ctypes.POINTER(BlockNormIO), P, SZ, V], I32),
            "gdn_attn_prep": ([ctypes.POINTER(AttnConfig), P, V], I32),
            "gdn_attn_prep_workspace_size": ([ctypes.POINTER(AttnConfig), I64], SZ),
            "gdn_attn_prep_backward": ([ctypes.POINTER(AttnConfig), P, P, SZ, V], I32),
            "gdn_attn_workspace_size": ([ctypes.POINTER(AttnConfig), I32, I32], SZ),
            "gdn_attn_decode": ([ctypes.POINTER(AttnConfig), P, P, SZ, V], I32),
            "gdn_page_workspace_size": ([ctypes.POINTER(AttnConfig), I32], SZ),
            "gdn_page_resize": ([ctypes.POINTER(AttnConfig), P, P, P, P, P, I32, P, P, P, P, SZ, V], I32),
            "gdn_page_fork": ([ctypes.POINTER(AttnConfig), P, P, P, P, P, I32, V], I32),
            "gdn_page_compact": ([ctypes.POINTER(AttnConfig), P, P, P, P, P, P, P, I32, P, SZ, V], I32),
            "gdn_page_copy": ([ctypes.POINTER(AttnConfig), P, P, I32, P, P, I32, P, P, I32, V], I32),
            "gdn_device_error": ([V, ctypes.POINTER(U32)], I32),
            "gdn_debug_set_wait": ([ctypes.c_uint64, U32], I32),
            "gdn_status_string": ([I32], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


# ---------------------------------------------------------------- helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _ld(t):
    if t is None:
        return 0
    return t.stride(0) if t.dim() > 1 else t.shape[0]


def _dt(t):
    import torch
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_FP32
    raise TypeError("unsupported dtype %s" % t.dtype)


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def _check(st, where):
    if st != 0:
        raise GDNError(st, where)


def make_config(HK, HV, dk, dv, chunk=64, act="bf16", n_slots=0, q_scale=1.0, l2_eps=1e-6,
                norm_eps=1e-6) -> Config:
    return Config(HK, HV, dk, dv, chunk, GDN_BF16 if act == "bf16" else GDN_FP32, n_slots,
                  q_scale, l2_eps, norm_eps)


# ------------------------------------------------------------ entry points

def gdn_workspace_size(cfg, max_tokens, max_seqs):
    return load().gdn_workspace_size(ctypes.byref(cfg), max_tokens, max_seqs)


def gdn_gate_prep(cfg, u, b_logit, A_log, dt_bias, g, beta, stream=None):
    T = u.shape[0]
    _check(load().gdn_gate_prep(ctypes.byref(cfg), _ptr(u), _ptr(b_logit), _ld(u), T,
                                _ptr(A_log), _ptr(dt_bias), _ptr(g), _ptr(beta),
                                _stream(stream)), "gdn_gate_prep")


def gdn_conv1d_prefill(cfg, x, cu_seqlens, w, conv_state, state_idx, out, stream=None):
    _check(load().gdn_conv1d_prefill(ctypes.byref(cfg), _ptr(x), _ld(x), _ptr(cu_seqlens),
                                     cu_seqlens.shape[0] - 1, x.shape[0], _ptr(w),
                                     _ptr(conv_state), _ptr(state_idx), _ptr(out), _dt(out),
                                     _stream(stream)), "gdn_conv1d_prefill")


def gdn_conv1d_step(cfg, x, w, conv_state, state_idx, out, stream=None):
    _check(load().gdn_conv1d_step(ctypes.byref(cfg), _ptr(x), _ld(x), x.shape[0], _ptr(w),
                                  _ptr(conv_state), _ptr(state_idx), _ptr(out), _dt(out),
                                  _stream(stream)), "gdn_conv1d_step")


def gdn_chunk_prefill(cfg, q, k, v, g, beta, cu_seqlens, state_in, state_out, state_idx, o,
                      flags=GDN_FLAG_L2NORM_QK, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_chunk_prefill(ctypes.byref(cfg), _ptr(q), _ptr(k), _ld(q), _ptr(v), _ld(v),
                                    _dt(q), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                    cu_seqlens.shape[0] - 1, q.shape[0], _ptr(state_in),
                                    _ptr(state_out), _ptr(state_idx), _ptr(o), _dt(o), flags,
                                    _ptr(workspace), ws_bytes, _stream(stream)),
           "gdn_chunk_prefill")


def gdn_recurrent_decode(cfg, q, k, v, g, beta, state, state_idx, o, flags=GDN_FLAG_L2NORM_QK,
                         stream=None):
    _check(load().gdn_recurrent_decode(ctypes.byref(cfg), _ptr(q), _ptr(k), _ld(q), _ptr(v),
                                       _ld(v), _dt(q), _ptr(g), _ptr(beta), q.shape[0],
                                       _ptr(state), _ptr(state_idx), _ptr(o), _dt(o), flags,
                                       _stream(stream)), "gdn_recurrent_decode")


def gdn_gated_rmsnorm(cfg, o, z, w, y, stream=None):
    _check(load().gdn_gated_rmsnorm(ctypes.byref(cfg), _ptr(o), _dt(o), _ptr(z), _ld(z), _ptr(w),
                                    o.shape[0], _ptr(y), _dt(y), _stream(stream)),
           "gdn_gated_rmsnorm")


def _mixer_io(x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, cu_seqlens, state_in, state_out,
              conv_state, state_idx, y, n_seqs):
    return MixerIO(_ptr(x), _ld(x), _ptr(z), _ld(z), _ptr(u), _ptr(b_logit), _ld(u),
                   _ptr(conv_w), _ptr(A_log), _ptr(dt_bias), _ptr(norm_w), _ptr(cu_seqlens),
                   n_seqs, x.shape[0], _ptr(state_idx), _ptr(state_in), _ptr(state_out),
                   _ptr(conv_state), _ptr(y), _dt(y))


def gdn_mixer_prefill(cfg, x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, cu_seqlens, y,
                      state_in=None, state_out=None, conv_state=None, state_idx=None,
                      workspace=None, stream=None):
    io = _mixer_io(x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, cu_seqlens, state_in,
                   state_out, conv_state, state_idx, y, cu_seqlens.shape[0] - 1)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_mixer_prefill(ctypes.byref(cfg), ctypes.byref(io), _ptr(workspace),
                                    ws_bytes, _stream(stream)), "gdn_mixer_prefill")


def gdn_mixer_prefill_static(cfg, x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, cu_seqlens, y,
                             state_in=None, state_out=None, conv_state=None, state_idx=None,
                             stream=None):
    """gdn_mixer_prefill without a workspace: the library's fixed scratch is used."""
    io = _mixer_io(x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, cu_seqlens, state_in,
                   state_out, conv_state, state_idx, y, cu_seqlens.shape[0] - 1)
    _check(load().gdn_mixer_prefill_static(ctypes.byref(cfg), ctypes.byref(io), _stream(stream)),
           "gdn_mixer_prefill_static")


def gdn_mixer_decode(cfg, x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, y, state,
                     conv_state, workspace, state_idx=None, stream=None):
    """workspace: a device byte tensor of gdn_workspace_size(cfg, n, n) bytes or more."""
    io = _mixer_io(x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, None, state, state,
                   conv_state, state_idx, y, x.shape[0])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_mixer_decode(ctypes.byref(cfg), ctypes.byref(io), _ptr(workspace), ws_bytes,
                                   _stream(stream)), "gdn_mixer_decode")


def gdn_state_to_q8(cfg, state, codes, scales, frame, stream=None, residual=None):
    """residual (bf16 [slots][HV][dk][dv], optional): written for an error-feedback pool."""
    _check(load().gdn_state_to_q8(ctypes.byref(cfg), _ptr(state), _ptr(codes), _ptr(scales),
                                  _ptr(residual), frame, _stream(stream)), "gdn_state_to_q8")


def gdn_state_from_q8(cfg, codes, scales, state, stream=None):
    _check(load().gdn_state_from_q8(ctypes.byref(cfg), _ptr(codes), _ptr(scales), _ptr(state),
                                    _stream(stream)), "gdn_state_from_q8")


def gdn_mixer_decode_q8(cfg, x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, y, codes, scales,
                        conv_state, frame, workspace, state_idx=None, stream=None, residual=None):
    """gdn_mixer_decode on a Q8 state pool (codes int8 [slots][HV][dk][dv], scales fp32
    [slots][HV][dk]); `frame` keys the rounding dither and should change every step.  A bf16
    `residual` pool of the codes' shape turns error feedback on."""
    io = _mixer_io(x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, None, None, None,
                   conv_state, state_idx, y, x.shape[0])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_mixer_decode_q8(ctypes.byref(cfg), ctypes.byref(io), _ptr(codes), _ptr(scales),
                                      _ptr(residual), frame, _ptr(workspace), ws_bytes, _stream(stream)),
           "gdn_mixer_decode_q8")


def gdn_backward_workspace_size(cfg, max_tokens, max_seqs) -> int:
    return load().gdn_backward_workspace_size(ctypes.byref(cfg), max_tokens, max_seqs)


def chunk_count(seqlens, chunk):
    """Boundary states of a batch: sum over sequences of ceil(len / chunk)."""
    return sum((int(L) + chunk - 1) // chunk for L in seqlens)


def gdn_chunk_states(cfg, k, v, g, beta, cu_seqlens, boundary_states, workspace, state_in=None,
                     state_idx=None, token_pw=None, stream=None):
    """token_pw: optional fp32 [T, HV, 2, dv] that receives every token's p and w, for
    gdn_chunk_backward's token_pw."""
    T = k.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_chunk_states(ctypes.byref(cfg), _ptr(k), _ld(k), _ptr(v), _ld(v), _dt(k),
                                   _ptr(g), _ptr(beta), _ptr(cu_seqlens), cu_seqlens.shape[0] - 1, T,
                                   _ptr(state_in), _ptr(state_idx), _ptr(boundary_states),
                                   _ptr(token_pw), _ptr(workspace), ws_bytes, _stream(stream)),
           "gdn_chunk_states")


def gdn_chunk_backward(cfg, q, k, v, g, beta, cu_seqlens, boundary_states, d_o, dq, dk, dv, dg,
                       dbeta, workspace, d_state_out=None, d_state_in=None, state_idx=None,
                       token_pw=None, stream=None):
    """token_pw: None, or the buffer gdn_chunk_states filled for the same batch."""
    T = q.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_chunk_backward(ctypes.byref(cfg), _ptr(q), _ptr(k), _ld(q), _ptr(v), _ld(v),
                                     _dt(q), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                     cu_seqlens.shape[0] - 1, T, _ptr(state_idx),
                                     _ptr(boundary_states), _ptr(token_pw), _ptr(d_o),
                                     _ptr(d_state_out), _ptr(dq),
                                     _ptr(dk), _ld(dq), _ptr(dv), _ptr(dg), _ptr(dbeta),
                                     _ptr(d_state_in), _ptr(workspace), ws_bytes, _stream(stream)),
           "gdn_chunk_backward")


def gdn_mixer_verify(cfg, x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, y, state,
                     conv_state, ckpt_idx, k, workspace, state_idx=None, stream=None):
    """k tokens per sequence (rows n*k .. n*k+k-1 of x, z, u, b_logit, y); the state and conv
    history after token j go to slot ckpt_idx[n] + j of the same pools."""
    n = x.shape[0] // k
    if n * k != x.shape[0]:
        raise ValueError("x holds %d rows, not a multiple of k=%d" % (x.shape[0], k))
    io = _mixer_io(x, z, u, b_logit, conv_w, A_log, dt_bias, norm_w, None, state, state,
                   conv_state, state_idx, y, x.shape[0])
    io.n_seqs = n
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_mixer_verify(ctypes.byref(cfg), ctypes.byref(io), k, _ptr(ckpt_idx),
                                   _ptr(workspace), ws_bytes, _stream(stream)), "gdn_mixer_verify")


def gdn_state_copy(cfg, src_state, src_conv, dst_state, dst_conv, src_idx, dst_idx, stream=None):
    """Snapshot / restore / reset: slot src_idx[i] -> slot dst_idx[i] (src < 0: reset to zeros,
    dst < 0: nothing).  The slot counts come from the pools' first dimension; src and dst may be
    the same tensors."""
    import torch
    CH = 2 * cfg.hk * cfg.dk + cfg.hv * cfg.dv
    act = torch.bfloat16 if cfg.act == GDN_BF16 else torch.float32
    for t in (src_state, dst_state):
        if t is not None and (tuple(t.shape[1:]) != (cfg.hv, cfg.dk, cfg.dv) or t.dtype != torch.float32
                              or not t.is_contiguous()):
            raise ValueError("state pools are contiguous fp32 [slots][HV][dk][dv]")
    for t in (src_conv, dst_conv):
        if t is not None and (tuple(t.shape[1:]) != (CH, 3) or t.dtype != act or not t.is_contiguous()):
            raise ValueError("history pools are contiguous [slots][CH][3] in the activation dtype")
    for t in (src_idx, dst_idx):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
            raise ValueError("slot indices are contiguous int32")
    if src_idx is not None and dst_idx is not None and src_idx.numel() != dst_idx.numel():
        raise ValueError("src_idx and dst_idx differ in length")

    def slots(*ts):
        return min([t.shape[0] for t in ts if t is not None] or [0])
    n = 0 if dst_idx is None else dst_idx.numel()
    _check(load().gdn_state_copy(ctypes.byref(cfg), _ptr(src_state), _ptr(src_conv),
                                 slots(src_state, src_conv), _ptr(dst_state), _ptr(dst_conv),
                                 slots(dst_state, dst_conv), _ptr(src_idx), _ptr(dst_idx), n,
                                 _stream(stream)), "gdn_state_copy")


# ------------------------------------- selective state space mixer, block norms

def make_ssm_config(groups, heads, d_state, head_dim, act="bf16", n_slots=0, dt_min=0.0,
                    dt_max=float("inf")) -> SSMConfig:
    return SSMConfig(groups, heads, d_state, head_dim, GDN_BF16 if act == "bf16" else GDN_FP32,
                     n_slots, dt_min, dt_max)


def _packer(cls):
    """Fill a ctypes structure from its fields' values in order, null pointers as 0: a third of the
    time that the structure's own constructor takes."""
    code = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    pack = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_)).pack
    tail = bytes(ctypes.sizeof(cls))
    size, make = len(tail), cls.from_buffer_copy

    def fill(*values):
        data = pack(*values)
        return make(data if len(data) == size else data + tail[len(data):])
    return fill


_ssm_io, _norm_io = _packer(SSMIO), _packer(BlockNormIO)
_torch = None


class _Args:
    """Checks of one call's tensors: all on the current device, of the expected type and shape.
    Pointers of missing ones are 0."""

    __slots__ = ("where", "device", "f32", "i32", "act")

    def __init__(self, where, act=None):
        global _torch
        if _torch is None:
            import torch
            torch.cuda.current_device()             # initialises CUDA
            _torch = torch
        self.where, self.device = where, _torch._C._cuda_getDevice()
        self.f32, self.i32 = _torch.float32, _torch.int32
        if act is not None:
            self.act = _torch.bfloat16 if act == GDN_BF16 else _torch.float32

    def refuse(self, name, what):
        raise ValueError("%s: %s %s" % (self.where, name, what))

    def explain(self, t, name, shape, dtype):
        if t.dtype != dtype:
            self.refuse(name, "is %s, not %s" % (t.dtype, dtype))
        if t.get_device() != self.device:
            self.refuse(name, "is on %s, not on the current device cuda:%d" % (t.device, self.device))
        if t.shape != shape:
            self.refuse(name, "has shape %s, not %s" % (tuple(t.shape), shape))
        self.refuse(name, "is not contiguous")

    def view(self, t, name, shape, dtype):
        """(pointer, row stride) of a two-dimensional view with contiguous rows."""
        if t is None:
            return 0, 0
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self.device:
            self.explain(t, name, shape, dtype)
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        ld, one = t.stride()
        if one != 1 and shape[1] > 1:
            self.refuse(name, "has rows that are not contiguous")
        if ld < shape[1]:
            if shape[0] > 1:
                self.refuse(name, "has rows that overlap")
            ld = shape[1]
        return t.data_ptr(), ld

    def whole(self, t, name, shape, dtype):
        """Pointer of a contiguous tensor."""
        if t is None:
            return 0
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self.device or not t.is_contiguous():
            self.explain(t, name, shape, dtype)
        return t.data_ptr()

    def pool(self, t, name, n_slots, shape, dtype):
        """Pointer of a contiguous pool of n_slots slots or more."""
        if t is None:
            return 0
        if t.dim() == 0 or t.shape[0] < n_slots:
            self.refuse(name, "has fewer than the configuration's %d slots" % n_slots)
        return self.whole(t, name, (t.shape[0],) + shape, dtype)

    def bytes_of(self, t):
        if t is None:
            return None, 0
        if t.get_device() != self.device or not t.is_contiguous():
            self.refuse("workspace", "is not a contiguous tensor on the current device")
        return t.data_ptr(), t.nbytes

    def stream(self, stream):
        if stream is None:
            return _torch._C._cuda_getCurrentRawStream(self.device)
        return getattr(stream, "cuda_stream", stream)


def gdn_ssm_workspace_size(cfg, max_tokens, max_seqs) -> int:
    return load().gdn_ssm_workspace_size(ctypes.byref(cfg), max_tokens, max_seqs)


def gdn_ssm_conv_prefill(cfg, x, cu_seqlens, w, bias, conv_state, state_idx, out, stream=None):
    """x [T, CH] raw channels -> out [T, CH]; bias, conv_state and state_idx may be None."""
    a = _Args("gdn_ssm_conv_prefill", cfg.act)
    CH = cfg.heads * cfg.head_dim + 2 * cfg.groups * cfg.d_state
    T, n = x.shape[0], cu_seqlens.shape[0] - 1
    px, ld_x = a.view(x, "x", (T, CH), a.act)
    _check((_lib or load()).gdn_ssm_conv_prefill(
        ctypes.byref(cfg), px, ld_x, a.whole(cu_seqlens, "cu_seqlens", (n + 1,), a.i32), n, T,
        a.whole(w, "w", (CH, 4), a.act), a.whole(bias, "bias", (CH,), a.act),
        a.pool(conv_state, "conv_state", cfg.n_slots, (CH, 3), a.act),
        a.whole(state_idx, "state_idx", (n,), a.i32), a.whole(out, "out", (T, CH), a.act),
        a.stream(stream)), "gdn_ssm_conv_prefill")


def gdn_ssm_prefill(cfg, x, b, c, dt, A_log, cu_seqlens, y, D=None, dt_bias=None, z=None, state_in=None,
                    state_out=None, state_idx=None, workspace=None, stream=None):
    """x [T, heads*head_dim], b and c [T, groups*d_state] (one row stride), dt [T, heads] -> y."""
    a = _Args("gdn_ssm_prefill", cfg.act)
    H, N, P, T, n = cfg.heads, cfg.d_state, cfg.head_dim, x.shape[0], cu_seqlens.shape[0] - 1
    px, ld_x = a.view(x, "x", (T, H * P), a.act)
    pb, ld_bc = a.view(b, "b", (T, cfg.groups * N), a.act)
    pc, ld_c = a.view(c, "c", (T, cfg.groups * N), a.act)
    if T > 1 and ld_c != ld_bc:
        a.refuse("c", "has another row stride than b")
    pdt, ld_dt = a.view(dt, "dt", (T, H), a.act)
    pz, ld_z = a.view(z, "z", (T, H * P), a.act)
    io = _ssm_io(px, ld_x, pb, pc, ld_bc, pdt, ld_dt, pz, ld_z, a.whole(A_log, "A_log", (H,), a.f32),
               a.whole(dt_bias, "dt_bias", (H,), a.f32), a.whole(D, "D", (H,), a.f32), 0, 0,
               a.whole(cu_seqlens, "cu_seqlens", (n + 1,), a.i32), n, T,
               a.whole(state_idx, "state_idx", (n,), a.i32),
               a.pool(state_in, "state_in", cfg.n_slots, (H, N, P), a.f32),
               a.pool(state_out, "state_out", cfg.n_slots, (H, N, P), a.f32), 0,
               a.whole(y, "y", (T, H * P), a.act))
    ws, ws_bytes = a.bytes_of(workspace)
    _check((_lib or load()).gdn_ssm_prefill(ctypes.byref(cfg), ctypes.byref(io), ws, ws_bytes, a.stream(stream)),
           "gdn_ssm_prefill")


def gdn_ssm_decode(cfg, x, dt, conv_w, conv_state, A_log, state, y, workspace, conv_bias=None, D=None,
                   dt_bias=None, z=None, state_idx=None, stream=None):
    """One token per sequence: x [n, CH] raw channels, dt [n, heads] -> y [n, heads*head_dim];
    conv_state and state are updated in place."""
    a = _Args("gdn_ssm_decode", cfg.act)
    H, N, P, n = cfg.heads, cfg.d_state, cfg.head_dim, x.shape[0]
    CH = H * P + 2 * cfg.groups * N
    px, ld_x = a.view(x, "x", (n, CH), a.act)
    pdt, ld_dt = a.view(dt, "dt", (n, H), a.act)
    pz, ld_z = a.view(z, "z", (n, H * P), a.act)
    ps = a.pool(state, "state", cfg.n_slots, (H, N, P), a.f32)
    io = _ssm_io(px, ld_x, 0, 0, 0, pdt, ld_dt, pz, ld_z, a.whole(A_log, "A_log", (H,), a.f32),
               a.whole(dt_bias, "dt_bias", (H,), a.f32), a.whole(D, "D", (H,), a.f32),
               a.whole(conv_w, "conv_w", (CH, 4), a.act), a.whole(conv_bias, "conv_bias", (CH,), a.act),
               0, n, n, a.whole(state_idx, "state_idx", (n,), a.i32), ps, ps,
               a.pool(conv_state, "conv_state", cfg.n_slots, (CH, 3), a.act),
               a.whole(y, "y", (n, H * P), a.act))
    ws, ws_bytes = a.bytes_of(workspace)
    _check((_lib or load()).gdn_ssm_decode(ctypes.byref(cfg), ctypes.byref(io), ws, ws_bytes, a.stream(stream)),
           "gdn_ssm_decode")


def gdn_block_norm_workspace_size(rows, dim) -> int:
    return load().gdn_block_norm_workspace_size(rows, dim)


def gdn_block_norm(residual, w_pre=None, h=None, block=None, res_out=None, w_post=None, gate=None,
                   res_scale=1.0, eps=1e-6, weight_offset=0.0, rstd_post=None, rstd_pre=None, stream=None):
    """r' = residual + res_scale * sigmoid(gate) * norm(block) -> res_out, norm(r') -> h; all [rows, dim]
    (gate: [rows, dim] or [rows, 1]).  res_out may be residual."""
    a = _Args("gdn_block_norm")
    rows, dim = wide = tuple(residual.shape)
    like = h if h is not None else block
    if like is None:
        a.refuse("h", "and block are both missing: nothing to do")
    act, res = like.dtype, residual.dtype
    cols = 0 if gate is None else gate.shape[-1]
    io = _norm_io(rows, dim, _dt(like), _dt(residual), eps, weight_offset, res_scale,
                     *a.view(block, "block", wide, act), *a.view(gate, "gate", (rows, cols), act), cols,
                     *a.view(residual, "residual", wide, res), a.whole(w_post, "w_post", (dim,), a.f32),
                     a.whole(w_pre, "w_pre", (dim,), a.f32), *a.view(res_out, "res_out", wide, res),
                     *a.view(h, "h", wide, act), a.whole(rstd_post, "rstd_post", (rows,), a.f32),
                     a.whole(rstd_pre, "rstd_pre", (rows,), a.f32), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    _check((_lib or load()).gdn_block_norm(ctypes.byref(io), a.stream(stream)), "gdn_block_norm")


def gdn_block_norm_backward(res_out, rstd_pre=None, w_pre=None, dh=None, d_res_out=None, d_residual=None,
                            dw_pre=None, block=None, rstd_post=None, w_post=None, gate=None, res_scale=1.0,
                            weight_offset=0.0, d_block=None, d_gate=None, dw_post=None, workspace=None,
                            stream=None):
    """Gradients of gdn_block_norm for sum(dh * h) + sum(d_res_out * r'): res_out, rstd_pre and
    rstd_post as the forward call wrote them.  Every output may be None."""
    a = _Args("gdn_block_norm_backward")
    rows, dim = wide = tuple(res_out.shape)
    like = next((t for t in (dh, block) if t is not None), None)
    if like is None:
        a.refuse("dh", "and block are both missing: nothing to do")
    act, res = like.dtype, res_out.dtype
    cols = 0 if gate is None else gate.shape[-1]
    io = _norm_io(rows, dim, _dt(like), _dt(res_out), 0.0, weight_offset, res_scale,
                     *a.view(block, "block", wide, act), *a.view(gate, "gate", (rows, cols), act), cols,
                     *a.view(res_out, "res_out", wide, res), a.whole(w_post, "w_post", (dim,), a.f32),
                     a.whole(w_pre, "w_pre", (dim,), a.f32), 0, 0, 0, 0,
                     a.whole(rstd_post, "rstd_post", (rows,), a.f32),
                     a.whole(rstd_pre, "rstd_pre", (rows,), a.f32), *a.view(dh, "dh", wide, act),
                     *a.view(d_res_out, "d_res_out", wide, res),
                     *a.view(d_residual, "d_residual", wide, res),
                     *a.view(d_block, "d_block", wide, act), *a.view(d_gate, "d_gate", (rows, cols), act),
                     a.whole(dw_post, "dw_post", (dim,), a.f32), a.whole(dw_pre, "dw_pre", (dim,), a.f32))
    ws, ws_bytes = a.bytes_of(workspace)
    _check((_lib or load()).gdn_block_norm_backward(ctypes.byref(io), ws, ws_bytes, a.stream(stream)),
           "gdn_block_norm_backward")


# ------------------------------------------------- attention layers and their cache
#
# The checks of _Args as plain functions (a third of its time), and argument structures passed as packed bytes: a call's
# host time counts where a decode step is not captured.

def make_attn_config(q_heads, kv_heads, head_dim, page_size=64, act="bf16", n_pages=0, n_rows=0,
                     max_pages=0) -> AttnConfig:
    return AttnConfig(q_heads, kv_heads, head_dim, GDN_BF16 if act == "bf16" else GDN_FP32, page_size, n_pages,
                      n_rows, max_pages)


def _bytes_packer(cls):
    """The memory image of a structure from its fields' values in order, null pointers as 0."""
    code = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    return struct.Struct("@" + "".join(code[t] for _, t in cls._fields_) + "0P").pack


_prep_io, _decode_io = _bytes_packer(AttnPrepIO), _bytes_packer(AttnDecodeIO)
_get_device = _get_stream = _ACT = _F32 = _I32 = None


def _start():
    """What the functions below take from torch, at the first call."""
    global _get_device, _get_stream, _ACT, _F32, _I32
    _Args("")                                       # imports torch and initialises CUDA
    _get_stream, _ACT, _F32, _I32 = _torch._C._cuda_getCurrentRawStream, (_torch.bfloat16, _torch.float32), _torch.float32, _torch.int32
    load()
    _get_device = _torch._C._cuda_getDevice


def _whole(where, dev, t, name, shape, dtype):
    """Pointer of a contiguous tensor; 0 for none."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _Args(where).explain(t, name, shape, dtype)


def _heads(where, dev, t, name, shape, dtype):
    """(pointer, token stride, head stride) of a [tokens, heads, dim] view with contiguous heads."""
    if t is None:
        return 0, 0, 0
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _Args(where).explain(t, name, shape, dtype)
    T, H, D = shape
    ld, hs, one = t.stride()
    if one != 1 and not t.is_contiguous():
        _Args(where).refuse(name, "has heads that are not contiguous")
    return t.data_ptr(), ld if T > 1 else H * D, hs if H > 1 else D


def _pool(where, dev, t, name, n_pages, shape, dtype):
    """Pointer of a contiguous pool of n_pages pages or more."""
    if t is None:
        return 0
    have = t.shape
    if len(have) == 4 and have[0] >= n_pages and t.dtype is dtype and have[1:] == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    a = _Args(where)
    if not have or have[0] < n_pages:
        a.refuse(name, "has fewer than the configuration's %d pages" % n_pages)
    a.explain(t, name, (have[0],) + shape, dtype)


def _workspace(where, dev, t):
    if t is None:
        return 0, 0
    if t.get_device() != dev or not t.is_contiguous():
        _Args(where).bytes_of(t)
    return t.data_ptr(), t.nbytes


def _on(stream, dev):
    return _get_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)


def _prep_batch(where, dev, T, cu_seqlens, tokens):
    """(pointer of cu_seqlens, sequences): packed by bounds, or `tokens` to each sequence (None: one sequence)."""
    if cu_seqlens is not None:
        if tokens is not None:
            raise ValueError("%s: tokens and cu_seqlens are both given" % where)
        n = cu_seqlens.shape[0] - 1
        return _whole(where, dev, cu_seqlens, "cu_seqlens", (n + 1,), _I32), n
    if tokens is None:
        return 0, 1
    if tokens < 1 or T % tokens:
        raise ValueError("%s: q holds %d tokens, not a multiple of tokens=%s" % (where, T, tokens))
    return 0, T // tokens


def gdn_attn_prep(cfg, q, k, q_out, inv_freq, k_out=None, v=None, k_pages=None, v_pages=None, page_table=None, lens=None,
                  rows=None, cu_seqlens=None, tokens=None, positions=None, w_q=None, w_k=None, weight_offset=0.0, eps=1e-6,
                  interleaved=False, stream=None):
    """q [T, q_heads, head_dim], k and v [T, kv_heads, head_dim] (views) -> q_out [T, q_heads, head_dim], and k_out or the
    pools' places of the new tokens.  inv_freq: fp32 [rotary_dim / 2] or None.  The batch is packed by cu_seqlens, or has
    `tokens` tokens a sequence; lens counts them already.  k may be None."""
    if _get_device is None:
        _start()
    where, dev, act = "gdn_attn_prep", _get_device(), _ACT[cfg.act]
    T, Hk, D = q.shape[0], cfg.kv_heads, cfg.head_dim
    wide, narrow, page = (T, cfg.q_heads, D), (T, Hk, D), (Hk, cfg.page_size, D)
    cu, n = _prep_batch(where, dev, T, cu_seqlens, tokens)
    half = 0 if inv_freq is None else inv_freq.shape[0]
    io = _prep_io(*_heads(where, dev, q, "q", wide, act), *_heads(where, dev, k, "k", narrow, act), *_heads(where, dev, v, "v", narrow, act), T,
                  _whole(where, dev, w_q, "w_q", (D,), _F32), _whole(where, dev, w_k, "w_k", (D,), _F32), weight_offset, eps, 2 * half,
                  1 if interleaved else 0, _whole(where, dev, inv_freq, "inv_freq", (half,), _F32),
                  _whole(where, dev, positions, "positions", (T,), _I32), cu, n, _whole(where, dev, rows, "rows", (n,), _I32),
                  _whole(where, dev, lens, "lens", (cfg.n_rows,), _I32),
                  _whole(where, dev, page_table, "page_table", (cfg.n_rows, cfg.max_pages), _I32),
                  _pool(where, dev, k_pages, "k_pages", cfg.n_pages, page, act), _pool(where, dev, v_pages, "v_pages", cfg.n_pages, page, act),
                  _whole(where, dev, q_out, "q_out", wide, act), _whole(where, dev, k_out, "k_out", narrow, act),
                  0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    st = _lib.gdn_attn_prep(ctypes.byref(cfg), io, _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_attn_prep_workspace_size(cfg, max_tokens) -> int:
    return (_lib or load()).gdn_attn_prep_workspace_size(ctypes.byref(cfg), max_tokens)


def gdn_attn_prep_backward(cfg, q, k, dq_out, dk_out, inv_freq, dq=None, dk=None, dw_q=None, dw_k=None, w_q=None, w_k=None,
                           weight_offset=0.0, eps=1e-6, interleaved=False, cu_seqlens=None, tokens=None, positions=None,
                           workspace=None, stream=None):
    """Gradients of gdn_attn_prep (without a cache) for sum(dq_out * q_out) + sum(dk_out * k_out): dq and dk (views), dw_q and
    dw_k fp32 [head_dim], each of which may be None."""
    if _get_device is None:
        _start()
    where, dev, act = "gdn_attn_prep_backward", _get_device(), _ACT[cfg.act]
    T, D = q.shape[0], cfg.head_dim
    wide, narrow, width = (T, cfg.q_heads, D), (T, cfg.kv_heads, D), (D,)
    cu, n = _prep_batch(where, dev, T, cu_seqlens, tokens)
    half = 0 if inv_freq is None else inv_freq.shape[0]
    io = _prep_io(*_heads(where, dev, q, "q", wide, act), *_heads(where, dev, k, "k", narrow, act), 0, 0, 0, T,
                  _whole(where, dev, w_q, "w_q", width, _F32), _whole(where, dev, w_k, "w_k", width, _F32), weight_offset, eps, 2 * half,
                  1 if interleaved else 0, _whole(where, dev, inv_freq, "inv_freq", (half,), _F32),
                  _whole(where, dev, positions, "positions", (T,), _I32), cu, n, 0, 0, 0, 0, 0, 0, 0,
                  _whole(where, dev, dq_out, "dq_out", wide, act), _whole(where, dev, dk_out, "dk_out", narrow, act),
                  *_heads(where, dev, dq, "dq", wide, act), *_heads(where, dev, dk, "dk", narrow, act),
                  _whole(where, dev, dw_q, "dw_q", width, _F32), _whole(where, dev, dw_k, "dw_k", width, _F32))
    st = _lib.gdn_attn_prep_backward(ctypes.byref(cfg), io, *_workspace(where, dev, workspace), _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_attn_workspace_size(cfg, max_seqs, tokens=1) -> int:
    return (_lib or load()).gdn_attn_workspace_size(ctypes.byref(cfg), max_seqs, tokens)


def gdn_attn_decode(cfg, q, k_pages, v_pages, page_table, lens, out, workspace, tokens=1, rows=None, window=0, scale=None,
                    lse=None, stream=None):
    """Attention of the last `tokens` tokens of each sequence: q [n * tokens, q_heads, head_dim] (a view) -> out of that shape,
    lse fp32 [n * tokens, q_heads] or None.  scale None: head_dim ** -0.5."""
    if _get_device is None:
        _start()
    where, dev, act = "gdn_attn_decode", _get_device(), _ACT[cfg.act]
    T, Hq, D = q.shape[0], cfg.q_heads, cfg.head_dim
    n = T // tokens if tokens > 0 else 0
    if n * tokens != T:
        raise ValueError("%s: q holds %d tokens, not a multiple of tokens=%s" % (where, T, tokens))
    wide, page = (T, Hq, D), (cfg.kv_heads, cfg.page_size, D)
    io = _decode_io(*_heads(where, dev, q, "q", wide, act), _pool(where, dev, k_pages, "k_pages", cfg.n_pages, page, act),
                    _pool(where, dev, v_pages, "v_pages", cfg.n_pages, page, act),
                    _whole(where, dev, page_table, "page_table", (cfg.n_rows, cfg.max_pages), _I32),
                    _whole(where, dev, lens, "lens", (cfg.n_rows,), _I32), _whole(where, dev, rows, "rows", (n,), _I32), n, tokens, window,
                    D ** -0.5 if scale is None else scale, _whole(where, dev, out, "out", wide, act),
                    _whole(where, dev, lse, "lse", (T, Hq), _F32))
    st = _lib.gdn_attn_decode(ctypes.byref(cfg), io, *_workspace(where, dev, workspace), _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_page_workspace_size(cfg, max_lanes) -> int:
    return (_lib or load()).gdn_page_workspace_size(ctypes.byref(cfg), max_lanes)


def _page_state(where, dev, cfg, page_table, lens, refs):
    n_rows = cfg.n_rows
    return (_whole(where, dev, page_table, "page_table", (n_rows, cfg.max_pages), _I32), _whole(where, dev, lens, "lens", (n_rows,), _I32),
            _whole(where, dev, refs, "refs", (cfg.n_pages,), _I32))


def gdn_page_resize(cfg, page_table, lens, refs, rows, new_lens, granted, src_idx, dst_idx, workspace, stream=None):
    """Sets the lengths of `rows` to new_lens: pages taken, let go, or replaced by copies (src_idx -> dst_idx, to be carried out
    with gdn_page_copy before they are written and before the next resize or compaction).  granted: the lengths after the call."""
    if _get_device is None:
        _start()
    where, dev, i32, n = "gdn_page_resize", _get_device(), _I32, rows.shape[0]
    lane = (n,)
    st = _lib.gdn_page_resize(
        ctypes.byref(cfg), *_page_state(where, dev, cfg, page_table, lens, refs), _whole(where, dev, rows, "rows", lane, i32),
        _whole(where, dev, new_lens, "new_lens", lane, i32), n, _whole(where, dev, granted, "granted", lane, i32),
        _whole(where, dev, src_idx, "src_idx", lane, i32), _whole(where, dev, dst_idx, "dst_idx", lane, i32),
        *_workspace(where, dev, workspace), _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_page_fork(cfg, page_table, lens, refs, src_rows, dst_rows, stream=None):
    """Empty rows dst_rows become copies of src_rows that share their pages."""
    if _get_device is None:
        _start()
    where, dev, n = "gdn_page_fork", _get_device(), dst_rows.shape[0]
    st = _lib.gdn_page_fork(
        ctypes.byref(cfg), *_page_state(where, dev, cfg, page_table, lens, refs), _whole(where, dev, src_rows, "src_rows", (n,), _I32),
        _whole(where, dev, dst_rows, "dst_rows", (n,), _I32), n, _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_page_compact(cfg, page_table, lens, refs, table_out, refs_out, src_idx, dst_idx, workspace, stream=None):
    """Plans the moves of held pages to the lowest places (src_idx -> dst_idx, -1 behind the last) and writes the table and the
    counts after them; table_out may be page_table, refs_out refs."""
    if _get_device is None:
        _start()
    where, dev, n = "gdn_page_compact", _get_device(), src_idx.shape[0]
    st = _lib.gdn_page_compact(
        ctypes.byref(cfg), *_page_state(where, dev, cfg, page_table, lens, refs),
        _whole(where, dev, table_out, "table_out", (cfg.n_rows, cfg.max_pages), _I32),
        _whole(where, dev, refs_out, "refs_out", (cfg.n_pages,), _I32), _whole(where, dev, src_idx, "src_idx", (n,), _I32),
        _whole(where, dev, dst_idx, "dst_idx", (n,), _I32), n, *_workspace(where, dev, workspace), _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_page_copy(cfg, src_k, src_v, dst_k, dst_v, src_idx, dst_idx, stream=None):
    """Pages src_idx[i] of the src pools to pages dst_idx[i] of the dst pools (src < 0: zeros, dst < 0: nothing); the pools
    may be the same, and have as many pages as their first dimension says."""
    if _get_device is None:
        _start()
    where, dev, act, n = "gdn_page_copy", _get_device(), _ACT[cfg.act], dst_idx.shape[0]
    page = (cfg.kv_heads, cfg.page_size, cfg.head_dim)

    def pages(a, b):
        return min(a.shape[0], b.shape[0]) if a is not None and b is not None else 0 if a is b else (b if a is None else a).shape[0]
    st = _lib.gdn_page_copy(
        ctypes.byref(cfg), _pool(where, dev, src_k, "src_k", 0, page, act), _pool(where, dev, src_v, "src_v", 0, page, act), pages(src_k, src_v),
        _pool(where, dev, dst_k, "dst_k", 0, page, act), _pool(where, dev, dst_v, "dst_v", 0, page, act), pages(dst_k, dst_v),
        _whole(where, dev, src_idx, "src_idx", (n,), _I32), _whole(where, dev, dst_idx, "dst_idx", (n,), _I32), n, _on(stream, dev))
    if st:
        raise GDNError(st, where)


def gdn_device_error(stream=None) -> int:
    code = ctypes.c_uint32(0)
    st = load().gdn_device_error(_stream(stream), ctypes.byref(code))
    if st not in (0, 5):
        raise GDNError(st, "gdn_device_error")
    return code.value


def gdn_debug_set_wait(wait_ns=2_000_000_000, lose=0):
    """Limit of every bounded device wait (ns) and the test hook that drops one operand copy
    (bit 0: decode, bit 1: state chain, bit 2: state space scan, bit 3: decode attention);
    gdn_debug_set_wait() restores the defaults."""
    _check(load().gdn_debug_set_wait(wait_ns, lose), "gdn_debug_set_wait")


def gdn_status_string(status: int) -> str:
    return load().gdn_status_string(status).decode()
