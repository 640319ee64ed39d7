"""ctypes binding of the KDA C ABI (include/kda.h, libkda.so).

Argument marshalling only: every step of the operator runs in the library's
CUDA kernels.  torch is used for device memory (outputs, workspace) and for
the current CUDA stream.  There is no CPU path: if ``libkda.so`` is missing
the first call raises, and CPU tensors are rejected.

Low-level functions keep the C names (every symbol in ``EXPORTS``) and take
raw pointers and ints.  Tensor-level helpers allocate outputs and workspaces
with torch, check every tensor's shape and dtype against its role, and pass
the current stream: ``forward``, ``forward_g``, ``forward_scalar_gate``,
``forward_checkpoints``, ``forward_norm_gate``, ``forward_conv``,
``short_conv_swish``, ``decode_step``, ``decode_step_norm_gate``,
``short_conv_swish_backward``, ``gated_scan`` / ``gated_scan_g`` and their
``_backward``, ``gated_scan_step``, ``qk_norm_rope`` and its ``_backward``,
``cp_local`` / ``cp_finish`` / ``state_compose`` (context parallelism; the
collective lives in ``cp.py``), ``workspace`` and ``check_device_error``.

No helper builds an autograd graph: outputs do not require gradients, whatever
the inputs do.  Where a ``_backward`` helper exists, the caller calls it with the
gradient of the output (from a ``torch.autograd.Function`` of their own, if they
want torch to do so).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT = 0, -1, -2, -3, -4
KDA_F32, KDA_BF16 = 0, 1

# Every symbol include/kda.h declares.
EXPORTS = ("kda_status_string", "kda_version", "kda_forward_workspace_size",
           "kda_forward_launches", "kda_forward",
           "kda_forward_g", "kda_decode_step", "kda_forward_noalloc", "kda_forward_checkpoints",
           "kda_forward_norm_gate", "kda_decode_step_norm_gate", "kda_forward_scalar_gate",
           "kda_short_conv_swish", "kda_forward_conv_workspace_size", "kda_forward_conv",
           "kda_cp_workspace_size", "kda_cp_local", "kda_cp_finish", "kda_state_compose",
           "kda_check_device_error", "kda_debug_set_wait_limit", "kda_decode_step_conv",
           "kda_short_conv_swish_backward_workspace_size", "kda_short_conv_swish_backward",
           "kda_gated_scan_workspace_size", "kda_gated_scan", "kda_gated_scan_g",
           "kda_gated_scan_backward", "kda_gated_scan_g_backward", "kda_gated_scan_step",
           "kda_qk_norm_rope", "kda_qk_norm_rope_backward_workspace_size",
           "kda_qk_norm_rope_backward")

# Tokens between the states that the gated scan saves for its gradient.
KDA_SCAN_INTERVAL = 32

# Bytes of the library's fixed scratch array used by kda_forward_noalloc.
KDA_NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None


class KdaError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def lib():
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m gated_delta_rule_98_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    L.kda_status_string.argtypes = [ctypes.c_int]
    L.kda_status_string.restype = ctypes.c_char_p
    L.kda_version.argtypes = []
    L.kda_version.restype = i32
    L.kda_forward_workspace_size.argtypes = [i32] * 6 + [ctypes.c_int, i32]
    L.kda_forward_workspace_size.restype = sz
    L.kda_forward_launches.argtypes = [i32] * 6 + [ctypes.c_int, i32]
    L.kda_forward_launches.restype = i32
    L.kda_forward.argtypes = [vp] * 8 + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp, sz, vp]
    L.kda_forward.restype = ctypes.c_int
    L.kda_forward_g.argtypes = [vp] * 7 + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp, sz, vp]
    L.kda_forward_g.restype = ctypes.c_int
    L.kda_decode_step.argtypes = [vp] * 7 + [i32] * 4 + [ctypes.c_int, vp, vp]
    L.kda_decode_step.restype = ctypes.c_int
    L.kda_forward_noalloc.argtypes = [vp] * 8 + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp]
    L.kda_forward_noalloc.restype = ctypes.c_int
    L.kda_forward_checkpoints.argtypes = ([vp] * 8 + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp,
                                          i32, vp, sz, vp])
    L.kda_forward_checkpoints.restype = ctypes.c_int
    L.kda_forward_norm_gate.argtypes = ([vp] * 8 + [i32] * 6 + [ctypes.c_int, i32, vp, vp,
                                        ctypes.c_float, vp, vp, vp, sz, vp])
    L.kda_forward_norm_gate.restype = ctypes.c_int
    L.kda_decode_step_norm_gate.argtypes = ([vp] * 7 + [i32] * 4 + [ctypes.c_int, vp, vp,
                                            ctypes.c_float, vp, vp])
    L.kda_decode_step_norm_gate.restype = ctypes.c_int
    L.kda_forward_scalar_gate.argtypes = [vp] * 7 + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp,
                                                                sz, vp]
    L.kda_forward_scalar_gate.restype = ctypes.c_int
    L.kda_decode_step_conv.argtypes = ([vp] * 6 + [i32, vp] + [vp] * 4 + [i32] * 4 +
                                       [ctypes.c_int, vp, vp])
    L.kda_decode_step_conv.restype = ctypes.c_int
    L.kda_short_conv_swish.argtypes = [vp, vp, vp] + [i32] * 5 + [ctypes.c_int, vp, vp]
    L.kda_short_conv_swish.restype = ctypes.c_int
    L.kda_short_conv_swish_backward_workspace_size.argtypes = [i32] * 3
    L.kda_short_conv_swish_backward_workspace_size.restype = sz
    L.kda_short_conv_swish_backward.argtypes = ([vp] * 4 + [i32] * 5 +
                                                [ctypes.c_int, vp, vp, vp, sz, vp])
    L.kda_short_conv_swish_backward.restype = ctypes.c_int
    L.kda_gated_scan_workspace_size.argtypes = [i32] * 2
    L.kda_gated_scan_workspace_size.restype = sz
    L.kda_gated_scan.argtypes = [vp] * 5 + [i32] * 4 + [ctypes.c_int] + [vp] * 4 + [sz, vp]
    L.kda_gated_scan.restype = ctypes.c_int
    L.kda_gated_scan_g.argtypes = [vp] * 4 + [i32] * 4 + [ctypes.c_int] + [vp] * 4 + [sz, vp]
    L.kda_gated_scan_g.restype = ctypes.c_int
    L.kda_gated_scan_backward.argtypes = ([vp] * 6 + [i32] * 4 + [ctypes.c_int] + [vp] * 7 +
                                          [sz, vp])
    L.kda_gated_scan_backward.restype = ctypes.c_int
    L.kda_gated_scan_g_backward.argtypes = ([vp] * 5 + [i32] * 4 + [ctypes.c_int] + [vp] * 6 +
                                            [sz, vp])
    L.kda_gated_scan_g_backward.restype = ctypes.c_int
    L.kda_gated_scan_step.argtypes = [vp] * 4 + [i32] * 2 + [ctypes.c_int, vp, vp]
    L.kda_gated_scan_step.restype = ctypes.c_int
    i64, f32 = ctypes.c_int64, ctypes.c_float
    L.kda_qk_norm_rope.argtypes = ([vp, i64, vp, i64] + [vp] * 4 + [f32] + [i32] * 6 +
                                   [ctypes.c_int, vp, i64, vp, i64, vp])
    L.kda_qk_norm_rope.restype = ctypes.c_int
    L.kda_qk_norm_rope_backward_workspace_size.argtypes = [i32] * 2
    L.kda_qk_norm_rope_backward_workspace_size.restype = sz
    L.kda_qk_norm_rope_backward.argtypes = ([vp, i64] * 4 + [vp] * 4 + [f32] + [i32] * 6 +
                                            [ctypes.c_int, vp, i64, vp, i64] + [vp] * 3 +
                                            [sz, vp])
    L.kda_qk_norm_rope_backward.restype = ctypes.c_int
    L.kda_forward_conv_workspace_size.argtypes = [i32] * 6 + [ctypes.c_int, i32]
    L.kda_forward_conv_workspace_size.restype = sz
    L.kda_forward_conv.argtypes = ([vp] * 6 + [i32] + [vp] * 5 + [i32] * 6 +
                                   [ctypes.c_int, i32, vp, vp, vp, sz, vp])
    L.kda_forward_conv.restype = ctypes.c_int
    L.kda_cp_workspace_size.argtypes = [i32] * 6 + [ctypes.c_int, i32]
    L.kda_cp_workspace_size.restype = sz
    L.kda_cp_local.argtypes = [vp] * 7 + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp, sz, vp]
    L.kda_cp_local.restype = ctypes.c_int
    L.kda_cp_finish.argtypes = [vp, vp] + [i32] * 6 + [ctypes.c_int, i32, vp, vp, vp, sz, vp]
    L.kda_cp_finish.restype = ctypes.c_int
    L.kda_state_compose.argtypes = [vp] * 4 + [i32] * 3 + [vp]
    L.kda_state_compose.restype = ctypes.c_int
    L.kda_check_device_error.argtypes = [vp, vp]
    L.kda_check_device_error.restype = ctypes.c_int
    L.kda_debug_set_wait_limit.argtypes = [ctypes.c_int64]
    L.kda_debug_set_wait_limit.restype = ctypes.c_int
    _lib = L
    return L


def status_string(s):
    return lib().kda_status_string(int(s)).decode()


# ------------------------------------------------------------ raw C names ---

def kda_forward_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk):
    return lib().kda_forward_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt,
                                            chunk)


def kda_forward_launches(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk):
    return lib().kda_forward_launches(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk)


def kda_forward(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs, total_tokens, max_seqlen, H,
                dk, dv, dt, chunk, o, S_final, workspace, workspace_bytes, stream):
    return lib().kda_forward(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs, total_tokens,
                             max_seqlen, H, dk, dv, dt, chunk, o, S_final, workspace,
                             workspace_bytes, stream)


def kda_forward_g(q, k, v, g, beta, S0, cu_seqlens, num_seqs, total_tokens, max_seqlen, H,
                  dk, dv, dt, chunk, o, S_final, workspace, workspace_bytes, stream):
    return lib().kda_forward_g(q, k, v, g, beta, S0, cu_seqlens, num_seqs, total_tokens,
                               max_seqlen, H, dk, dv, dt, chunk, o, S_final, workspace,
                               workspace_bytes, stream)


def kda_decode_step(q, k, v, z, A, beta, S_inout, B, H, dk, dv, dt, o, stream):
    return lib().kda_decode_step(q, k, v, z, A, beta, S_inout, B, H, dk, dv, dt, o, stream)


def kda_forward_noalloc(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs, total_tokens,
                        max_seqlen, H, dk, dv, dt, chunk, o, S_final, stream):
    """kda_forward on the library's fixed scratch array (no workspace argument).
    For callers that cannot allocate device memory; see include/kda.h."""
    return lib().kda_forward_noalloc(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs,
                                     total_tokens, max_seqlen, H, dk, dv, dt, chunk, o, S_final,
                                     stream)


def kda_forward_checkpoints(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs, total_tokens,
                            max_seqlen, H, dk, dv, dt, chunk, o, S_final, S_ckpt, interval,
                            workspace, workspace_bytes, stream):
    return lib().kda_forward_checkpoints(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs,
                                         total_tokens, max_seqlen, H, dk, dv, dt, chunk, o,
                                         S_final, S_ckpt, interval, workspace, workspace_bytes,
                                         stream)


def kda_forward_norm_gate(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs, total_tokens,
                          max_seqlen, H, dk, dv, dt, chunk, out_gate, norm_weight, eps, o,
                          S_final, workspace, workspace_bytes, stream):
    return lib().kda_forward_norm_gate(q, k, v, z, A, beta, S0, cu_seqlens, num_seqs,
                                       total_tokens, max_seqlen, H, dk, dv, dt, chunk, out_gate,
                                       norm_weight, eps, o, S_final, workspace, workspace_bytes,
                                       stream)


def kda_decode_step_norm_gate(q, k, v, z, A, beta, S_inout, B, H, dk, dv, dt, out_gate,
                              norm_weight, eps, o, stream):
    return lib().kda_decode_step_norm_gate(q, k, v, z, A, beta, S_inout, B, H, dk, dv, dt,
                                           out_gate, norm_weight, eps, o, stream)


def kda_forward_scalar_gate(q, k, v, g_head, beta, S0, cu_seqlens, num_seqs, total_tokens,
                            max_seqlen, H, dk, dv, dt, chunk, o, S_final, workspace,
                            workspace_bytes, stream):
    return lib().kda_forward_scalar_gate(q, k, v, g_head, beta, S0, cu_seqlens, num_seqs,
                                         total_tokens, max_seqlen, H, dk, dv, dt, chunk, o,
                                         S_final, workspace, workspace_bytes, stream)


def kda_decode_step_conv(x_q, x_k, x_v, w_q, w_k, w_v, conv_width, conv_state, z, A, beta,
                         S_inout, B, H, dk, dv, dt, o, stream):
    return lib().kda_decode_step_conv(x_q, x_k, x_v, w_q, w_k, w_v, conv_width, conv_state, z,
                                      A, beta, S_inout, B, H, dk, dv, dt, o, stream)


def kda_short_conv_swish(x, w, cu_seqlens, num_seqs, total_tokens, max_seqlen, channels, width,
                         dt, y, stream):
    return lib().kda_short_conv_swish(x, w, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                                      channels, width, dt, y, stream)


def kda_short_conv_swish_backward_workspace_size(total_tokens, channels, width):
    return lib().kda_short_conv_swish_backward_workspace_size(total_tokens, channels, width)


def kda_short_conv_swish_backward(x, w, dy, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                                  channels, width, dt, dx, dw, workspace, workspace_bytes,
                                  stream):
    return lib().kda_short_conv_swish_backward(x, w, dy, cu_seqlens, num_seqs, total_tokens,
                                               max_seqlen, channels, width, dt, dx, dw,
                                               workspace, workspace_bytes, stream)


def kda_gated_scan_workspace_size(total_tokens, channels):
    return lib().kda_gated_scan_workspace_size(total_tokens, channels)


def kda_gated_scan(x, z, A, h0, cu_seqlens, num_seqs, total_tokens, max_seqlen, channels, dt, y,
                   h_final, states, workspace, workspace_bytes, stream):
    return lib().kda_gated_scan(x, z, A, h0, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                                channels, dt, y, h_final, states, workspace, workspace_bytes,
                                stream)


def kda_gated_scan_g(x, g, h0, cu_seqlens, num_seqs, total_tokens, max_seqlen, channels, dt, y,
                     h_final, states, workspace, workspace_bytes, stream):
    return lib().kda_gated_scan_g(x, g, h0, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                                  channels, dt, y, h_final, states, workspace, workspace_bytes,
                                  stream)


def kda_gated_scan_backward(x, z, A, states, h0, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                            channels, dt, dy, dh_final, dx, dz, dA, dh0, workspace,
                            workspace_bytes, stream):
    return lib().kda_gated_scan_backward(x, z, A, states, h0, cu_seqlens, num_seqs,
                                         total_tokens, max_seqlen, channels, dt, dy, dh_final,
                                         dx, dz, dA, dh0, workspace, workspace_bytes, stream)


def kda_gated_scan_g_backward(x, g, states, h0, cu_seqlens, num_seqs, total_tokens, max_seqlen,
                              channels, dt, dy, dh_final, dx, dg, dh0, workspace,
                              workspace_bytes, stream):
    return lib().kda_gated_scan_g_backward(x, g, states, h0, cu_seqlens, num_seqs, total_tokens,
                                           max_seqlen, channels, dt, dy, dh_final, dx, dg, dh0,
                                           workspace, workspace_bytes, stream)


def kda_gated_scan_step(x, z, A, h_inout, B, channels, dt, y, stream):
    return lib().kda_gated_scan_step(x, z, A, h_inout, B, channels, dt, y, stream)


def kda_qk_norm_rope(q, q_stride, k, k_stride, positions, freqs, q_weight, k_weight, eps,
                     total_tokens, Hq, Hk, d, rot, interleaved, dt, q_out, q_out_stride, k_out,
                     k_out_stride, stream):
    return lib().kda_qk_norm_rope(q, q_stride, k, k_stride, positions, freqs, q_weight, k_weight,
                                  eps, total_tokens, Hq, Hk, d, rot, interleaved, dt, q_out,
                                  q_out_stride, k_out, k_out_stride, stream)


def kda_qk_norm_rope_backward_workspace_size(total_tokens, d):
    return lib().kda_qk_norm_rope_backward_workspace_size(total_tokens, d)


def kda_qk_norm_rope_backward(q, q_stride, k, k_stride, dq_out, dq_out_stride, dk_out,
                              dk_out_stride, positions, freqs, q_weight, k_weight, eps,
                              total_tokens, Hq, Hk, d, rot, interleaved, dt, dq, dq_stride, dk,
                              dk_stride, dq_weight, dk_weight, workspace, workspace_bytes,
                              stream):
    return lib().kda_qk_norm_rope_backward(
        q, q_stride, k, k_stride, dq_out, dq_out_stride, dk_out, dk_out_stride, positions, freqs,
        q_weight, k_weight, eps, total_tokens, Hq, Hk, d, rot, interleaved, dt, dq, dq_stride,
        dk, dk_stride, dq_weight, dk_weight, workspace, workspace_bytes, stream)


def kda_forward_conv_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk):
    return lib().kda_forward_conv_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv,
                                                 dt, chunk)


def kda_forward_conv(x_q, x_k, x_v, w_q, w_k, w_v, conv_width, z, A, beta, S0, cu_seqlens,
                     num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk, o, S_final,
                     workspace, workspace_bytes, stream):
    return lib().kda_forward_conv(x_q, x_k, x_v, w_q, w_k, w_v, conv_width, z, A, beta, S0,
                                  cu_seqlens, num_seqs, total_tokens, max_seqlen, H, dk, dv, dt,
                                  chunk, o, S_final, workspace, workspace_bytes, stream)


def kda_cp_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk):
    return lib().kda_cp_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk)


def kda_cp_local(q, k, v, z, A, beta, cu_seqlens, num_seqs, total_tokens, max_seqlen, H, dk, dv,
                 dt, chunk, M_out, N_out, workspace, workspace_bytes, stream):
    return lib().kda_cp_local(q, k, v, z, A, beta, cu_seqlens, num_seqs, total_tokens,
                              max_seqlen, H, dk, dv, dt, chunk, M_out, N_out, workspace,
                              workspace_bytes, stream)


def kda_cp_finish(S_in, cu_seqlens, num_seqs, total_tokens, max_seqlen, H, dk, dv, dt, chunk, o,
                  S_final, workspace, workspace_bytes, stream):
    return lib().kda_cp_finish(S_in, cu_seqlens, num_seqs, total_tokens, max_seqlen, H, dk, dv,
                               dt, chunk, o, S_final, workspace, workspace_bytes, stream)


def kda_state_compose(M, N, S_in, S_out, count, dk, dv, stream):
    return lib().kda_state_compose(M, N, S_in, S_out, count, dk, dv, stream)


def kda_check_device_error(workspace, stream):
    return lib().kda_check_device_error(workspace, stream)


def kda_debug_set_wait_limit(cycles):
    return lib().kda_debug_set_wait_limit(cycles)


# ------------------------------------------------------- tensor helpers ---

def _dt(t):
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("KDA runs on the GPU only: pass CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("KDA tensors must be contiguous")


_F32_ROLES = ("A", "g", "g_head", "S0", "S_final", "S", "norm_weight", "S_ckpt")


def _shapes(T, H, dk, dv, N, dtype, **ts):
    """Raise ValueError unless every tensor given has the shape and dtype of its
    role (the C ABI takes raw pointers and cannot see either)."""
    want = {"q": (T, H, dk), "k": (T, H, dk), "z": (T, H, dk), "g": (T, H, dk),
            "v": (T, H, dv), "o": (T, H, dv), "out_gate": (T, H, dv), "beta": (T, H),
            "g_head": (T, H), "A": (H,), "S0": (N, H, dk, dv), "S_final": (N, H, dk, dv),
            "S": (N, H, dk, dv), "norm_weight": (dv,), "cu_seqlens": (N + 1,)}
    for name, t in ts.items():
        if t is None:
            continue
        if name in want and tuple(t.shape) != want[name]:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {want[name]}")
        if name == "S_ckpt" and (t.dim() != 5 or tuple(t.shape[:2]) != (N, H) or
                                 tuple(t.shape[3:]) != (dk, dv)):
            raise ValueError(f"S_ckpt: shape {tuple(t.shape)}, expected ({N}, {H}, J, {dk}, {dv})")
        need = (torch.float32 if name in _F32_ROLES else
                torch.int32 if name == "cu_seqlens" else dtype)
        if t.dtype != need:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {need}")


def _geometry(q, v, cu_seqlens, num_seqs, max_seqlen):
    T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is None:
        N = 1 if num_seqs is None else int(num_seqs)
        L = T // N if N else 0
        max_len = L if max_seqlen is None else int(max_seqlen)
    else:
        N = cu_seqlens.numel() - 1
        if max_seqlen is None:
            raise ValueError("max_seqlen is required with cu_seqlens")
        max_len = int(max_seqlen)
    return T, H, dk, dv, N, max_len


def workspace(num_seqs, total_tokens, max_seqlen, H, dk, dv, dtype, chunk, device=None):
    """A uint8 device tensor of kda_forward_workspace_size() bytes."""
    nbytes = kda_forward_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv,
                                        _dt(torch.empty(0, dtype=dtype)), chunk)
    if nbytes == 0:
        raise KdaError(KDA_ERR_UNSUPPORTED, "kda_forward_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


# the helpers below take a ``workspace`` argument that shadows the function
_new_workspace = workspace


def _forward(entry, q, k, v, gate_a, gate_b, beta, S0, cu_seqlens, num_seqs, max_seqlen, chunk,
             o, S_final, ws, stream, want_state):
    _check_cuda(q, k, v, gate_a, gate_b, beta, S0, cu_seqlens, o, S_final, ws)
    T, H, dk, dv, N, max_len = _geometry(q, v, cu_seqlens, num_seqs, max_seqlen)
    gate_roles = {"z": dict(z=gate_a, A=gate_b), "g": dict(g=gate_a),
                  "gs": dict(g_head=gate_a)}[entry]
    _shapes(T, H, dk, dv, N, q.dtype, q=q, k=k, v=v, beta=beta, S0=S0, cu_seqlens=cu_seqlens,
            o=o, S_final=S_final, **gate_roles)
    dt = _dt(q)
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    if S_final is None and want_state:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(N, T, max_len, H, dk, dv, q.dtype, chunk, device=q.device)
    args = [_p(q), _p(k), _p(v), _p(gate_a)]
    if entry == "z":
        args.append(_p(gate_b))
    args += [_p(beta), _p(S0), _p(cu_seqlens), N, T, max_len, H, dk, dv, dt, chunk, _p(o),
             _p(S_final), _p(ws), ws.numel(), _stream(stream)]
    fn = {"z": kda_forward, "g": kda_forward_g, "gs": kda_forward_scalar_gate}[entry]
    st = fn(*args)
    if st != KDA_OK:
        raise KdaError(st, fn.__name__)
    return o, S_final


def forward(q, k, v, z, A, beta, *, S0=None, cu_seqlens=None, num_seqs=None, max_seqlen=None,
            chunk=64, o=None, S_final=None, workspace=None, stream=None, output_final_state=True):
    """KDA prefill.  q,k,z [T,H,dk], v [T,H,dv], beta [T,H] (all one dtype),
    A [H] fp32, S0 [N,H,dk,dv] fp32 or None, cu_seqlens int32 [N+1] or None
    (then ``num_seqs`` equal sequences).  Returns (o, S_final)."""
    return _forward("z", q, k, v, z, A, beta, S0, cu_seqlens, num_seqs, max_seqlen, chunk, o,
                    S_final, workspace, stream, output_final_state)


def forward_checkpoints(q, k, v, z, A, beta, interval, *, S0=None, cu_seqlens=None,
                        num_seqs=None, max_seqlen=None, chunk=64, o=None, S_final=None,
                        S_ckpt=None, workspace=None, stream=None):
    """KDA prefill that also returns the state after every ``interval`` tokens of
    each sequence: (o, S_final, S_ckpt) with S_ckpt [N, H, max_seqlen // interval,
    dk, dv] fp32 (entries past a sequence's end are left as allocated: zeros
    when the binding allocates them)."""
    _check_cuda(q, k, v, z, A, beta, S0, cu_seqlens, o, S_final, S_ckpt, workspace)
    T, H, dk, dv, N, max_len = _geometry(q, v, cu_seqlens, num_seqs, max_seqlen)
    _shapes(T, H, dk, dv, N, q.dtype, q=q, k=k, v=v, z=z, A=A, beta=beta, S0=S0,
            cu_seqlens=cu_seqlens, o=o, S_final=S_final, S_ckpt=S_ckpt)
    if S_ckpt is not None and S_ckpt.shape[2] != max_len // int(interval):
        raise ValueError(f"S_ckpt: {S_ckpt.shape[2]} checkpoints, expected "
                         f"{max_len // int(interval)}")
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    if S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if S_ckpt is None:
        S_ckpt = torch.zeros((N, H, max_len // interval, dk, dv), dtype=torch.float32,
                             device=q.device)
    ws = workspace if workspace is not None else _new_workspace(N, T, max_len, H, dk, dv,
                                                                q.dtype, chunk, device=q.device)
    st = kda_forward_checkpoints(_p(q), _p(k), _p(v), _p(z), _p(A), _p(beta), _p(S0),
                                 _p(cu_seqlens), N, T, max_len, H, dk, dv, _dt(q), chunk, _p(o),
                                 _p(S_final), _p(S_ckpt), int(interval), _p(ws), ws.numel(),
                                 _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_forward_checkpoints")
    return o, S_final, S_ckpt


def forward_g(q, k, v, g, beta, *, S0=None, cu_seqlens=None, num_seqs=None, max_seqlen=None,
              chunk=64, o=None, S_final=None, workspace=None, stream=None,
              output_final_state=True):
    """KDA prefill with the fp32 log-decay g [T,H,dk] given directly (g in [-5, 0])."""
    return _forward("g", q, k, v, g, None, beta, S0, cu_seqlens, num_seqs, max_seqlen, chunk, o,
                    S_final, workspace, stream, output_final_state)


def forward_scalar_gate(q, k, v, g_head, beta, *, S0=None, cu_seqlens=None, num_seqs=None,
                        max_seqlen=None, chunk=64, o=None, S_final=None, workspace=None,
                        stream=None, output_final_state=True):
    """Gated DeltaNet special case: one fp32 log-decay per token and head,
    g_head [T,H] in [-5, 0], shared by the dk channels."""
    return _forward("gs", q, k, v, g_head, None, beta, S0, cu_seqlens, num_seqs, max_seqlen,
                    chunk, o, S_final, workspace, stream, output_final_state)


def decode_step(q, k, v, z, A, beta, S, *, o=None, stream=None):
    """One recurrent step: q,k,z [B,H,dk], v [B,H,dv], beta [B,H]; S [B,H,dk,dv]
    fp32 is updated in place.  Returns o [B,H,dv]."""
    _check_cuda(q, k, v, z, A, beta, S, o)
    B, H, dk = q.shape
    dv = v.shape[-1]
    _shapes(B, H, dk, dv, B, q.dtype, q=q, k=k, v=v, z=z, A=A, beta=beta, S=S, o=o)
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    st = kda_decode_step(_p(q), _p(k), _p(v), _p(z), _p(A), _p(beta), _p(S), B, H, dk, dv,
                         _dt(q), _p(o), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step")
    return o


def conv_state_zeros(B, H, dk, dv, width, dtype, device="cuda"):
    """The rolling input window of decode_step_conv before a sequence's first
    token: [B, H*(2*dk+dv), width-1] zeros."""
    return torch.zeros((B, H * (2 * dk + dv), width - 1), dtype=dtype, device=device)


def decode_step_conv(x_q, x_k, x_v, w_q, w_k, w_v, conv_state, z, A, beta, S, *, o=None,
                     stream=None):
    """One recurrent step with the input prologue carried across steps: x_q,
    x_k [B,H,dk], x_v [B,H,dv] are this token's convolution inputs, w_* [H*d,
    width] fp32 the taps, conv_state [B, H*(2dk+dv), width-1] (x's dtype) the
    rolling window, S [B,H,dk,dv] fp32; conv_state and S are updated in place.
    Returns o [B,H,dv]."""
    _check_cuda(x_q, x_k, x_v, w_q, w_k, w_v, conv_state, z, A, beta, S, o)
    B, H, dk = x_q.shape
    dv = x_v.shape[-1]
    _shapes(B, H, dk, dv, B, x_q.dtype, q=x_q, k=x_k, v=x_v, z=z, A=A, beta=beta, S=S, o=o)
    width = w_q.shape[-1]
    for name, w, rows in (("w_q", w_q, H * dk), ("w_k", w_k, H * dk), ("w_v", w_v, H * dv)):
        if tuple(w.shape) != (rows, width) or w.dtype != torch.float32:
            raise ValueError(f"{name}: {tuple(w.shape)} {w.dtype}, expected ({rows}, {width}) "
                             "float32")
    want = (B, H * (2 * dk + dv), width - 1)
    if conv_state is None or tuple(conv_state.shape) != want or conv_state.dtype != x_q.dtype \
            or not conv_state.is_contiguous():
        got = None if conv_state is None else (tuple(conv_state.shape), conv_state.dtype)
        raise ValueError(f"conv_state: {got}, expected contiguous {want} {x_q.dtype}")
    if o is None:
        o = torch.empty((B, H, dv), dtype=x_q.dtype, device=x_q.device)
    st = kda_decode_step_conv(_p(x_q), _p(x_k), _p(x_v), _p(w_q), _p(w_k), _p(w_v), width,
                              _p(conv_state), _p(z), _p(A), _p(beta), _p(S), B, H, dk, dv,
                              _dt(x_q), _p(o), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step_conv")
    return o


def forward_norm_gate(q, k, v, z, A, beta, out_gate, *, norm_weight=None, eps=1e-6, S0=None,
                      cu_seqlens=None, num_seqs=None, max_seqlen=None, chunk=64, o=None,
                      S_final=None, workspace=None, stream=None):
    """KDA prefill followed by the output epilogue: o = RMSNorm(attention output
    over dv) * norm_weight * sigmoid(out_gate), out_gate [T,H,dv] in q's dtype,
    norm_weight [dv] fp32 or None.  Returns (o, S_final)."""
    _check_cuda(q, k, v, z, A, beta, out_gate, norm_weight, S0, cu_seqlens, o, S_final,
                workspace)
    T, H, dk, dv, N, max_len = _geometry(q, v, cu_seqlens, num_seqs, max_seqlen)
    _shapes(T, H, dk, dv, N, q.dtype, q=q, k=k, v=v, z=z, A=A, beta=beta, out_gate=out_gate,
            norm_weight=norm_weight, S0=S0, cu_seqlens=cu_seqlens, o=o, S_final=S_final)
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    if S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = workspace if workspace is not None else _new_workspace(N, T, max_len, H, dk, dv,
                                                                q.dtype, chunk, device=q.device)
    st = kda_forward_norm_gate(_p(q), _p(k), _p(v), _p(z), _p(A), _p(beta), _p(S0),
                               _p(cu_seqlens), N, T, max_len, H, dk, dv, _dt(q), chunk,
                               _p(out_gate), _p(norm_weight), float(eps), _p(o), _p(S_final),
                               _p(ws), ws.numel(), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_forward_norm_gate")
    return o, S_final


def decode_step_norm_gate(q, k, v, z, A, beta, S, out_gate, *, norm_weight=None, eps=1e-6,
                          o=None, stream=None):
    """decode_step followed by the output epilogue (see forward_norm_gate);
    out_gate [B,H,dv].  S is updated in place.  Returns o [B,H,dv]."""
    _check_cuda(q, k, v, z, A, beta, S, out_gate, norm_weight, o)
    B, H, dk = q.shape
    dv = v.shape[-1]
    _shapes(B, H, dk, dv, B, q.dtype, q=q, k=k, v=v, z=z, A=A, beta=beta, S=S, o=o,
            out_gate=out_gate, norm_weight=norm_weight)
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    st = kda_decode_step_norm_gate(_p(q), _p(k), _p(v), _p(z), _p(A), _p(beta), _p(S), B, H, dk,
                                   dv, _dt(q), _p(out_gate), _p(norm_weight), float(eps), _p(o),
                                   _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step_norm_gate")
    return o


def short_conv_swish(x, w, *, cu_seqlens=None, num_seqs=None, max_seqlen=None, y=None,
                     stream=None):
    """Input prologue on one tensor x [T, ...] (trailing axes = channels):
    y = Swish(causal depthwise convolution with taps w [channels, width]).  No
    autograd graph is built: short_conv_swish_backward gives the gradients."""
    _check_cuda(x, w, cu_seqlens, y)
    T = x.shape[0]
    C = x.numel() // T if T else int(np.prod(x.shape[1:]))
    if cu_seqlens is None:
        N = 1 if num_seqs is None else int(num_seqs)
        L = T // N if N else 0
    else:
        N = cu_seqlens.numel() - 1
        if max_seqlen is None:
            raise ValueError("max_seqlen is required with cu_seqlens")
        L = int(max_seqlen)
    if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or
                                   cu_seqlens.numel() != N + 1):
        raise ValueError("cu_seqlens: int32 [N+1] expected")
    if w.dtype != torch.float32 or w.dim() != 2 or w.shape[0] != C:
        raise ValueError(f"w: {tuple(w.shape)} {w.dtype}, expected ({C}, width) float32")
    if y is not None and (y.shape != x.shape or y.dtype != x.dtype):
        raise ValueError("y: must match x in shape and dtype")
    if y is None:
        y = torch.empty_like(x)
    st = kda_short_conv_swish(_p(x), _p(w), _p(cu_seqlens), N, T, L, C, w.shape[-1], _dt(x),
                              _p(y), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_short_conv_swish")
    return y


def _packed(x, cu_seqlens, num_seqs, max_seqlen):
    """(tokens, channels, sequences, longest) of a packed [T, ...] tensor."""
    shape = x.shape
    T = shape[0]
    C = shape[1] if len(shape) == 2 else int(np.prod(shape[1:]))
    if cu_seqlens is None:
        N = 1 if num_seqs is None else int(num_seqs)
        return T, C, N, T // N if N else 0
    if max_seqlen is None:
        raise ValueError("max_seqlen is required with cu_seqlens")
    return T, C, cu_seqlens.numel() - 1, int(max_seqlen)


def _role(name, t, shape, dtype, device):
    """Raise ValueError unless t is on the GPU of index ``device``, contiguous, and
    of its role's shape and dtype.  Returns its address (None for None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected contiguous "
                     f"{tuple(shape)} {dtype} on the GPU of the first tensor")


def _first(name, t):
    """Address of the tensor that the others are held to."""
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The helpers below run on ``stream`` by making it current, so that the outputs and
# workspaces they allocate belong to it (a freed workspace could otherwise be handed
# out again while the kernels still use it).

def _on(stream, t):
    """``stream`` as the current one.  It has to be of t's GPU: the call runs on the
    current stream of that GPU, which one of another GPU would not change."""
    if stream.device != t.device:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def _call(fn, device, *args):
    """Run a C entry point on GPU ``device`` and its current stream, and raise
    unless it returns KDA_OK."""
    if device < 0:
        raise ValueError("KDA runs on the GPU only: pass CUDA tensors")
    if _raw_stream is not None:
        stream = _raw_stream(device)
    else:
        stream = torch.cuda.current_stream(device).cuda_stream
    if device == torch.cuda.current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != KDA_OK:
        raise KdaError(st, fn.__name__)


def _workspace_of(nbytes, ws, like, what):
    """(tensor, address, bytes) of a call's workspace; the caller keeps the tensor
    until it has enqueued its work."""
    if nbytes == 0:
        raise KdaError(KDA_ERR_UNSUPPORTED, what)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        return ws, ws.data_ptr(), nbytes
    if ws.dtype != torch.uint8 or ws.get_device() != like.get_device() or not ws.is_contiguous():
        raise ValueError(f"workspace: contiguous uint8 on {like.device} expected")
    return ws, ws.data_ptr(), ws.numel()


def short_conv_swish_backward(x, w, dy, *, cu_seqlens=None, num_seqs=None, max_seqlen=None,
                              dx=None, dw=None, workspace=None, stream=None):
    """Gradient of short_conv_swish: dy is the gradient of y (x's shape and
    dtype).  Returns (dx, dw), dw [channels, width] fp32.  Rows from
    cu_seqlens[N] on (a padded batch) are left as they were in dx."""
    if stream is not None:
        with _on(stream, x):
            return short_conv_swish_backward(x, w, dy, cu_seqlens=cu_seqlens, num_seqs=num_seqs,
                                             max_seqlen=max_seqlen, dx=dx, dw=dw,
                                             workspace=workspace)
    T, C, N, L = _packed(x, cu_seqlens, num_seqs, max_seqlen)
    width = w.shape[-1]
    dev, dt, f32, shape, taps = x.get_device(), x.dtype, torch.float32, x.shape, (C, width)
    xp, wp = _first("x", x), _role("w", w, taps, f32, dev)
    dyp = _role("dy", dy, shape, dt, dev)
    cup = _role("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    if dx is None:
        dx = torch.empty_like(x)
    else:
        _role("dx", dx, shape, dt, dev)
    if dw is None:
        dw = torch.empty_like(w)
    else:
        _role("dw", dw, taps, f32, dev)
    ws, wsp, nbytes = _workspace_of(
        lib().kda_short_conv_swish_backward_workspace_size(T, C, width), workspace, x,
        "kda_short_conv_swish_backward_workspace_size")
    _call(lib().kda_short_conv_swish_backward, dev, xp, wp, dyp, cup, N, T, L, C, width,
          _dt(x), dx.data_ptr(), dw.data_ptr(), wsp, nbytes)
    return dx, dw


def _gated_scan(x, z, A, g, h0, cu_seqlens, num_seqs, max_seqlen, y, h_final, states,
                save_states, ws, stream):
    if stream is not None:
        with _on(stream, x):
            return _gated_scan(x, z, A, g, h0, cu_seqlens, num_seqs, max_seqlen, y, h_final,
                               states, save_states, ws, None)
    T, C, N, L = _packed(x, cu_seqlens, num_seqs, max_seqlen)
    dev, dt, f32, shape, per_seq = x.get_device(), x.dtype, torch.float32, x.shape, (N, C)
    rows = ((T + KDA_SCAN_INTERVAL - 1) // KDA_SCAN_INTERVAL, C)
    xp, h0p = _first("x", x), _role("h0", h0, per_seq, f32, dev)
    cup = _role("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    if z is None:
        fn, gate = lib().kda_gated_scan_g, (_role("g", g, shape, f32, dev),)
    else:
        fn = lib().kda_gated_scan
        gate = (_role("z", z, shape, dt, dev), _role("A", A, (C,), f32, dev))
    like = A if g is None else g
    if y is None:
        y = torch.empty_like(x)
    else:
        _role("y", y, shape, dt, dev)
    if h_final is None:
        h_final = like.new_empty(N, C)
    else:
        _role("h_final", h_final, per_seq, f32, dev)
    if states is not None:
        _role("states", states, rows, f32, dev)
    elif save_states:
        states = like.new_empty(*rows)
    ws, wsp, nbytes = _workspace_of(lib().kda_gated_scan_workspace_size(T, C), ws, x,
                                    "kda_gated_scan_workspace_size")
    _call(fn, dev, xp, *gate, h0p, cup, N, T, L, C, _dt(x),
          y.data_ptr(),
          h_final.data_ptr(), None if states is None else states.data_ptr(), wsp, nbytes)
    return (y, h_final) if states is None else (y, h_final, states)


def gated_scan(x, z, A, *, h0=None, cu_seqlens=None, num_seqs=None, max_seqlen=None,
               save_states=False, y=None, h_final=None, states=None, workspace=None,
               stream=None):
    """Gated linear recurrence over packed sequences, one number of state per
    channel: a = exp(-5 sigmoid(e^A z)), h_t = a h_{t-1} + (1 - a) x_t.  x, z
    [T, ...] (trailing axes = channels) in one dtype, A [channels] fp32, h0
    [N, channels] fp32 or None.  Returns (y, h_final), and with ``save_states``
    also the states that gated_scan_backward needs,
    [ceil(T / KDA_SCAN_INTERVAL), channels] fp32.  Rows from cu_seqlens[N] on
    (a padded batch) are left as they were in y.  No autograd graph is built:
    gated_scan_backward gives the gradients."""
    return _gated_scan(x, z, A, None, h0, cu_seqlens, num_seqs, max_seqlen, y, h_final, states,
                       save_states, workspace, stream)


def gated_scan_g(x, g, *, h0=None, cu_seqlens=None, num_seqs=None, max_seqlen=None,
                 save_states=False, y=None, h_final=None, states=None, workspace=None,
                 stream=None):
    """gated_scan with the fp32 log-decay g (x's shape) given directly and the
    input unscaled: h_t = exp(g_t) h_{t-1} + x_t.  Gradients: gated_scan_g_backward."""
    return _gated_scan(x, None, None, g, h0, cu_seqlens, num_seqs, max_seqlen, y, h_final,
                       states, save_states, workspace, stream)


def _gated_scan_backward(x, z, A, g, states, dy, h0, dh_final, cu_seqlens, num_seqs, max_seqlen,
                         ws, stream):
    if stream is not None:
        with _on(stream, x):
            return _gated_scan_backward(x, z, A, g, states, dy, h0, dh_final, cu_seqlens,
                                        num_seqs, max_seqlen, ws, None)
    T, C, N, L = _packed(x, cu_seqlens, num_seqs, max_seqlen)
    dev, dt, f32, shape, per_seq = x.get_device(), x.dtype, torch.float32, x.shape, (N, C)
    rows = ((T + KDA_SCAN_INTERVAL - 1) // KDA_SCAN_INTERVAL, C)
    xp = _first("x", x)
    common = (_role("states", states, rows, f32, dev), _role("h0", h0, per_seq, f32, dev),
              _role("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev), N, T, L, C, _dt(x),
              _role("dy", dy, shape, dt, dev), _role("dh_final", dh_final, per_seq, f32, dev))
    if z is None:
        gp = _role("g", g, shape, f32, dev)
    else:
        zp, Ap = _role("z", z, shape, dt, dev), _role("A", A, (C,), f32, dev)
    dx, dh0 = torch.empty_like(x), states.new_empty(N, C)
    ws, wsp, nbytes = _workspace_of(lib().kda_gated_scan_workspace_size(T, C), ws, x,
                                    "kda_gated_scan_workspace_size")
    if z is None:
        dg = torch.empty_like(g)
        _call(lib().kda_gated_scan_g_backward, dev, xp, gp, *common, dx.data_ptr(),
              dg.data_ptr(), dh0.data_ptr(), wsp, nbytes)
        return dx, dg, dh0
    dz, dA = torch.empty_like(z), torch.empty_like(A)
    _call(lib().kda_gated_scan_backward, dev, xp, zp, Ap, *common, dx.data_ptr(),
          dz.data_ptr(), dA.data_ptr(), dh0.data_ptr(), wsp, nbytes)
    return dx, dz, dA, dh0


def gated_scan_backward(x, z, A, states, dy, *, h0=None, dh_final=None, cu_seqlens=None,
                        num_seqs=None, max_seqlen=None, workspace=None, stream=None):
    """Gradients of gated_scan: x, z, A, h0 and the packing as given to it,
    states as it returned them, dy the gradient of y, dh_final [N, channels]
    fp32 that of h_final (None: zeros).  Returns (dx, dz, dA, dh0)."""
    return _gated_scan_backward(x, z, A, None, states, dy, h0, dh_final, cu_seqlens, num_seqs,
                                max_seqlen, workspace, stream)


def gated_scan_g_backward(x, g, states, dy, *, h0=None, dh_final=None, cu_seqlens=None,
                          num_seqs=None, max_seqlen=None, workspace=None, stream=None):
    """Gradients of gated_scan_g (see gated_scan_backward): (dx, dg, dh0)."""
    return _gated_scan_backward(x, None, None, g, states, dy, h0, dh_final, cu_seqlens,
                                num_seqs, max_seqlen, workspace, stream)


def gated_scan_step(x, z, A, h, *, y=None, stream=None):
    """One step of gated_scan for B sequences: x, z [B, ...], A [channels] fp32;
    h [B, channels] fp32 is updated in place.  Returns y (x's shape and dtype)."""
    if stream is not None:
        with _on(stream, x):
            return gated_scan_step(x, z, A, h, y=y)
    B, C, _, _ = _packed(x, None, 1, None)
    dev, dt, f32, shape = x.get_device(), x.dtype, torch.float32, x.shape
    if y is None:
        y = torch.empty_like(x)
    else:
        _role("y", y, shape, dt, dev)
    _call(lib().kda_gated_scan_step, dev, _first("x", x),
          _role("z", z, shape, dt, dev), _role("A", A, (C,), f32, dev),
          _role("h", h, (B, C), f32, dev), B, C, _dt(x), y.data_ptr())
    return y


def _head_rows(name, t, shape, dtype, device):
    """(address, token stride) of a [T, heads, d] tensor whose heads lie side by side."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected "
                         f"{tuple(shape)} {dtype} on the GPU of the first tensor")
    T, H, d = shape
    st, sh, sd = t.stride()
    if T * H and (sd != 1 or (H > 1 and sh != d)):
        raise ValueError(f"{name}: heads must lie side by side (strides {t.stride()})")
    return t.data_ptr(), (st if T > 1 else H * d)


def _new_heads(t):
    """A contiguous tensor like t [T, heads, d], which may be a slice."""
    out = torch.empty_like(t)
    return out if out.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _qk(q, k, positions, freqs, q_weight, k_weight):
    """(T, d, rot) and the addresses of what both directions read besides q and k."""
    dev, f32 = q.get_device(), torch.float32
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}: [T, Hq, d] and [T, Hk, d] "
                         "expected")
    T, _, d = q.shape
    half = freqs.numel()
    return T, d, 2 * half, (_role("positions", positions, (T,), torch.int32, dev),
                            _role("freqs", freqs, (half,), torch.float64, dev),
                            _role("q_weight", q_weight, (d,), f32, dev),
                            _role("k_weight", k_weight, (d,), f32, dev))


def qk_norm_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm over d of every query head (q [T,Hq,d]) and key head (k
    [T,Hk,d]) with gains q_weight, k_weight [d] fp32 (None: ones), then the
    rotation by positions [T] int32 times freqs [rot/2] fp64 of the first rot
    channels, paired (i, i + rot/2), or (2i, 2i+1) when ``interleaved``.  q and
    k may be slices of one projection's output (heads side by side, any token
    stride); q_out = q, k_out = k works in place.  Returns (q_out, k_out).  No
    autograd graph is built: qk_norm_rope_backward gives the gradients, from q and
    k as they were before."""
    if stream is not None:
        with _on(stream, q):
            return qk_norm_rope(q, k, positions, freqs, q_weight=q_weight, k_weight=k_weight,
                                eps=eps, interleaved=interleaved, q_out=q_out, k_out=k_out)
    T, d, rot, read = _qk(q, k, positions, freqs, q_weight, k_weight)
    dev, dt, qs, ks = q.get_device(), q.dtype, q.shape, k.shape
    if q_out is None:
        q_out = _new_heads(q)
        qo = q_out.data_ptr(), qs[1] * d
    else:
        qo = _head_rows("q_out", q_out, qs, dt, dev)
    if k_out is None:
        k_out = _new_heads(k)
        ko = k_out.data_ptr(), ks[1] * d
    else:
        ko = _head_rows("k_out", k_out, ks, dt, dev)
    _call(lib().kda_qk_norm_rope, dev, *_head_rows("q", q, qs, dt, dev),
          *_head_rows("k", k, ks, dt, dev), *read, eps, T, qs[1], ks[1], d, rot,
          1 if interleaved else 0, _dt(q), *qo, *ko)
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, positions, freqs, *, q_weight=None,
                          k_weight=None, eps=1e-6, interleaved=False, dq=None, dk=None,
                          workspace=None, stream=None):
    """Gradients of qk_norm_rope: dq_out, dk_out are those of its outputs, the
    rest as given to it; dq = dq_out, dk = dk_out works in place.  Returns
    (dq, dk, dq_weight, dk_weight), the last two [d] fp32 or None where the
    gain is None."""
    if stream is not None:
        with _on(stream, q):
            return qk_norm_rope_backward(q, k, dq_out, dk_out, positions, freqs,
                                         q_weight=q_weight, k_weight=k_weight, eps=eps,
                                         interleaved=interleaved, dq=dq, dk=dk,
                                         workspace=workspace)
    T, d, rot, read = _qk(q, k, positions, freqs, q_weight, k_weight)
    dev, dt, qs, ks = q.get_device(), q.dtype, q.shape, k.shape
    if dq is None:
        dq = _new_heads(q)
        qo = dq.data_ptr(), qs[1] * d
    else:
        qo = _head_rows("dq", dq, qs, dt, dev)
    if dk is None:
        dk = _new_heads(k)
        ko = dk.data_ptr(), ks[1] * d
    else:
        ko = _head_rows("dk", dk, ks, dt, dev)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    ws, wsp, nbytes = _workspace_of(lib().kda_qk_norm_rope_backward_workspace_size(T, d),
                                    workspace, q, "kda_qk_norm_rope_backward_workspace_size")
    _call(lib().kda_qk_norm_rope_backward, dev, *_head_rows("q", q, qs, dt, dev),
          *_head_rows("k", k, ks, dt, dev), *_head_rows("dq_out", dq_out, qs, dt, dev),
          *_head_rows("dk_out", dk_out, ks, dt, dev), *read, eps, T, qs[1], ks[1], d, rot,
          1 if interleaved else 0, _dt(q), *qo, *ko, None if dqw is None else dqw.data_ptr(),
          None if dkw is None else dkw.data_ptr(), wsp, nbytes)
    return dq, dk, dqw, dkw


def forward_conv(x_q, x_k, x_v, w_q, w_k, w_v, z, A, beta, *, S0=None, cu_seqlens=None,
                 num_seqs=None, max_seqlen=None, chunk=64, o=None, S_final=None, workspace=None,
                 stream=None):
    """KDA prefill on the input prologue's outputs: q, k, v = Swish(short causal
    convolution of x_q, x_k, x_v) with taps w_* [H*d, width] fp32.  Returns
    (o, S_final)."""
    _check_cuda(x_q, x_k, x_v, w_q, w_k, w_v, z, A, beta, S0, cu_seqlens, o, S_final, workspace)
    T, H, dk, dv, N, max_len = _geometry(x_q, x_v, cu_seqlens, num_seqs, max_seqlen)
    _shapes(T, H, dk, dv, N, x_q.dtype, q=x_q, k=x_k, v=x_v, z=z, A=A, beta=beta, S0=S0,
            cu_seqlens=cu_seqlens, o=o, S_final=S_final)
    width = w_q.shape[-1]
    for name, w, rows in (("w_q", w_q, H * dk), ("w_k", w_k, H * dk), ("w_v", w_v, H * dv)):
        if tuple(w.shape) != (rows, width) or w.dtype != torch.float32:
            raise ValueError(f"{name}: {tuple(w.shape)} {w.dtype}, expected ({rows}, {width}) "
                             "float32")
    if o is None:
        o = torch.empty((T, H, dv), dtype=x_q.dtype, device=x_q.device)
    if S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=x_q.device)
    dt = _dt(x_q)
    if workspace is None:
        nbytes = kda_forward_conv_workspace_size(N, T, max_len, H, dk, dv, dt, chunk)
        if nbytes == 0:
            raise KdaError(KDA_ERR_UNSUPPORTED, "kda_forward_conv_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x_q.device)
    st = kda_forward_conv(_p(x_q), _p(x_k), _p(x_v), _p(w_q), _p(w_k), _p(w_v), w_q.shape[-1],
                          _p(z), _p(A), _p(beta), _p(S0), _p(cu_seqlens), N, T, max_len, H, dk,
                          dv, dt, chunk, _p(o), _p(S_final), _p(workspace), workspace.numel(),
                          _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_forward_conv")
    return o, S_final


class CpShard:
    """A shard's context-parallel state between cp_local and cp_finish: its
    geometry and the workspace that holds its chunk preparation."""

    def __init__(self, geometry, dtype, cu_seqlens, workspace, chunk):
        self.geometry, self.dtype, self.cu_seqlens = geometry, dtype, cu_seqlens
        self.workspace, self.chunk = workspace, chunk


def cp_local(q, k, v, z, A, beta, *, cu_seqlens=None, num_seqs=None, max_seqlen=None, chunk=64,
             workspace=None, stream=None):
    """Context parallelism, step 1 on this rank's shard: returns (M [N,H,dk,dk],
    N [N,H,dk,dv], shard) with S_after = M S_before + N for each sequence and
    head; ``shard`` carries the workspace to cp_finish."""
    _check_cuda(q, k, v, z, A, beta, cu_seqlens, workspace)
    T, H, dk, dv, N, max_len = _geometry(q, v, cu_seqlens, num_seqs, max_seqlen)
    _shapes(T, H, dk, dv, N, q.dtype, q=q, k=k, v=v, z=z, A=A, beta=beta, cu_seqlens=cu_seqlens)
    dt = _dt(q)
    if workspace is None:
        nbytes = kda_cp_workspace_size(N, T, max_len, H, dk, dv, dt, chunk)
        if nbytes == 0:
            raise KdaError(KDA_ERR_UNSUPPORTED, "kda_cp_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    M = torch.empty((N, H, dk, dk), dtype=torch.float32, device=q.device)
    Nt = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    st = kda_cp_local(_p(q), _p(k), _p(v), _p(z), _p(A), _p(beta), _p(cu_seqlens), N, T, max_len,
                      H, dk, dv, dt, chunk, _p(M), _p(Nt), _p(workspace), workspace.numel(),
                      _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_cp_local")
    return M, Nt, CpShard((T, H, dk, dv, N, max_len), q.dtype, cu_seqlens, workspace, chunk)


def cp_finish(shard, S_in=None, *, o=None, S_final=None, stream=None):
    """Context parallelism, step 4: o of the shard and the state after it, from
    the state entering it (None: zeros) and the workspace cp_local filled."""
    T, H, dk, dv, N, max_len = shard.geometry
    _check_cuda(S_in, o, S_final)
    _shapes(T, H, dk, dv, N, shard.dtype, S0=S_in, o=o, S_final=S_final)
    if o is None:
        o = torch.empty((T, H, dv), dtype=shard.dtype, device=shard.workspace.device)
    if S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=shard.workspace.device)
    st = kda_cp_finish(_p(S_in), _p(shard.cu_seqlens), N, T, max_len, H, dk, dv,
                       _dt(torch.empty(0, dtype=shard.dtype)), shard.chunk, _p(o), _p(S_final),
                       _p(shard.workspace), shard.workspace.numel(), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_cp_finish")
    return o, S_final


def state_compose(M, N, S_in=None, *, S_out=None, stream=None):
    """S_out = M S_in + N over leading batch axes (fp32; S_in None reads as 0)."""
    _check_cuda(M, N, S_in, S_out)
    dk, dv = N.shape[-2], N.shape[-1]
    count = N.numel() // (dk * dv)
    for name, t, shape in (("M", M, N.shape[:-2] + (dk, dk)), ("S_in", S_in, N.shape),
                           ("S_out", S_out, N.shape)):
        if t is not None and (tuple(t.shape) != tuple(shape) or t.dtype != torch.float32):
            raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype}, expected {tuple(shape)} float32")
    if N.dtype != torch.float32:
        raise ValueError("N: float32 expected")
    if S_out is None:
        S_out = torch.empty_like(N)
    st = kda_state_compose(_p(M), _p(N), _p(S_in), _p(S_out), count, dk, dv, _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_state_compose")
    return S_out


def check_device_error(ws, stream=None):
    """Status recorded on the device by the last forward call on ``ws``."""
    return kda_check_device_error(_p(ws), _stream(stream))
