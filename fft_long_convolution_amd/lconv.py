"""Python binding of liblconv.so (the gfx950 causal long-convolution library).

Argument marshalling only: every step of the computation runs in the HIP kernels behind the
C ABI declared in include/lconv.h.  torch provides device memory and the current stream.
There is no CPU fallback: if the library is missing, importing the entry points fails loudly.

Raw entry points keep the C names (``lconv_filter_fft``, ``lconv_fftconv_fwd``, ...), taking
integer device pointers.  ``filter_fft``, ``fftconv``, ``fftconv_partial``, ``fftconv_sparse``,
``fftconv_bwd``, ``fftconv_save``, ``filter_fft2d`` and ``fftconv2d`` are convenience wrappers over torch
tensors, and so are the mixer operators ``linear_attention``, ``linear_attention_bwd``,
``linear_attention_step``, ``rotary`` (with ``rotary_frequencies``), ``layer_norm``,
``layer_norm_bwd``, ``qk_norm_rotary``, ``qk_norm_rotary_bwd``, ``gated_scan``, ``gated_scan_bwd``,
``gated_scan_step``, ``short_conv``, ``short_conv_bwd`` and ``short_conv_step``, which also take strided views whose last
dimension is contiguous.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import re
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblconv.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "lconv.h")

F32, F16, BF16 = 0, 1, 2
STATUS = {0: "LCONV_SUCCESS", 1: "LCONV_ERR_NULL_POINTER", 2: "LCONV_ERR_INVALID_SHAPE",
          3: "LCONV_ERR_UNSUPPORTED", 4: "LCONV_ERR_MISALIGNED", 5: "LCONV_ERR_ALIASING",
          6: "LCONV_ERR_WORKSPACE", 7: "LCONV_ERR_HIP", 8: "LCONV_ERR_NOT_PREPARED",
          9: "LCONV_ERR_SCRATCH_LIMIT"}
NOALLOC_SCRATCH_BYTES = 64 << 20   # LCONV_NOALLOC_SCRATCH_BYTES


ROTARY_HALF, ROTARY_INTERLEAVED, ROTARY_INVERSE = 0, 1, 2


class Strides(ctypes.Structure):
    """lconv_strides_t: element strides of an operand [B][H][N][D]."""
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


class LconvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


_lib = None


def load(path: str = LIB_PATH):
    """Load liblconv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build the HIP library first "
                           "(python -m fft_long_convolution_amd.build)")
    lib = ctypes.CDLL(path)
    vp, i64, sz, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    f32, sp = ctypes.c_float, ctypes.POINTER(Strides)
    sig = {
        "lconv_filter_fft_bytes": (sz, [i64, i64, i]),
        "lconv_filter_fft_workspace_bytes": (sz, [i64, i64, i]),
        "lconv_fftconv_workspace_bytes": (sz, [i64, i64, i64, i]),
        "lconv_filter_fft2d_bytes": (sz, [i64, i64, i64, i]),
        "lconv_fftconv2d_workspace_bytes": (sz, [i64, i64, i64, i64, i]),
        "lconv_filter_fft": (i, [vp, vp, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv_fwd": (i, [vp, vp, vp, vp, vp, vp, i64, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv_bwd_workspace_bytes": (sz, [i64, i64, i64, i]),
        "lconv_fftconv_bwd": (i, [vp] * 11 + [i64, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv_fwd_save": (i, [vp] * 7 + [i64, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv_bwd_saved": (i, [vp] * 12 + [i64, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv_partial_fwd": (i, [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i, vp]),
        "lconv_fftconv_partial_bwd_workspace_bytes": (sz, [i64, i64, i64, i]),
        "lconv_fftconv_partial_bwd": (i, [vp] * 11 + [i64, i64, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv_sparse_fwd": (i, [vp, vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_uint32, i, vp]),
        "lconv_freq_blocks": (i, [i64]),
        "lconv_butterfly_blocks_count": (i64, [i64]),
        "lconv_butterfly_tables_bytes": (sz, [i64, i]),
        "lconv_butterfly_tables": (i, [vp, vp, i64, i, vp]),
        "lconv_butterfly_filter": (i, [vp, vp, vp, i64, i64, i, vp]),
        "lconv_butterfly_fwd": (i, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i, vp]),
        "lconv_filter_fft2d": (i, [vp, vp, i64, i64, i64, i, vp]),
        "lconv_fftconv2d_bwd_workspace_bytes": (sz, [i64, i64, i64, i64, i]),
        "lconv_fftconv2d_bwd": (i, [vp] * 7 + [i64, i64, i64, i64, i, vp, sz, vp]),
        "lconv_ssm_prep_bytes": (sz, [i64, i64, i64, i]),
        "lconv_ssm_prepare": (i, [vp, vp, vp, i64, i64, i64, i, vp]),
        "lconv_fftconv_ssm_workspace_bytes": (sz, [i64, i64, i64, i64, i64]),
        "lconv_fftconv_ssm_fwd": (i, [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i, vp, sz, vp]),
        "lconv_filter_fft3d_bytes": (sz, [i64, i64, i]),
        "lconv_filter_fft3d_workspace_bytes": (sz, [i64, i64, i]),
        "lconv_fftconv3d_workspace_bytes": (sz, [i64, i64, i64, i]),
        "lconv_filter_fft3d": (i, [vp, vp, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv3d_fwd": (i, [vp, vp, vp, vp, i64, i64, i64, i, vp, sz, vp]),
        "lconv_fftconv2d_fwd": (i, [vp, vp, vp, vp, i64, i64, i64, i64, i, vp, sz, vp]),
        "lconv_prepare": (i, [i64, i]),
        "lconv_fftconv_fwd_noalloc": (i, [vp, vp, vp, vp, vp, vp, i64, i64, i64, i, vp]),
        "lconv_linattn_workspace_bytes": (sz, [i64] * 6 + [i]),
        "lconv_linattn_fwd": (i, [vp, sp, vp, sp, vp, sp, vp, f32, vp, vp, vp, sp, vp] + [i64] * 6 + [i, vp, sz, vp]),
        "lconv_linattn_bwd_workspace_bytes": (sz, [i64] * 6 + [i]),
        "lconv_linattn_bwd": (i, [vp, sp, vp, sp, vp, sp, vp, sp, vp, f32, vp, vp, vp, vp, sp, vp, sp, vp, sp, vp, vp]
                              + [i64] * 6 + [i, vp, sz, vp]),
        "lconv_linattn_step": (i, [vp, sp, vp, sp, vp, sp, vp, f32, vp, vp, vp, sp] + [i64] * 6 + [i, vp]),
        "lconv_rotary": (i, [vp, sp, vp, sp, vp, i64, vp, f32, vp, sp, vp, sp] + [i64] * 6 + [i, i, vp]),
        "lconv_layernorm_fwd": (i, [vp, i64, vp, vp, vp, i64, vp, vp, i64, i64, f32, i, vp]),
        "lconv_layernorm_bwd_workspace_bytes": (sz, [i64, i64]),
        "lconv_layernorm_bwd": (i, [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, i64, i64, i, vp, sz, vp]),
        "lconv_gated_scan_marks_bytes": (sz, [i64] * 3),
        "lconv_gated_scan_workspace_bytes": (sz, [i64] * 3 + [i]),
        "lconv_gated_scan_fwd": (i, [vp, sp, vp, sp, vp, sp, vp, vp, vp, vp, sp, vp, vp] + [i64] * 3 + [i, i, vp, sz, vp]),
        "lconv_gated_scan_bwd_workspace_bytes": (sz, [i64] * 3 + [i, i]),
        "lconv_gated_scan_bwd": (i, [vp, sp, vp, sp, vp, sp, vp, sp, vp, vp, vp, vp, vp, sp, vp, sp, vp, sp, vp, vp]
                                 + [i64] * 3 + [i, i, vp, sz, vp]),
        "lconv_gated_scan_step": (i, [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64] + [i64] * 3 + [i, i, vp]),
        "lconv_qknorm_rotary_fwd": (i, [vp, sp, vp, sp, vp, vp, vp, i64, vp, f32, f32, vp, sp, vp, sp] + [i64] * 6 + [i, i, vp]),
        "lconv_qknorm_rotary_bwd_workspace_bytes": (sz, [i64] * 6),
        "lconv_qknorm_rotary_bwd": (i, [vp, sp, vp, sp, vp, sp, vp, sp, vp, vp, vp, i64, vp, f32, f32, vp, sp, vp, sp, vp, vp]
                                    + [i64] * 6 + [i, i, vp, sz, vp]),
        "lconv_shortconv_fwd": (i, [vp, sp, vp, vp, vp, vp, vp, sp, vp] + [i64] * 4 + [i, i, vp]),
        "lconv_shortconv_bwd_workspace_bytes": (sz, [i64] * 4),
        "lconv_shortconv_bwd": (i, [vp, sp, vp, sp, vp, vp, vp, vp, vp, vp, sp, vp, vp, vp] + [i64] * 4 + [i, i, vp, sz, vp]),
        "lconv_shortconv_step": (i, [vp, i64, vp, vp, vp, vp, vp, i64] + [i64] * 4 + [i, i, vp]),
        "lconv_status_string": (ctypes.c_char_p, [i]),
        "lconv_abi_version": (i, []),
        "lconv_release": (i, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name, None)
        if f is None:      # the version does not count entry points that were only added
            raise RuntimeError(f"{path} has no {name}: it was built from older sources, build it again "
                               "(python -m fft_long_convolution_amd.build)")
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def header_functions(path: str = HEADER):
    """Names of the functions declared in include/lconv.h."""
    src = open(path).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(lconv_[a-z0-9_]+)\s*\(", src)))


# ---- raw C entry points (same names as the ABI) -------------------------------------------

def lconv_filter_fft_bytes(H, N, dtype):
    return load().lconv_filter_fft_bytes(H, N, dtype)


def lconv_filter_fft_workspace_bytes(H, N, dtype):
    return load().lconv_filter_fft_workspace_bytes(H, N, dtype)


def lconv_fftconv_workspace_bytes(B, H, N, dtype):
    return load().lconv_fftconv_workspace_bytes(B, H, N, dtype)


def lconv_filter_fft2d_bytes(C, Hs, Ws, dtype):
    return load().lconv_filter_fft2d_bytes(C, Hs, Ws, dtype)


def lconv_fftconv2d_workspace_bytes(B, C, Hs, Ws, dtype):
    return load().lconv_fftconv2d_workspace_bytes(B, C, Hs, Ws, dtype)


def lconv_filter_fft(k, k_f, H, N, dtype, workspace, workspace_bytes, stream):
    return load().lconv_filter_fft(k, k_f, H, N, dtype, workspace, workspace_bytes, stream)


def lconv_fftconv_fwd(u, k_f, D, y, q, v, B, H, N, dtype, workspace, workspace_bytes, stream):
    return load().lconv_fftconv_fwd(u, k_f, D, y, q, v, B, H, N, dtype, workspace,
                                    workspace_bytes, stream)


def lconv_prepare(N, dtype):
    return load().lconv_prepare(N, dtype)


def lconv_fftconv_fwd_noalloc(u, k_f, D, y, q, v, B, H, N, dtype, stream):
    return load().lconv_fftconv_fwd_noalloc(u, k_f, D, y, q, v, B, H, N, dtype, stream)


def lconv_fftconv_bwd_workspace_bytes(B, H, N, dtype):
    return load().lconv_fftconv_bwd_workspace_bytes(B, H, N, dtype)


def lconv_fftconv_bwd(dy, u, k_f, D, q, v, du, dq, dv, dk, dD, B, H, N, dtype, workspace, workspace_bytes,
                      stream):
    return load().lconv_fftconv_bwd(dy, u, k_f, D, q, v, du, dq, dv, dk, dD, B, H, N, dtype, workspace,
                                    workspace_bytes, stream)


def lconv_fftconv_fwd_save(u, k_f, D, y, c, q, v, B, H, N, dtype, workspace, workspace_bytes, stream):
    return load().lconv_fftconv_fwd_save(u, k_f, D, y, c, q, v, B, H, N, dtype, workspace, workspace_bytes,
                                         stream)


def lconv_fftconv_bwd_saved(dy, u, k_f, D, q, v, c, du, dq, dv, dk, dD, B, H, N, dtype, workspace,
                            workspace_bytes, stream):
    return load().lconv_fftconv_bwd_saved(dy, u, k_f, D, q, v, c, du, dq, dv, dk, dD, B, H, N, dtype,
                                          workspace, workspace_bytes, stream)


def lconv_fftconv_partial_fwd(u, k_f, D, y, q, v, B, H, N, L, dtype, stream):
    return load().lconv_fftconv_partial_fwd(u, k_f, D, y, q, v, B, H, N, L, dtype, stream)


def lconv_fftconv_partial_bwd_workspace_bytes(B, H, N, dtype):
    return load().lconv_fftconv_partial_bwd_workspace_bytes(B, H, N, dtype)


def lconv_fftconv_partial_bwd(dy, u, k_f, D, q, v, du, dq, dv, dk, dD, B, H, N, L, dtype, workspace,
                              workspace_bytes, stream):
    return load().lconv_fftconv_partial_bwd(dy, u, k_f, D, q, v, du, dq, dv, dk, dD, B, H, N, L, dtype,
                                            workspace, workspace_bytes, stream)


def lconv_fftconv_sparse_fwd(u, k_f, D, y, q, v, B, H, N, keep, dtype, stream):
    return load().lconv_fftconv_sparse_fwd(u, k_f, D, y, q, v, B, H, N, keep, dtype, stream)


def lconv_butterfly_blocks_count(N):
    return load().lconv_butterfly_blocks_count(N)


def lconv_butterfly_tables_bytes(N, dtype):
    return load().lconv_butterfly_tables_bytes(N, dtype)


def lconv_butterfly_tables(blocks, tables, N, dtype, stream):
    return load().lconv_butterfly_tables(blocks, tables, N, dtype, stream)


def lconv_butterfly_filter(k, k_f, tables, H, N, dtype, stream):
    return load().lconv_butterfly_filter(k, k_f, tables, H, N, dtype, stream)


def lconv_butterfly_fwd(u, k_f, D, y, q, v, tables, B, H, N, dtype, stream):
    return load().lconv_butterfly_fwd(u, k_f, D, y, q, v, tables, B, H, N, dtype, stream)


def lconv_freq_blocks(N):
    return load().lconv_freq_blocks(N)


def lconv_filter_fft2d(k, k_f, C, Hs, Ws, dtype, stream):
    return load().lconv_filter_fft2d(k, k_f, C, Hs, Ws, dtype, stream)


def lconv_fftconv2d_fwd(u, k_f, D, y, B, C, Hs, Ws, dtype, workspace, workspace_bytes, stream):
    return load().lconv_fftconv2d_fwd(u, k_f, D, y, B, C, Hs, Ws, dtype, workspace, workspace_bytes, stream)


def lconv_fftconv2d_bwd_workspace_bytes(B, C, Hs, Ws, dtype):
    return load().lconv_fftconv2d_bwd_workspace_bytes(B, C, Hs, Ws, dtype)


def lconv_fftconv2d_bwd(dy, u, k_f, D, du, dk, dD, B, C, Hs, Ws, dtype, workspace, workspace_bytes, stream):
    return load().lconv_fftconv2d_bwd(dy, u, k_f, D, du, dk, dD, B, C, Hs, Ws, dtype, workspace,
                                      workspace_bytes, stream)


def lconv_ssm_prep_bytes(H, NS, T, dtype):
    return load().lconv_ssm_prep_bytes(H, NS, T, dtype)


def lconv_ssm_prepare(lam, W, prep, H, NS, T, dtype, stream):
    return load().lconv_ssm_prepare(lam, W, prep, H, NS, T, dtype, stream)


def lconv_fftconv_ssm_workspace_bytes(B, H, N, NS, T):
    return load().lconv_fftconv_ssm_workspace_bytes(B, H, N, NS, T)


def lconv_fftconv_ssm_fwd(u, prep, D, y, q, v, B, H, N, NS, T, dtype, workspace, workspace_bytes, stream):
    return load().lconv_fftconv_ssm_fwd(u, prep, D, y, q, v, B, H, N, NS, T, dtype, workspace,
                                        workspace_bytes, stream)


def lconv_filter_fft3d_bytes(C, S, dtype):
    return load().lconv_filter_fft3d_bytes(C, S, dtype)


def lconv_filter_fft3d_workspace_bytes(C, S, dtype):
    return load().lconv_filter_fft3d_workspace_bytes(C, S, dtype)


def lconv_fftconv3d_workspace_bytes(B, C, S, dtype):
    return load().lconv_fftconv3d_workspace_bytes(B, C, S, dtype)


def lconv_filter_fft3d(k, k_f, C, S, dtype, workspace, workspace_bytes, stream):
    return load().lconv_filter_fft3d(k, k_f, C, S, dtype, workspace, workspace_bytes, stream)


def lconv_fftconv3d_fwd(u, k_f, D, y, B, C, S, dtype, workspace, workspace_bytes, stream):
    return load().lconv_fftconv3d_fwd(u, k_f, D, y, B, C, S, dtype, workspace, workspace_bytes, stream)


def lconv_linattn_workspace_bytes(B, H, G, N, Dk, Dv, dtype):
    return load().lconv_linattn_workspace_bytes(B, H, G, N, Dk, Dv, dtype)


def lconv_linattn_fwd(q, qs, k, ks, v, vs, log_decay, scale, state_in, lengths, y, ys, state_out, B, H, G, N, Dk, Dv,
                      dtype, workspace, workspace_bytes, stream):
    return load().lconv_linattn_fwd(q, qs, k, ks, v, vs, log_decay, scale, state_in, lengths, y, ys, state_out, B, H,
                                    G, N, Dk, Dv, dtype, workspace, workspace_bytes, stream)


def lconv_linattn_bwd_workspace_bytes(B, H, G, N, Dk, Dv, dtype):
    return load().lconv_linattn_bwd_workspace_bytes(B, H, G, N, Dk, Dv, dtype)


def lconv_linattn_bwd(dy, dys, q, qs, k, ks, v, vs, log_decay, scale, state_in, dstate_out, lengths, dq, dqs, dk, dks,
                      dv, dvs, dstate_in, dlog_decay, B, H, G, N, Dk, Dv, dtype, workspace, workspace_bytes, stream):
    return load().lconv_linattn_bwd(dy, dys, q, qs, k, ks, v, vs, log_decay, scale, state_in, dstate_out, lengths, dq,
                                    dqs, dk, dks, dv, dvs, dstate_in, dlog_decay, B, H, G, N, Dk, Dv, dtype, workspace,
                                    workspace_bytes, stream)


def lconv_linattn_step(q, qs, k, ks, v, vs, log_decay, scale, state, slots, y, ys, B, H, G, Dk, Dv, nslots, dtype,
                       stream):
    return load().lconv_linattn_step(q, qs, k, ks, v, vs, log_decay, scale, state, slots, y, ys, B, H, G, Dk, Dv,
                                     nslots, dtype, stream)


def lconv_rotary(q, qs, k, ks, positions, pos_stride, inv_freq, magnitude, yq, yqs, yk, yks, B, H, G, N, D, rot, flags,
                 dtype, stream):
    return load().lconv_rotary(q, qs, k, ks, positions, pos_stride, inv_freq, magnitude, yq, yqs, yk, yks, B, H, G, N,
                               D, rot, flags, dtype, stream)


def lconv_layernorm_fwd(x, x_stride, weight, bias, y, y_stride, mean, rstd, rows, C, eps, dtype, stream):
    return load().lconv_layernorm_fwd(x, x_stride, weight, bias, y, y_stride, mean, rstd, rows, C, eps, dtype, stream)


def lconv_layernorm_bwd_workspace_bytes(rows, C):
    return load().lconv_layernorm_bwd_workspace_bytes(rows, C)


def lconv_layernorm_bwd(dy, dy_stride, x, x_stride, weight, mean, rstd, dx, dx_stride, dweight, dbias, rows, C, dtype,
                        workspace, workspace_bytes, stream):
    return load().lconv_layernorm_bwd(dy, dy_stride, x, x_stride, weight, mean, rstd, dx, dx_stride, dweight, dbias,
                                      rows, C, dtype, workspace, workspace_bytes, stream)


def lconv_gated_scan_marks_bytes(B, N, C):
    return load().lconv_gated_scan_marks_bytes(B, N, C)


def lconv_gated_scan_workspace_bytes(B, N, C, dtype):
    return load().lconv_gated_scan_workspace_bytes(B, N, C, dtype)


def lconv_gated_scan_fwd(x, xs, z, zs, input_gate, igs, rate, state_in, lengths, y, ys, state_out, marks, B, N, C, flags,
                         dtype, workspace, workspace_bytes, stream):
    return load().lconv_gated_scan_fwd(x, xs, z, zs, input_gate, igs, rate, state_in, lengths, y, ys, state_out, marks, B,
                                       N, C, flags, dtype, workspace, workspace_bytes, stream)


def lconv_gated_scan_bwd_workspace_bytes(B, N, C, flags, dtype):
    return load().lconv_gated_scan_bwd_workspace_bytes(B, N, C, flags, dtype)


def lconv_gated_scan_bwd(dy, dys, x, xs, z, zs, input_gate, igs, rate, marks, dstate_out, lengths, dx, dxs, dz, dzs,
                         dinput_gate, digs, drate, dstate_in, B, N, C, flags, dtype, workspace, workspace_bytes, stream):
    return load().lconv_gated_scan_bwd(dy, dys, x, xs, z, zs, input_gate, igs, rate, marks, dstate_out, lengths, dx, dxs,
                                       dz, dzs, dinput_gate, digs, drate, dstate_in, B, N, C, flags, dtype, workspace,
                                       workspace_bytes, stream)


def lconv_gated_scan_step(x, xs, z, zs, input_gate, igs, rate, state, slots, y, ys, B, C, nslots, flags, dtype, stream):
    return load().lconv_gated_scan_step(x, xs, z, zs, input_gate, igs, rate, state, slots, y, ys, B, C, nslots, flags,
                                        dtype, stream)


def lconv_qknorm_rotary_fwd(q, qs, k, ks, q_weight, k_weight, positions, pos_stride, inv_freq, magnitude, eps, yq, yqs, yk, yks,
                            B, H, G, N, D, rot, flags, dtype, stream):
    return load().lconv_qknorm_rotary_fwd(q, qs, k, ks, q_weight, k_weight, positions, pos_stride, inv_freq, magnitude, eps,
                                          yq, yqs, yk, yks, B, H, G, N, D, rot, flags, dtype, stream)


def lconv_qknorm_rotary_bwd_workspace_bytes(B, H, G, N, D, rot):
    return load().lconv_qknorm_rotary_bwd_workspace_bytes(B, H, G, N, D, rot)


def lconv_qknorm_rotary_bwd(dyq, dyqs, dyk, dyks, q, qs, k, ks, q_weight, k_weight, positions, pos_stride, inv_freq, magnitude,
                            eps, dq, dqs, dk, dks, dq_weight, dk_weight, B, H, G, N, D, rot, flags, dtype, workspace,
                            workspace_bytes, stream):
    return load().lconv_qknorm_rotary_bwd(dyq, dyqs, dyk, dyks, q, qs, k, ks, q_weight, k_weight, positions, pos_stride,
                                          inv_freq, magnitude, eps, dq, dqs, dk, dks, dq_weight, dk_weight, B, H, G, N, D, rot,
                                          flags, dtype, workspace, workspace_bytes, stream)


def lconv_shortconv_fwd(x, xs, weight, bias, state_in, lengths, y, ys, state_out, B, N, C, K, flags, dtype, stream):
    return load().lconv_shortconv_fwd(x, xs, weight, bias, state_in, lengths, y, ys, state_out, B, N, C, K, flags, dtype, stream)


def lconv_shortconv_bwd_workspace_bytes(B, N, C, K):
    return load().lconv_shortconv_bwd_workspace_bytes(B, N, C, K)


def lconv_shortconv_bwd(dy, dys, x, xs, weight, bias, state_in, dstate_out, lengths, dx, dxs, dweight, dbias, dstate_in, B, N, C,
                        K, flags, dtype, workspace, workspace_bytes, stream):
    return load().lconv_shortconv_bwd(dy, dys, x, xs, weight, bias, state_in, dstate_out, lengths, dx, dxs, dweight, dbias,
                                      dstate_in, B, N, C, K, flags, dtype, workspace, workspace_bytes, stream)


def lconv_shortconv_step(x, xs, weight, bias, state, slots, y, ys, B, C, K, nslots, flags, dtype, stream):
    return load().lconv_shortconv_step(x, xs, weight, bias, state, slots, y, ys, B, C, K, nslots, flags, dtype, stream)


def lconv_abi_version():
    return load().lconv_abi_version()


def lconv_release():
    return load().lconv_release()


def lconv_status_string(status):
    return load().lconv_status_string(status)


def status_string(status: int) -> str:
    return lconv_status_string(status).decode()


# ---- torch wrappers ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _torch():
    """torch, imported when a tensor first comes (and kept: an import statement takes a quarter of a microsecond each time, of
    which a call for single tokens would meet a dozen)."""
    import torch
    return torch


def dtype_code(t) -> int:
    torch = _torch()
    return {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}[t]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(status, where):
    if status != 0:
        raise LconvError(status, where)


def _need(name, t, shape, dtype, optional=False):
    """Host-side checks the C ABI cannot make on a torch tensor: the dtype, the shape and a dense
    layout (the kernels read memory as contiguous rows, so a transposed or strided view would be
    read wrongly, not rejected).  The device is checked by _on_gpu once every operand passed."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (a strided or transposed view would be read as dense rows)")


def _need_buf(name, t, nbytes):
    """An opaque library buffer (filter spectrum, state-space tables): a contiguous 1-D uint8
    tensor of exactly the size the library's size query gives for this shape and dtype (a buffer
    made for another shape or dtype would be read out of bounds)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 1:
        raise ValueError(f"{name} must be the 1-D uint8 tensor the library wrote")
    if t.numel() not in (nbytes, max(nbytes, 1)):
        raise ValueError(f"{name} holds {t.numel()} bytes; this shape and dtype need {nbytes} "
                         "(it was made for another shape or dtype)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(**operands):
    """Every given operand is a GPU tensor, all on the same device; returns that device."""
    dev = None
    for name, t in operands.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a GPU tensor, got device {t.device}")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")
        dev = t.device
    return dev


def _act(u, name="u", dims=3):
    """(torch dtype, shape) of the activation that fixes the call's shape."""
    torch = _torch()
    if not isinstance(u, torch.Tensor) or u.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-D torch tensor")
    if u.dtype not in (torch.float32, torch.float16, torch.bfloat16):
        raise ValueError(f"{name} has dtype {u.dtype}; supported: float32, float16, bfloat16")
    _need(name, u, u.shape, u.dtype)
    return u.dtype, tuple(u.shape)


def filter_fft(k, stream=None):
    """Opaque filter spectrum (uint8 device tensor) for k [H, N]."""
    torch = _torch()
    _act(k, "k", dims=2)
    _on_gpu(k=k)
    H, N = k.shape
    dt = dtype_code(k.dtype)
    nbytes = lconv_filter_fft_bytes(H, N, dt)
    if nbytes == 0 and H * N > 0:
        raise LconvError(3, "lconv_filter_fft_bytes")
    k_f = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=k.device)
    wsb = lconv_filter_fft_workspace_bytes(H, N, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=k.device) if wsb else None
    _check(lconv_filter_fft(_ptr(k), k_f.data_ptr(), H, N, dt, _ptr(ws), wsb, _stream(stream)),
           "lconv_filter_fft")
    return k_f


def _gated_inputs(u, k_f, D, q, v, out, L=None, **more):
    """Checks of the 1D calls' operands; the spectrum was made for [H, L] (L = N if None).
    `more`: further [B, H, N] operands of u's dtype (None: absent)."""
    tdt, (B, H, N) = _act(u)
    _need("D", D, (H,), tdt)
    _need("q", q, (B, H, N), tdt, optional=True)
    _need("v", v, (B, H, N), tdt, optional=True)
    _need("out", out, (B, H, N), tdt, optional=True)
    for name, t in more.items():
        _need(name, t, (B, H, N), tdt, optional=True)
    _need_buf("k_f", k_f, lconv_filter_fft_bytes(H, N if L is None else L, dtype_code(tdt)))
    _on_gpu(u=u, k_f=k_f, D=D, q=q, v=v, out=out, **more)
    return B, H, N


def fftconv(u, k_f, D, q=None, v=None, out=None, stream=None):
    """y = v * ((k * (q*u))[:N] + D * (q*u)) for u [B, H, N]."""
    torch = _torch()
    B, H, N = _gated_inputs(u, k_f, D, q, v, out)
    dt = dtype_code(u.dtype)
    y = torch.empty_like(u) if out is None else out
    wsb = lconv_fftconv_workspace_bytes(B, H, N, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=u.device) if wsb else None
    _check(lconv_fftconv_fwd(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), _ptr(q), _ptr(v), B, H, N, dt,
                             _ptr(ws), wsb, _stream(stream)), "lconv_fftconv_fwd")
    return y


def fftconv_save(u, k_f, D, q=None, v=None, stream=None):
    """(y, c): y = v * c with the pre-gate output c = (k * (q*u))[:N] + D * (q*u), for the
    gradient call."""
    torch = _torch()
    B, H, N = _gated_inputs(u, k_f, D, q, v, None)
    dt = dtype_code(u.dtype)
    y = torch.empty_like(u)
    c = torch.empty_like(u)
    wsb = lconv_fftconv_workspace_bytes(B, H, N, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=u.device) if wsb else None
    _check(lconv_fftconv_fwd_save(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), _ptr(c), _ptr(q), _ptr(v),
                                  B, H, N, dt, _ptr(ws), wsb, _stream(stream)), "lconv_fftconv_fwd_save")
    return y, c


def fftconv_bwd(dy, u, k_f, D, q=None, v=None, need_dk=True, c=None, stream=None):
    """Gradients of y = v * ((k * (q*u))[:N] + D * (q*u)) given dy [B, H, N].

    With c (the pre-gate output from fftconv_save), dv = dy * c without a transform.
    Returns (du, dq, dv, dk, dD): du, dq, dv in u's dtype (dq is None without q, dv is None
    without v); dk [H, N] and dD [H] in float32 (None when need_dk is False)."""
    torch = _torch()
    if dy is None:
        raise ValueError("dy is required")
    B, H, N = _gated_inputs(u, k_f, D, q, v, None, dy=dy, c=c)
    dt = dtype_code(u.dtype)
    du = torch.empty_like(u)
    dq = torch.empty_like(u) if q is not None else None
    dv = torch.empty_like(u) if v is not None else None
    dk = torch.empty((H, N), dtype=torch.float32, device=u.device) if need_dk else None
    dD = torch.empty((H,), dtype=torch.float32, device=u.device) if need_dk else None
    wsb = lconv_fftconv_bwd_workspace_bytes(B, H, N, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=u.device) if wsb else None
    if c is None:
        _check(lconv_fftconv_bwd(_ptr(dy), _ptr(u), _ptr(k_f), _ptr(D), _ptr(q), _ptr(v), _ptr(du),
                                 _ptr(dq), _ptr(dv), _ptr(dk), _ptr(dD), B, H, N, dt, _ptr(ws), wsb,
                                 _stream(stream)), "lconv_fftconv_bwd")
    else:
        _check(lconv_fftconv_bwd_saved(_ptr(dy), _ptr(u), _ptr(k_f), _ptr(D), _ptr(q), _ptr(v), _ptr(c),
                                       _ptr(du), _ptr(dq), _ptr(dv), _ptr(dk), _ptr(dD), B, H, N, dt,
                                       _ptr(ws), wsb, _stream(stream)), "lconv_fftconv_bwd_saved")
    return du, dq, dv, dk, dD


def fftconv_partial(u, k_f, D, L, q=None, v=None, out=None, stream=None):
    """y = v * ((k * (q*u))[:N] + D * (q*u)) for a filter of L taps (k_f = filter_fft(k [H, L]))
    and u [B, H, N] of any length N."""
    torch = _torch()
    B, H, N = _gated_inputs(u, k_f, D, q, v, out, L=L)
    y = torch.empty_like(u) if out is None else out
    _check(lconv_fftconv_partial_fwd(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), _ptr(q), _ptr(v), B, H, N,
                                     L, dtype_code(u.dtype), _stream(stream)),
           "lconv_fftconv_partial_fwd")
    return y


def fftconv_partial_bwd(dy, u, k_f, D, L, q=None, v=None, need_dk=True, stream=None):
    """Gradients of fftconv_partial (a filter of L taps, k_f = filter_fft(k [H, L])) given dy
    [B, H, N].  Returns (du, dq, dv, dk, dD): du, dq, dv in u's dtype (dq None without q, dv None
    without v); dk [H, L] and dD [H] in float32 (None when need_dk is False)."""
    torch = _torch()
    if dy is None:
        raise ValueError("dy is required")
    B, H, N = _gated_inputs(u, k_f, D, q, v, None, L=L, dy=dy)
    dt = dtype_code(u.dtype)
    du = torch.empty_like(u)
    dq = torch.empty_like(u) if q is not None else None
    dv = torch.empty_like(u) if v is not None else None
    dk = torch.empty((H, L), dtype=torch.float32, device=u.device) if need_dk else None
    dD = torch.empty((H,), dtype=torch.float32, device=u.device) if need_dk else None
    wsb = lconv_fftconv_partial_bwd_workspace_bytes(B, H, N, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=u.device) if wsb else None
    _check(lconv_fftconv_partial_bwd(_ptr(dy), _ptr(u), _ptr(k_f), _ptr(D), _ptr(q), _ptr(v), _ptr(du),
                                     _ptr(dq), _ptr(dv), _ptr(dk), _ptr(dD), B, H, N, L, dt, _ptr(ws), wsb,
                                     _stream(stream)), "lconv_fftconv_partial_bwd")
    return du, dq, dv, dk, dD


def fftconv_sparse(u, k_f, D, keep, q=None, v=None, out=None, stream=None):
    """Frequency-sparse convolution: as fftconv, with the filter spectrum kept only on the
    frequency blocks r (f mod R = r, R = lconv_freq_blocks(N)) in `keep` (an iterable of block
    indices closed under r -> R - r, or a bit mask)."""
    torch = _torch()
    B, H, N = _gated_inputs(u, k_f, D, q, v, out)
    mask = keep if isinstance(keep, int) else sum(1 << int(r) for r in set(keep))
    y = torch.empty_like(u) if out is None else out
    _check(lconv_fftconv_sparse_fwd(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), _ptr(q), _ptr(v), B, H, N,
                                    mask, dtype_code(u.dtype), _stream(stream)),
           "lconv_fftconv_sparse_fwd")
    return y


def butterfly_tables(blocks, N, dtype, stream=None):
    """Matrix-core images (uint8 device tensor) of learned-Butterfly factor blocks for length N:
    `blocks` a complex64 device tensor of lconv_butterfly_blocks_count(N) values (A1, A2, A3,
    B1, B2, B3 back to back, as include/lconv.h lays them out); dtype a torch dtype."""
    torch = _torch()
    dt = dtype_code(dtype)
    count = lconv_butterfly_blocks_count(N)
    if count == 0:
        raise LconvError(4, "lconv_butterfly_blocks_count")
    _need("blocks", blocks, (count,), torch.complex64)
    _on_gpu(blocks=blocks)
    nbytes = lconv_butterfly_tables_bytes(N, dt)
    tables = torch.empty(nbytes, dtype=torch.uint8, device=blocks.device)
    _check(lconv_butterfly_tables(blocks.data_ptr(), tables.data_ptr(), N, dt, _stream(stream)),
           "lconv_butterfly_tables")
    return tables


def butterfly_filter(k, tables, stream=None):
    """Filter spectrum of k [H, N] through the learned forward factors (same opaque layout as
    filter_fft)."""
    torch = _torch()
    _act(k, "k", dims=2)
    H, N = k.shape
    dt = dtype_code(k.dtype)
    _need_buf("tables", tables, lconv_butterfly_tables_bytes(N, dt))
    _on_gpu(k=k, tables=tables)
    nbytes = lconv_filter_fft_bytes(H, N, dt)
    if nbytes == 0 and H * N > 0:
        raise LconvError(3, "lconv_filter_fft_bytes")
    k_f = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=k.device)
    _check(lconv_butterfly_filter(_ptr(k), k_f.data_ptr(), tables.data_ptr(), H, N, dt, _stream(stream)),
           "lconv_butterfly_filter")
    return k_f


def butterfly(u, k_f, D, tables, q=None, v=None, out=None, stream=None):
    """Learned-Butterfly convolution y = v * (Re(S (K . T (q*u)))[:N] + D (q*u)) for u [B, H, N],
    k_f from butterfly_filter, tables from butterfly_tables."""
    torch = _torch()
    B, H, N = _gated_inputs(u, k_f, D, q, v, out)
    dt = dtype_code(u.dtype)
    _need_buf("tables", tables, lconv_butterfly_tables_bytes(N, dt))
    _on_gpu(tables=tables)
    y = torch.empty_like(u) if out is None else out
    _check(lconv_butterfly_fwd(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), _ptr(q), _ptr(v), tables.data_ptr(),
                               B, H, N, dt, _stream(stream)), "lconv_butterfly_fwd")
    return y


def filter_fft2d(k, stream=None):
    """Opaque 2D filter spectrum for centred kernels k [C, Hs, Ws]."""
    torch = _torch()
    _act(k, "k", dims=3)
    _on_gpu(k=k)
    C, Hs, Ws = k.shape
    dt = dtype_code(k.dtype)
    nbytes = lconv_filter_fft2d_bytes(C, Hs, Ws, dt)
    if nbytes == 0 and C > 0:
        raise LconvError(3, "lconv_filter_fft2d_bytes")
    k_f = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=k.device)
    _check(lconv_filter_fft2d(_ptr(k), k_f.data_ptr(), C, Hs, Ws, dt, _stream(stream)), "lconv_filter_fft2d")
    return k_f


def ssm_prepare(lam, W, T, dtype, stream=None):
    """Tables for the state-space filter k[h, t] = Re sum_n W lam^t: lam, W complex64 device
    tensors [H, NS]; T the chunk length.  Returns the opaque prep buffer."""
    torch = _torch()
    if not isinstance(lam, torch.Tensor) or lam.dim() != 2:
        raise ValueError("lam must be a 2-D complex64 tensor [H, NS]")
    H, NS = lam.shape
    _need("lam", lam, (H, NS), torch.complex64)
    _need("W", W, (H, NS), torch.complex64)
    _on_gpu(lam=lam, W=W)
    dt = dtype_code(dtype)
    nbytes = lconv_ssm_prep_bytes(H, NS, T, dt)
    if nbytes == 0:
        raise LconvError(3, "lconv_ssm_prep_bytes")
    prep = torch.empty(nbytes, dtype=torch.uint8, device=lam.device)
    lam_f = torch.view_as_real(lam.contiguous()).contiguous()
    W_f = torch.view_as_real(W.contiguous()).contiguous()
    _check(lconv_ssm_prepare(lam_f.data_ptr(), W_f.data_ptr(), prep.data_ptr(), H, NS, T, dt, _stream(stream)),
           "lconv_ssm_prepare")
    return prep


def fftconv_ssm(u, prep, D, NS, T, q=None, v=None, out=None, stream=None):
    """Causal convolution with a state-space filter, chunked with state passing."""
    torch = _torch()
    tdt, (B, H, N) = _act(u)
    _need("D", D, (H,), tdt)
    _need("q", q, (B, H, N), tdt, optional=True)
    _need("v", v, (B, H, N), tdt, optional=True)
    _need("out", out, (B, H, N), tdt, optional=True)
    _need_buf("prep", prep, lconv_ssm_prep_bytes(H, NS, T, dtype_code(tdt)))
    _on_gpu(u=u, prep=prep, D=D, q=q, v=v, out=out)
    y = torch.empty_like(u) if out is None else out
    wsb = lconv_fftconv_ssm_workspace_bytes(B, H, N, NS, T)
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=u.device)
    _check(lconv_fftconv_ssm_fwd(_ptr(u), _ptr(prep), _ptr(D), _ptr(y), _ptr(q), _ptr(v), B, H, N, NS, T,
                                 dtype_code(u.dtype), ws.data_ptr(), wsb, _stream(stream)),
           "lconv_fftconv_ssm_fwd")
    return y


def filter_fft3d(k, stream=None):
    """Opaque 3D filter spectrum for k [C, S, S, S]."""
    torch = _torch()
    _act(k, "k", dims=4)
    _on_gpu(k=k)
    C, S = k.shape[0], k.shape[1]
    if tuple(k.shape) != (C, S, S, S):
        raise ValueError(f"k has shape {tuple(k.shape)}, expected a cube [C, S, S, S]")
    dt = dtype_code(k.dtype)
    k_f = torch.empty(max(lconv_filter_fft3d_bytes(C, S, dt), 1), dtype=torch.uint8, device=k.device)
    wsb = lconv_filter_fft3d_workspace_bytes(C, S, dt)
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=k.device)
    _check(lconv_filter_fft3d(_ptr(k), k_f.data_ptr(), C, S, dt, ws.data_ptr(), wsb, _stream(stream)),
           "lconv_filter_fft3d")
    return k_f


def fftconv3d(u, k_f, D, out=None, stream=None):
    """3D centred linear convolution plus skip for u [B, C, S, S, S]."""
    torch = _torch()
    tdt, shape = _act(u, dims=5)
    B, C, S = shape[:3]
    if shape != (B, C, S, S, S):
        raise ValueError(f"u has shape {shape}, expected [B, C, S, S, S]")
    dt = dtype_code(tdt)
    _need("D", D, (C,), tdt)
    _need("out", out, shape, tdt, optional=True)
    _need_buf("k_f", k_f, lconv_filter_fft3d_bytes(C, S, dt))
    _on_gpu(u=u, k_f=k_f, D=D, out=out)
    y = torch.empty_like(u) if out is None else out
    wsb = lconv_fftconv3d_workspace_bytes(B, C, S, dt)
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=u.device)
    _check(lconv_fftconv3d_fwd(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), B, C, S, dt, ws.data_ptr(), wsb,
                               _stream(stream)), "lconv_fftconv3d_fwd")
    return y


def fftconv2d(u, k_f, D, out=None, stream=None):
    """2D centred linear convolution plus skip for u [B, C, Hs, Ws]."""
    torch = _torch()
    tdt, (B, C, Hs, Ws) = _act(u, dims=4)
    dt = dtype_code(tdt)
    _need("D", D, (C,), tdt)
    _need("out", out, (B, C, Hs, Ws), tdt, optional=True)
    _need_buf("k_f", k_f, lconv_filter_fft2d_bytes(C, Hs, Ws, dt))
    dev = _on_gpu(u=u, k_f=k_f, D=D, out=out)
    y = torch.empty_like(u) if out is None else out
    wsb = lconv_fftconv2d_workspace_bytes(B, C, Hs, Ws, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _check(lconv_fftconv2d_fwd(_ptr(u), _ptr(k_f), _ptr(D), _ptr(y), B, C, Hs, Ws, dt, _ptr(ws), wsb,
                               _stream(stream)), "lconv_fftconv2d_fwd")
    return y


def fftconv2d_bwd(dy, u, k_f, D, need_dk=True, stream=None):
    """Gradients of fftconv2d given dy [B, C, Hs, Ws]: (du in u's dtype, dk [C, Hs, Ws] and dD [C]
    in float32; dk and dD are None when need_dk is False)."""
    torch = _torch()
    tdt, (B, C, Hs, Ws) = _act(u, dims=4)
    dt = dtype_code(tdt)
    _need("dy", dy, (B, C, Hs, Ws), tdt)
    _need("D", D, (C,), tdt)
    _need_buf("k_f", k_f, lconv_filter_fft2d_bytes(C, Hs, Ws, dt))
    dev = _on_gpu(dy=dy, u=u, k_f=k_f, D=D)
    du = torch.empty_like(u)
    dk = torch.empty((C, Hs, Ws), dtype=torch.float32, device=dev) if need_dk else None
    dD = torch.empty((C,), dtype=torch.float32, device=dev) if need_dk else None
    wsb = lconv_fftconv2d_bwd_workspace_bytes(B, C, Hs, Ws, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _check(lconv_fftconv2d_bwd(_ptr(dy), _ptr(u), _ptr(k_f), _ptr(D), _ptr(du), _ptr(dk), _ptr(dD), B, C, Hs, Ws,
                               dt, _ptr(ws), wsb, _stream(stream)), "lconv_fftconv2d_bwd")
    return du, dk, dD


# ---- linear attention, rotary positions, layer norm ---------------------------------------------

_HERE = contextlib.nullcontext()


def _at(dev, stream):
    """(context, raw stream) of a mixer call on `dev`: outputs and workspaces made inside the context
    belong to the stream that the call runs on, so they are not handed out again before it is done."""
    torch = _torch()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the operands on cuda:{dev}")
        return torch.cuda.stream(stream), stream.cuda_stream     # also makes its device the current one
    raw = _raw_stream()(dev)
    return (_HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev)), raw


@functools.lru_cache(maxsize=None)
def _raw_stream():
    """The call that gives a device's current stream as a raw handle: torch's direct one (0.2 us) where this torch has
    it, else through a Stream object (2.8 us, a fifth of a single-token call)."""
    torch = _torch()
    direct = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return direct or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _same_gpu(names, operands):
    """The device's index, once every given operand is a GPU tensor on one device (the cheap form of
    _on_gpu for calls of a few microseconds)."""
    dev = None
    for t in operands:
        if t is not None:
            at = t.get_device()                                   # less than zero: not a GPU
            if at != dev:
                if at < 0 or dev is not None:
                    _on_gpu(**dict(zip(names.split(), operands)))    # says which
                dev = at
    return dev


@functools.lru_cache(maxsize=256)
def _strides_of(b, h, n):
    return Strides(b, h, n)


def _view(name, t, shape, dtype):
    """An operand of any strides whose last dimension is contiguous: its lconv_strides_t (None: dense)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return None
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    s = t.stride()
    return _strides_of(s[0], s[1], s[2] if len(s) == 4 else 0)


def _in_order_of(x, shape):
    """An empty [B, H, N, D] tensor with x's order of heads and tokens."""
    torch = _torch()
    if x.dim() == 4 and x.shape[1] > 1 and x.shape[2] > 1:
        s = x.stride()
        if s[1] < s[2]:
            B, H, N, D = shape
            return torch.empty_strided(shape, (N * H * D, D, H * D, 1), dtype=x.dtype, device=x.device)
    return torch.empty(shape, dtype=x.dtype, device=x.device)


def _float_dtype(name, t):
    """The library's code of a tensor's dtype."""
    code = _FLOATS.get(t.dtype) if _FLOATS else None
    if code is None:
        torch = _torch()
        _FLOATS.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
        code = _FLOATS.get(t.dtype)
        if code is None:
            raise ValueError(f"{name} has dtype {t.dtype}; supported: float32, float16, bfloat16")
    return code


_FLOATS = {}


def _linattn_shape(q, k, v, dims):
    """(dtype, its code, B, H, G, N, Dk, Dv) of a call's operands, checked where they fix the shape (dims 4: with
    tokens, 3: single tokens)."""
    torch = _torch()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a {dims}-D torch tensor")
    dt = _float_dtype("q", q)
    if dims == 4:
        B, H, N, Dk = q.shape
    else:
        (B, H, Dk), N = q.shape, 1
    G, Dv = k.shape[1], v.shape[-1]
    if G == 0 and H > 0 or G and H % G:
        raise ValueError(f"q has {H} heads, not a multiple of k's {G}")
    return q.dtype, dt, B, H, G, N, Dk, Dv


def _lengths(lengths, B):
    torch = _torch()
    if lengths is not None:
        _need("lengths", lengths, (B,), torch.int32)


def _outputs(name, t, shape, like):
    """An output given by the caller, or a new one in `like`'s order: (tensor, strides)."""
    if t is None:
        torch = _torch()
        if like.is_contiguous() and like.shape == shape:
            return torch.empty_like(like), None
        if len(shape) == 3 or like.is_contiguous():
            return torch.empty(shape, dtype=like.dtype, device=like.device), None
        t = _in_order_of(like, shape)
        return t, None if t.is_contiguous() else _strides_of(*t.stride()[:3])
    return t, _view(name, t, shape, like.dtype)


def linear_attention(q, k, v, log_decay, scale=None, state=None, lengths=None, need_state=True, out=None,
                     state_out=None, stream=None):
    """Linear attention with a decay for each head over q [B, H, N, Dk], k [B, G, N, Dk] and
    v [B, G, N, Dv] (head h uses k/v head h // (H // G)), from a state [B, H, Dk, Dv] in float32:

        S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,    y_t = scale S_t^T q_t

    scale: 1 / sqrt(Dk) unless given.  lengths: int32 [B], tokens past a row's length count for
    nothing and give y = 0.  Returns (y [B, H, N, Dv] in q's dtype and order of dimensions, the state
    after each row's last token; None without need_state).  state_out may be `state` itself."""
    torch = _torch()
    tdt, dt, B, H, G, N, Dk, Dv = _linattn_shape(q, k, v, 4)
    qs, ks, vs = _view("q", q, (B, H, N, Dk), tdt), _view("k", k, (B, G, N, Dk), tdt), _view("v", v, (B, G, N, Dv), tdt)
    _need("log_decay", log_decay, (H,), torch.float32)
    _need("state", state, (B, H, Dk, Dv), torch.float32, optional=True)
    _need("state_out", state_out, (B, H, Dk, Dv), torch.float32, optional=True)
    _lengths(lengths, B)
    dev = _same_gpu("q k v log_decay state lengths out state_out", (q, k, v, log_decay, state, lengths, out, state_out))
    scale = 1.0 / math.sqrt(max(Dk, 1)) if scale is None else float(scale)
    ctx, st = _at(dev, stream)
    with ctx:
        y, ys = _outputs("out", out, (B, H, N, Dv), q)
        if state_out is None and need_state:
            state_out = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
        wsb = lconv_linattn_workspace_bytes(B, H, G, N, Dk, Dv, dt)
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_linattn_fwd(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(log_decay), scale, _ptr(state),
                                 _ptr(lengths), _ptr(y), ys, _ptr(state_out), B, H, G, N, Dk, Dv, dt, _ptr(ws), wsb, st),
               "lconv_linattn_fwd")
    return y, state_out


LinearAttentionGrads = namedtuple("LinearAttentionGrads", "dq dk dv dstate dlog_decay")


def linear_attention_bwd(dy, q, k, v, log_decay, scale=None, state=None, dstate=None, lengths=None,
                         need_dlog_decay=False, stream=None):
    """Gradients of linear_attention given dy [B, H, N, Dv] and, where the state it returned was used,
    dstate [B, H, Dk, Dv] in float32.  Returns (dq, dk, dv, dstate, dlog_decay): dq, dk, dv shaped and
    typed like q, k, v (dk and dv summed over the heads that share them), dstate the gradient of the
    state that entered (None without one), dlog_decay [H] in float32 (None unless asked for)."""
    torch = _torch()
    tdt, dt, B, H, G, N, Dk, Dv = _linattn_shape(q, k, v, 4)
    qs, ks, vs = _view("q", q, (B, H, N, Dk), tdt), _view("k", k, (B, G, N, Dk), tdt), _view("v", v, (B, G, N, Dv), tdt)
    dys = _view("dy", dy, (B, H, N, Dv), tdt)
    _need("log_decay", log_decay, (H,), torch.float32)
    _need("state", state, (B, H, Dk, Dv), torch.float32, optional=True)
    _need("dstate", dstate, (B, H, Dk, Dv), torch.float32, optional=True)
    _lengths(lengths, B)
    dev = _same_gpu("dy q k v log_decay state dstate lengths", (dy, q, k, v, log_decay, state, dstate, lengths))
    scale = 1.0 / math.sqrt(max(Dk, 1)) if scale is None else float(scale)
    ctx, st = _at(dev, stream)
    with ctx:
        dq, dqs = _outputs("dq", None, (B, H, N, Dk), q)
        dk, dks = _outputs("dk", None, (B, G, N, Dk), k)
        dv, dvs = _outputs("dv", None, (B, G, N, Dv), v)
        ds = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev) if state is not None else None
        dl = torch.empty((H,), dtype=torch.float32, device=dev) if need_dlog_decay else None
        wsb = lconv_linattn_bwd_workspace_bytes(B, H, G, N, Dk, Dv, dt)
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_linattn_bwd(_ptr(dy), dys, _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(log_decay), scale,
                                 _ptr(state), _ptr(dstate), _ptr(lengths), _ptr(dq), dqs, _ptr(dk), dks, _ptr(dv), dvs,
                                 _ptr(ds), _ptr(dl), B, H, G, N, Dk, Dv, dt, _ptr(ws), wsb, st), "lconv_linattn_bwd")
    return LinearAttentionGrads(dq, dk, dv, ds, dl)


def linear_attention_step(q, k, v, log_decay, state, scale=None, slots=None, out=None, stream=None):
    """One token of every sequence: q [B, H, Dk], k [B, G, Dk], v [B, G, Dv]; the states
    [slots, H, Dk, Dv] in float32 are moved on in place.  slots: int32 [B], the state that each row
    continues (outside the states: an idle row, y = 0); without it row b has state b.  No two rows may
    have the same slot.  Returns y [B, H, Dv]."""
    torch = _torch()
    tdt, dt, B, H, G, _, Dk, Dv = _linattn_shape(q, k, v, 3)
    qs, ks, vs = _view("q", q, (B, H, Dk), tdt), _view("k", k, (B, G, Dk), tdt), _view("v", v, (B, G, Dv), tdt)
    _need("log_decay", log_decay, (H,), torch.float32)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a 4-D torch tensor")
    nslots = state.shape[0]
    _need("state", state, (nslots, H, Dk, Dv), torch.float32)
    if slots is not None:
        _need("slots", slots, (B,), torch.int32)
    elif nslots < B:
        raise ValueError(f"{B} rows and {nslots} states: slots are needed")
    dev = _same_gpu("q k v log_decay state slots out", (q, k, v, log_decay, state, slots, out))
    scale = 1.0 / math.sqrt(max(Dk, 1)) if scale is None else float(scale)
    ctx, st = _at(dev, stream)
    with ctx:
        y, ys = _outputs("out", out, (B, H, Dv), q)
        _check(lconv_linattn_step(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(log_decay), scale, _ptr(state),
                                  _ptr(slots), _ptr(y), ys, B, H, G, Dk, Dv, nslots, dt, st),
               "lconv_linattn_step")
    return y


def rotary_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=4096, fast=32.0, slow=1.0, device="cuda"):
    """(inv_freq [rot / 2] in float32, magnitude) for ``rotary``.  Unscaled: base^(-2p / rot), 1.
    scaling, for contexts `factor` times the original's length:
      "linear"    every frequency divided by factor (positions interpolated);
      "base"      the base raised to base * factor^(rot / (rot - 2)): the fastest pair keeps its
                  frequency, the slowest is divided by factor;
      "by_parts"  the interpolation by parts of YaRN (Peng, Quesnelle, Fan, Shippole 2023): pairs that turn
                  at least `fast` times within `original` positions keep their frequency, those that turn at
                  most `slow` times are divided by factor, a ramp in the pair's index between (from the last
                  whole index of the one kind to the first of the other); magnitude 1 + 0.1 ln(factor)."""
    torch = _torch()
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if scaling not in (None, "linear", "base", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if factor < 1.0:
        raise ValueError(f"factor must be at least 1, got {factor}")
    if scaling == "by_parts" and not (base > 1.0 and original > 0 and fast > slow > 0):
        raise ValueError(f"by_parts needs base > 1, original > 0 and fast > slow > 0, got {base}, {original}, {fast}, {slow}")
    magnitude = 1.0
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    p = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * p / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        # the index, whole or not, whose wavelength 2 pi base^(2p / rot) fits `turns` times into the original context; it falls
        # with the turns, so the ramp's ends are at least one apart.  They may lie outside the pairs that there are.
        pair = lambda turns: rot * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        lo, hi = math.floor(pair(fast)), math.ceil(pair(slow))
        ramp = ((p - lo) / (hi - lo)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
        magnitude = 1.0 + 0.1 * math.log(factor)
    return f.to(torch.float32).to(device), magnitude


def rotary(q, k, positions, inv_freq, interleaved=False, inverse=False, magnitude=1.0, out=None, stream=None):
    """Rotary positions of q [B, H, N, D] and k [B, G, N, D] (or None) in one launch: the first
    2 * len(inv_freq) dimensions of every head are turned in pairs by position * inv_freq, the others
    copied.  Pairs are (p, p + rot / 2), or (2p, 2p + 1) with interleaved.  inverse turns back (with the
    same magnitude: the gradient).  positions: int32 [B, N] or [N], or None for 0 .. N-1.  out: a pair of
    outputs (q and k themselves for in place).  Returns (q', k')."""
    torch = _torch()
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D torch tensor")
    dt = _float_dtype("q", q)
    B, H, N, D = q.shape
    qs = _view("q", q, (B, H, N, D), q.dtype)
    G, ks = 0, None
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a 4-D torch tensor")
        G = k.shape[1]
        ks = _view("k", k, (B, G, N, D), q.dtype)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a 1-D torch tensor")
    rot = 2 * inv_freq.shape[0]
    _need("inv_freq", inv_freq, (rot // 2,), torch.float32)
    pos_stride = 0
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32:
            raise ValueError("positions must be an int32 torch tensor")
        if tuple(positions.shape) not in ((B, N), (N,)):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(B, N)} or {(N,)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous in its last dimension")
        pos_stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    oq, ok = (None, None) if out is None else out
    if k is None and ok is not None:
        raise ValueError("an output for k without k")
    dev = _same_gpu("q k positions inv_freq out_q out_k", (q, k, positions, inv_freq, oq, ok))
    flags = (ROTARY_INTERLEAVED if interleaved else ROTARY_HALF) | (ROTARY_INVERSE if inverse else 0)
    ctx, st = _at(dev, stream)
    with ctx:
        yq, yqs = _outputs("out of q", oq, (B, H, N, D), q)
        yk, yks = (None, None) if k is None else _outputs("out of k", ok, (B, G, N, D), k)
        _check(lconv_rotary(_ptr(q), qs, _ptr(k), ks, _ptr(positions), pos_stride, _ptr(inv_freq), float(magnitude),
                            _ptr(yq), yqs, _ptr(yk), yks, B, H, G, N, D, rot, flags, dt, st),
               "lconv_rotary")
    return yq, yk


def _dense_like(x):
    torch = _torch()
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _rows(name, t, shape, dtype):
    """(rows, C, row stride) of a tensor normalised over its last dimension: dense, or with contiguous rows that are evenly
    spaced (a slice of the last dimension, one token of every sequence)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    C = shape[-1]
    rows = 1
    for n in shape[:-1]:
        rows *= n
    if t.is_contiguous():
        return rows, C, C
    step = whole = None                      # the spacing of rows, and what the dimensions so far span
    for n, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = st
        elif st != whole:
            step = -1
            break
        whole = st * n
    if (t.stride(-1) != 1 and C > 1) or (step is not None and step < C):
        raise ValueError(f"{name} must be contiguous, or have contiguous rows that are evenly spaced and do not overlap")
    return rows, C, C if step is None else step


def layer_norm(x, weight=None, bias=None, eps=1e-5, need_stats=True, out=None, stream=None):
    """Layer norm over the last dimension of x [..., C], dense or with evenly spaced rows: (x - mean) rstd weight + bias;
    weight and bias [C] in x's dtype, or None.  Returns (y, mean, rstd), the statistics in float32 and x's leading shape
    (None without need_stats).  out may be x."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a torch tensor of at least one dimension")
    dt = _float_dtype("x", x)
    rows, C, xs = _rows("x", x, x.shape, x.dtype)
    _need("weight", weight, (C,), x.dtype, optional=True)
    _need("bias", bias, (C,), x.dtype, optional=True)
    dev = _same_gpu("x weight bias out", (x, weight, bias, out))
    ctx, st = _at(dev, stream)
    with ctx:
        y = _dense_like(x) if out is None else out
        ys = C if out is None else _rows("out", y, x.shape, x.dtype)[2]
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev) if need_stats else None
        rstd = torch.empty_like(mean) if need_stats else None
        _check(lconv_layernorm_fwd(_ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(y), ys, _ptr(mean), _ptr(rstd), rows, C,
                                   float(eps), dt, st), "lconv_layernorm_fwd")
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd, need_dweight=True, need_dbias=True, out=None, stream=None):
    """Gradients of layer_norm given dy like x, with the statistics that it returned.  Returns
    (dx in x's dtype, dweight [C], dbias [C] in float32); dweight is None without weight or
    need_dweight, dbias without need_dbias.  out (dx) may be dy or x."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a torch tensor of at least one dimension")
    dt = _float_dtype("x", x)
    rows, C, xs = _rows("x", x, x.shape, x.dtype)
    dys = _rows("dy", dy, x.shape, x.dtype)[2]
    _need("weight", weight, (C,), x.dtype, optional=True)
    _need("mean", mean, x.shape[:-1], torch.float32)
    _need("rstd", rstd, x.shape[:-1], torch.float32)
    dev = _same_gpu("dy x weight mean rstd out", (dy, x, weight, mean, rstd, out))
    ctx, st = _at(dev, stream)
    with ctx:
        dx = _dense_like(x) if out is None else out
        dxs = C if out is None else _rows("out", dx, x.shape, x.dtype)[2]
        dw = torch.empty((C,), dtype=torch.float32, device=dev) if need_dweight and weight is not None else None
        db = None if not need_dbias else torch.empty_like(dw) if dw is not None else torch.empty((C,), dtype=torch.float32, device=dev)
        wsb = lconv_layernorm_bwd_workspace_bytes(rows, C) if dw is not None or db is not None else 0
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_layernorm_bwd(_ptr(dy), dys, _ptr(x), xs, _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dx), dxs,
                                   _ptr(dw), _ptr(db), rows, C, dt, _ptr(ws), wsb, st),
               "lconv_layernorm_bwd")
    return dx, dw, db


# ---- norms of q and k with rotary positions ------------------------------------------------------

QKNORM_CENTRED = 4


def _qk_operands(q, k, q_weight, k_weight, positions, inv_freq):
    """(dtype code, B, H, G, N, D, rot, position stride, strides of q and k), checked."""
    torch = _torch()
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D torch tensor")
    dt = _float_dtype("q", q)
    B, H, N, D = q.shape
    qs = _view("q", q, q.shape, q.dtype)
    G, ks = 0, None
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a 4-D torch tensor")
        G = k.shape[1]
        ks = _view("k", k, (B, G, N, D), q.dtype)
    elif k_weight is not None:
        raise ValueError("a weight for k without k")
    _need("q_weight", q_weight, (D,), q.dtype, optional=True)
    _need("k_weight", k_weight, (D,), q.dtype, optional=True)
    rot, pos_stride = 0, 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a 1-D torch tensor")
        rot = 2 * inv_freq.shape[0]
        _need("inv_freq", inv_freq, (rot // 2,), torch.float32)
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32:
            raise ValueError("positions must be an int32 torch tensor")
        if positions.shape != (N,) and positions.shape != (B, N):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(B, N)} or {(N,)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous in its last dimension")
        pos_stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    return dt, B, H, G, N, D, rot, pos_stride, qs, ks


def qk_norm_rotary(q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, centred=False, interleaved=False, magnitude=1.0,
                   out=None, stream=None):
    """Every head's row of q [B, H, N, D] and k [B, G, N, D] (or None) over its root mean square (centred: of the row less its
    mean), times a weight [D] in q's dtype (None: ones), then ``rotary`` of its first 2 * len(inv_freq) dimensions (inv_freq
    None: none), in one pass.  positions, interleaved, magnitude and out as for ``rotary``.  Returns (q', k')."""
    dt, B, H, G, N, D, rot, pos_stride, qs, ks = _qk_operands(q, k, q_weight, k_weight, positions, inv_freq)
    oq, ok = (None, None) if out is None else out
    if k is None and ok is not None:
        raise ValueError("an output for k without k")
    dev = _same_gpu("q k q_weight k_weight positions inv_freq out_q out_k",
                    (q, k, q_weight, k_weight, positions, inv_freq, oq, ok))
    flags = (ROTARY_INTERLEAVED if interleaved else ROTARY_HALF) | (QKNORM_CENTRED if centred else 0)
    ctx, st = _at(dev, stream)
    with ctx:
        yq, yqs = _outputs("out of q", oq, (B, H, N, D), q)
        yk, yks = (None, None) if k is None else _outputs("out of k", ok, (B, G, N, D), k)
        _check(lconv_qknorm_rotary_fwd(_ptr(q), qs, _ptr(k), ks, _ptr(q_weight), _ptr(k_weight), _ptr(positions), pos_stride,
                                       _ptr(inv_freq), float(magnitude), float(eps), _ptr(yq), yqs, _ptr(yk), yks, B, H, G, N,
                                       D, rot, flags, dt, st), "lconv_qknorm_rotary_fwd")
    return yq, yk


QkNormGrads = namedtuple("QkNormGrads", "dq dk dq_weight dk_weight")


def qk_norm_rotary_bwd(dyq, dyk, q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, centred=False, interleaved=False,
                       magnitude=1.0, need_dweight=True, stream=None):
    """Gradients of qk_norm_rotary given those of its results, from its inputs.  Returns (dq, dk in q's dtype, dq_weight,
    dk_weight [D] in float32; None for what is not there or, the weights', without need_dweight)."""
    torch = _torch()
    dt, B, H, G, N, D, rot, pos_stride, qs, ks = _qk_operands(q, k, q_weight, k_weight, positions, inv_freq)
    dyqs = _view("dyq", dyq, (B, H, N, D), q.dtype)
    if (k is None) != (dyk is None):
        raise ValueError("dyk goes with k")
    dyks = None if k is None else _view("dyk", dyk, (B, G, N, D), q.dtype)
    dev = _same_gpu("dyq dyk q k q_weight k_weight positions inv_freq", (dyq, dyk, q, k, q_weight, k_weight, positions, inv_freq))
    flags = (ROTARY_INTERLEAVED if interleaved else ROTARY_HALF) | (QKNORM_CENTRED if centred else 0)
    ctx, st = _at(dev, stream)
    with ctx:
        dq, dqs = _outputs("dq", None, (B, H, N, D), q)
        dk, dks = (None, None) if k is None else _outputs("dk", None, (B, G, N, D), k)
        new = lambda w: torch.empty((D,), dtype=torch.float32, device=dev) if need_dweight and w is not None else None  # noqa: E731
        dwq, dwk = new(q_weight), new(k_weight)
        wsb = lconv_qknorm_rotary_bwd_workspace_bytes(B, H, G, N, D, rot) if dwq is not None or dwk is not None else 0
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_qknorm_rotary_bwd(_ptr(dyq), dyqs, _ptr(dyk), dyks, _ptr(q), qs, _ptr(k), ks, _ptr(q_weight), _ptr(k_weight),
                                       _ptr(positions), pos_stride, _ptr(inv_freq), float(magnitude), float(eps), _ptr(dq), dqs,
                                       _ptr(dk), dks, _ptr(dwq), _ptr(dwk), B, H, G, N, D, rot, flags, dt, _ptr(ws), wsb, st),
               "lconv_qknorm_rotary_bwd")
    return QkNormGrads(dq, dk, dwq, dwk)


# ---- gated linear recurrence --------------------------------------------------------------------

GATES = {"log": 0, "sigmoid": 1, "rate": 2}            # LCONV_GATE_*
MIXES = {"plain": 0, "convex": 4, "norm": 8}           # LCONV_MIX_*


def _scan_operands(x, z, gate, mix, input_gate, rate, dims):
    """(dtype code, flags, strides of x, z and input_gate) of a call's operands, checked where they fix the shape (dims 3:
    with tokens, 2: single tokens, whose strides are those of their rows)."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() != dims:
        raise ValueError(f"x must be a {dims}-D torch tensor")
    dt = _float_dtype("x", x)
    if gate not in GATES or mix not in MIXES:
        raise ValueError(f"unknown gate {gate!r} or mix {mix!r}; gates: {', '.join(GATES)}; mixes: {', '.join(MIXES)}")
    if (rate is not None) != (gate == "rate"):
        raise ValueError('rate goes with gate="rate", and only with it')
    _need("rate", rate, (x.shape[-1],), torch.float32, optional=True)
    shape, like = x.shape, x.dtype
    s = (_tokens("x", x, shape, like), _tokens("z", z, shape, like),
         None if input_gate is None else _tokens("input_gate", input_gate, shape, like))
    return dt, GATES[gate] | MIXES[mix], s


def _tokens(name, t, shape, dtype):
    """An operand [B, N, C] (or [B, C]) of any strides whose last dimension is contiguous: its lconv_strides_t, None for a
    dense one ([B, C]: the stride of its rows)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return None if len(shape) == 3 else shape[-1]
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    s = t.stride()
    return _strides_of(s[0], 0, s[1]) if len(shape) == 3 else s[0]


def _token_output(name, t, like):
    """An output given by the caller, or a new dense one shaped like x: (tensor, strides)."""
    if t is None:
        torch = _torch()
        t = torch.empty_like(like) if like.is_contiguous() else torch.empty(like.shape, dtype=like.dtype, device=like.device)
        return t, None if like.dim() == 3 else like.shape[-1]
    return t, _tokens(name, t, like.shape, like.dtype)


GatedScan = namedtuple("GatedScan", "y state marks")


def gated_scan(x, z, gate="sigmoid", mix="plain", input_gate=None, rate=None, state=None, lengths=None, need_state=True,
               need_marks=False, out=None, state_out=None, stream=None):
    """Gated linear recurrence over x [B, N, C] with decays from z [B, N, C], from a state [B, C] in float32:

        h_t = a_t h_{t-1} + m_t s_t x_t,    y_t = h_t

    gate: "log" (log a = z, at most 0; a z above 0 is not refused, and leaves its channel's results without meaning), "sigmoid"
    (a = sigmoid(z)) or "rate" (log a = -rate sigmoid(z), rate [C] in float32, at least 0).  mix: "plain" (m = 1), "convex" (1 - a) or "norm" (sqrt(1 - a^2)).  s is sigmoid(input_gate), or 1
    without one.  lengths: int32 [B], tokens past a row's length count for nothing and give y = 0.  Returns (y in x's dtype,
    the state after each row's last token; None without need_state, marks for the gradient call; None without need_marks).
    state_out may be `state` itself."""
    torch = _torch()
    dt, flags, (xs, zs, igs) = _scan_operands(x, z, gate, mix, input_gate, rate, 3)
    B, N, C = x.shape
    _need("state", state, (B, C), torch.float32, optional=True)
    _need("state_out", state_out, (B, C), torch.float32, optional=True)
    _lengths(lengths, B)
    dev = _same_gpu("x z input_gate rate state lengths out state_out", (x, z, input_gate, rate, state, lengths, out, state_out))
    ctx, st = _at(dev, stream)
    with ctx:
        y, ys = _token_output("out", out, x)
        if state_out is None and need_state:
            state_out = torch.empty((B, C), dtype=torch.float32, device=dev) if state is None else torch.empty_like(state)
        marks = torch.empty(lconv_gated_scan_marks_bytes(B, N, C) // 4, dtype=torch.float32, device=dev) if need_marks else None
        wsb = lconv_gated_scan_workspace_bytes(B, N, C, dt)
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_gated_scan_fwd(_ptr(x), xs, _ptr(z), zs, _ptr(input_gate), igs, _ptr(rate), _ptr(state), _ptr(lengths),
                                    _ptr(y), ys, _ptr(state_out), _ptr(marks), B, N, C, flags, dt, _ptr(ws), wsb, st),
               "lconv_gated_scan_fwd")
    return GatedScan(y, state_out, marks)


GatedScanGrads = namedtuple("GatedScanGrads", "dx dz dinput_gate drate dstate")


def gated_scan_bwd(dy, x, z, marks, gate="sigmoid", mix="plain", input_gate=None, rate=None, dstate=None, lengths=None,
                   need_drate=True, need_dstate=True, stream=None):
    """Gradients of gated_scan given dy [B, N, C], the marks that it returned for the same operands and, where the state it
    returned was used, dstate [B, C] in float32.  Returns (dx, dz, dinput_gate in x's dtype, drate [C] and dstate [B, C], the
    gradient of the state that entered, in float32); dinput_gate is None without one, drate without a rate or need_drate,
    dstate without need_dstate."""
    torch = _torch()
    dt, flags, (xs, zs, igs) = _scan_operands(x, z, gate, mix, input_gate, rate, 3)
    B, N, C = x.shape
    dys = _tokens("dy", dy, x.shape, x.dtype)
    _need("dstate", dstate, (B, C), torch.float32, optional=True)
    _need("marks", marks, (lconv_gated_scan_marks_bytes(B, N, C) // 4,), torch.float32)
    _lengths(lengths, B)
    dev = _same_gpu("dy x z marks input_gate rate dstate lengths", (dy, x, z, marks, input_gate, rate, dstate, lengths))
    ctx, st = _at(dev, stream)
    with ctx:
        dx, dxs = _token_output("dx", None, x)
        dz, dzs = _token_output("dz", None, x)
        dig, digs = (None, None) if input_gate is None else _token_output("dinput_gate", None, x)
        dr = torch.empty((C,), dtype=torch.float32, device=dev) if rate is not None and need_drate else None
        ds = torch.empty((B, C), dtype=torch.float32, device=dev) if need_dstate else None
        wsb = lconv_gated_scan_bwd_workspace_bytes(B, N, C, flags, dt)
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_gated_scan_bwd(_ptr(dy), dys, _ptr(x), xs, _ptr(z), zs, _ptr(input_gate), igs, _ptr(rate), _ptr(marks),
                                    _ptr(dstate), _ptr(lengths), _ptr(dx), dxs, _ptr(dz), dzs, _ptr(dig), digs, _ptr(dr),
                                    _ptr(ds), B, N, C, flags, dt, _ptr(ws), wsb, st), "lconv_gated_scan_bwd")
    return GatedScanGrads(dx, dz, dig, dr, ds)


def gated_scan_step(x, z, state, gate="sigmoid", mix="plain", input_gate=None, rate=None, slots=None, out=None, stream=None):
    """One token of every sequence: x, z and input_gate [B, C]; the states [slots, C] in float32 are moved on in place.
    slots: int32 [B], the state that each row continues (outside the states: an idle row, y = 0); without it row b has state
    b.  No two rows may have the same slot.  Returns y [B, C]."""
    torch = _torch()
    dt, flags, (xs, zs, igs) = _scan_operands(x, z, gate, mix, input_gate, rate, 2)
    B, C = x.shape
    nslots = _pool("state", state, 2, slots, B)
    _need("state", state, (nslots, C), torch.float32)
    dev = _same_gpu("x z input_gate rate state slots out", (x, z, input_gate, rate, state, slots, out))
    ctx, st = _at(dev, stream)
    with ctx:
        y, ys = _token_output("out", out, x)
        _check(lconv_gated_scan_step(_ptr(x), xs, _ptr(z), zs, _ptr(input_gate), igs or 0, _ptr(rate), _ptr(state), _ptr(slots),
                                     _ptr(y), ys, B, C, nslots, flags, dt, st), "lconv_gated_scan_step")
    return y


def _pool(name, state, dims, slots, B):
    """The number of states in a pool that single tokens find theirs in."""
    torch = _torch()
    if not isinstance(state, torch.Tensor) or state.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-D torch tensor")
    if slots is not None:
        _need("slots", slots, (B,), torch.int32)
    elif state.shape[0] < B:
        raise ValueError(f"{B} rows and {state.shape[0]} states: slots are needed")
    return state.shape[0]


# ---- short convolution --------------------------------------------------------------------------

SHORTCONV_SILU = 1


def _conv_operands(x, weight, bias, activation, dims):
    """(dtype code, flags, K, strides of x), checked."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() != dims:
        raise ValueError(f"x must be a {dims}-D torch tensor")
    dt = _float_dtype("x", x)
    if activation not in (None, "silu"):
        raise ValueError(f"unknown activation {activation!r}; there are None and 'silu'")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a 2-D torch tensor")
    K = weight.shape[1]
    if not 2 <= K <= 8:
        raise ValueError(f"weight has {K} taps; supported: 2 to 8")
    C = x.shape[-1]
    _need("weight", weight, (C, K), x.dtype)
    _need("bias", bias, (C,), x.dtype, optional=True)
    return dt, SHORTCONV_SILU if activation else 0, K, _tokens("x", x, x.shape, x.dtype)


def short_conv(x, weight, bias=None, activation=None, state=None, lengths=None, need_state=True, out=None, state_out=None,
               stream=None):
    """Causal convolution along the tokens of x [B, N, C], one filter weight[c] of K taps (2 to 8, the last one on the token
    itself) per channel, a bias [C] and, with activation "silu", p sigmoid(p), all in x's dtype.  state: [B, K - 1, C] in x's
    dtype, the inputs before the first token, oldest first.  lengths: int32 [B], tokens past a row's length count for nothing
    and give y = 0.  Returns (y, the last K - 1 inputs before each row's end; None without need_state).  state_out may be
    `state` itself."""
    torch = _torch()
    dt, flags, K, xs = _conv_operands(x, weight, bias, activation, 3)
    B, N, C = x.shape
    _need("state", state, (B, K - 1, C), x.dtype, optional=True)
    _need("state_out", state_out, (B, K - 1, C), x.dtype, optional=True)
    _lengths(lengths, B)
    dev = _same_gpu("x weight bias state lengths out state_out", (x, weight, bias, state, lengths, out, state_out))
    ctx, st = _at(dev, stream)
    with ctx:
        y, ys = _token_output("out", out, x)
        if state_out is None and need_state:
            state_out = torch.empty((B, K - 1, C), dtype=x.dtype, device=dev) if state is None else torch.empty_like(state)
        _check(lconv_shortconv_fwd(_ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(y), ys, _ptr(state_out),
                                   B, N, C, K, flags, dt, st), "lconv_shortconv_fwd")
    return y, state_out


ShortConvGrads = namedtuple("ShortConvGrads", "dx dweight dbias dstate")


def short_conv_bwd(dy, x, weight, bias=None, activation=None, state=None, dstate=None, lengths=None, need_dweight=True,
                   stream=None):
    """Gradients of short_conv given dy [B, N, C] and, where the state it returned was used, dstate [B, K - 1, C], from its
    inputs.  Returns (dx in x's dtype, dweight [C, K] and dbias [C] in float32, dstate in x's dtype, the gradient of the state
    that entered); dweight and dbias are None without need_dweight, dbias without a bias, dstate without a state."""
    torch = _torch()
    dt, flags, K, xs = _conv_operands(x, weight, bias, activation, 3)
    B, N, C = x.shape
    dys = _tokens("dy", dy, x.shape, x.dtype)
    _need("state", state, (B, K - 1, C), x.dtype, optional=True)
    _need("dstate", dstate, (B, K - 1, C), x.dtype, optional=True)
    _lengths(lengths, B)
    dev = _same_gpu("dy x weight bias state dstate lengths", (dy, x, weight, bias, state, dstate, lengths))
    ctx, st = _at(dev, stream)
    with ctx:
        dx, dxs = _token_output("dx", None, x)
        dw = torch.empty((C, K), dtype=torch.float32, device=dev) if need_dweight else None
        db = torch.empty((C,), dtype=torch.float32, device=dev) if need_dweight and bias is not None else None
        ds = None if state is None else torch.empty_like(state)
        wsb = lconv_shortconv_bwd_workspace_bytes(B, N, C, K) if need_dweight else 0
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
        _check(lconv_shortconv_bwd(_ptr(dy), dys, _ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(state), _ptr(dstate), _ptr(lengths),
                                   _ptr(dx), dxs, _ptr(dw), _ptr(db), _ptr(ds), B, N, C, K, flags, dt, _ptr(ws), wsb, st),
               "lconv_shortconv_bwd")
    return ShortConvGrads(dx, dw, db, ds)


def short_conv_step(x, weight, state, bias=None, activation=None, slots=None, out=None, stream=None):
    """One token of every sequence: x [B, C]; the inputs [slots, K - 1, C] in x's dtype move on by one in place.  slots: int32
    [B], the state that each row continues (outside the states: an idle row, y = 0); without it row b has state b.  No two rows
    may have the same slot.  Returns y [B, C]."""
    dt, flags, K, xs = _conv_operands(x, weight, bias, activation, 2)
    B, C = x.shape
    nslots = _pool("state", state, 3, slots, B)
    _need("state", state, (nslots, K - 1, C), x.dtype)
    dev = _same_gpu("x weight bias state slots out", (x, weight, bias, state, slots, out))
    ctx, st = _at(dev, stream)
    with ctx:
        y, ys = _token_output("out", out, x)
        _check(lconv_shortconv_step(_ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(state), _ptr(slots), _ptr(y), ys, B, C, K, nslots,
                                    flags, dt, st), "lconv_shortconv_step")
    return y
