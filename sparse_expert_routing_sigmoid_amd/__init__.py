"""Python binding of libmoe_mi355x (DeepSeekMoE layer forward and backward, and
latent attention, on MI355X).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors are torch tensors on the current HIP device; their data
pointers and torch's current stream go through ctypes to the C ABI declared
in include/moe_mi355x.h, with the same entry-point names.

There is no CPU fallback: importing works without a GPU (so the library can
be inspected), but every compute call raises if the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = range(5)
MOE_F32, MOE_BF16, MOE_E4M3, MOE_E2M1 = 0, 1, 2, 3
MOE_COMBINE_NO_RESIDUAL, MOE_COMBINE_NO_SHARED, MOE_COMBINE_NO_ROUTED = 1, 2, 4
MOE_TILE_ROWS = 256
MOE_MAX_K = 16
MOE_MAX_EXPERTS = 1024
MOE_NORM_MAX_D = 32768
MOE_FEW_TOKENS = 32
MLA_MAX_REQUESTS = 8192

# Every symbol the header declares, with its ctypes signature.
_vp, _i, _ll, _sz, _f, _u = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float, ctypes.c_uint
SIGNATURES = {
    "moe_abi_version": (_i, []),
    "moe_status_str": (ctypes.c_char_p, [_i]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_route_workspace_bytes": (_sz, [_i, _i, _i]),
    "moe_route": (_i, [_vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_permute_rows": (_sz, [_i, _i, _i, _i, _i]),
    "moe_permute_tiles_max": (_sz, [_i, _i, _i, _i, _i]),
    "moe_permute_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "moe_permute": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_permute_noalloc_scratch_bytes": (_sz, []),
    "moe_permute_noalloc": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_gemm_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "moe_expert_gemm": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                             _vp, _vp, _vp, _vp, _vp, _sz, _vp, _i, _vp]),
    "moe_gemm_combine_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "moe_expert_gemm_combine": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _vp] + [_i] * 7 + [_vp] * 6 +
                                [_vp, _i, _u, _vp, _sz, _vp, _vp]),
    "moe_combine": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _u, _vp, _i, _vp]),
    "moe_bias_update": (_i, [_vp, _i, _ll, _f, _vp, _vp]),
    "fp8_quantize_tiles": (_i, [_vp, _i, _ll, _ll, _i, _i, _vp, _vp, _vp]),
    "fp8_dequantize_tiles": (_i, [_vp, _vp, _ll, _ll, _i, _i, _vp, _i, _vp]),
    "moe_gemm_train_workspace_bytes": (_sz, [_i] * 7),
    "moe_expert_gemm_train": (_i, [_vp] * 3 + [_i] * 7 + [_vp] * 5 + [_sz] + [_vp] * 3 + [_i, _vp]),
    "moe_combine_backward": (_i, [_vp, _i, _vp, _i] + [_vp] * 4 + [_i] * 5 + [_vp] * 5),
    "moe_gemm_backward_workspace_bytes": (_sz, [_i] * 7),
    "moe_expert_gemm_backward": (_i, [_vp] * 6 + [_i] * 7 + [_vp] * 5 + [_sz] + [_vp] * 3 + [_i, _vp]),
    "moe_gemm_train_w8_workspace_bytes": (_sz, [_i] * 7),
    "moe_expert_gemm_train_w8": (_i, [_vp] * 6 + [_i] * 7 + [_vp] * 5 + [_sz] + [_vp] * 3 + [_i, _vp]),
    "moe_gemm_backward_w8_workspace_bytes": (_sz, [_i] * 7),
    "moe_expert_gemm_backward_w8": (_i, [_vp] * 8 + [_i] * 7 + [_vp] * 5 + [_sz] + [_vp] * 3 + [_i, _vp]),
    "moe_gemm_backward_f8_workspace_bytes": (_sz, [_i] * 7),
    "moe_expert_gemm_backward_f8": (_i, [_vp] * 8 + [_i] * 7 + [_vp] * 5 + [_sz] + [_vp] * 3 + [_i, _vp]),
    "fp8_quantize_runs_max": (_ll, [_ll, _i]),
    "fp8_quantize_runs": (_i, [_vp, _i, _ll, _i, _vp, _i, _vp, _i, _ll, _vp, _vp, _vp, _vp]),
    "moe_route_backward": (_i, [_vp, _i, _vp, _vp, _i] + [_vp] * 7 + [_i] * 5 + [_vp, _i, _vp, _vp]),
    "moe_rmsnorm": (_i, [_vp, _i, _vp, _i, _vp, _i, _f, _ll, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp]),
    "moe_rmsnorm_backward_workspace_bytes": (_sz, [_ll, _i]),
    "moe_rmsnorm_backward": (_i, [_vp, _i, _vp, _i, _vp, _i, _vp, _vp, _ll, _i, _vp, _vp, _vp, _sz, _vp]),
    "fp4_quantize_groups": (_i, [_vp, _i, _ll, _ll, _vp, _vp, _vp]),
    "fp4_dequantize_groups": (_i, [_vp, _vp, _ll, _ll, _vp, _i, _vp]),
    "fp4_matvec_workspace_bytes": (_sz, [_i, _ll, _i]),
    "fp4_matvec": (_i, [_vp, _i, _vp, _vp, _i, _ll, _i, _vp, _i, _vp, _sz, _vp]),
    "moe_layer_few_workspace_bytes": (_sz, [_i] * 7),
    "moe_layer_few": (_i, [_vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp] + [_i] * 6 + [_vp, _i] + [_vp] * 5 +
                      [_sz, _vp, _i, _vp]),
    "mla_pages_workspace_bytes": (_sz, [_i]),
    "mla_pages_extend": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _i] + [_vp] * 7 + [_i, _vp, _sz, _vp]),
    "mla_pages_release": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _i, _vp, _vp]),
    "mla_cache_write": (_i, [_vp, _ll, _vp, _ll, _vp, _ll, _i, _i, _vp, _ll, _vp]),
    "mla_decode_workspace_bytes": (_sz, [_i] * 7 + [_ll]),
    "mla_decode": (_i, [_vp, _vp, _vp, _ll, _i, _vp, _i, _vp] + [_i] * 7 + [_ll, _f, _vp, _i, _vp, _sz, _vp]),
    "mla_attention": (_i, [_vp, _vp, _vp, _ll, _vp, _vp, _i, _ll, _ll, _i, _i, _i, _i, _i, _f, _vp, _i, _vp, _vp]),
    "mla_attention_backward_workspace_bytes": (_sz, [_ll, _ll, _i, _i]),
    "mla_attention_backward": (_i, [_vp] * 4 + [_ll, _vp, _i, _vp, _vp, _vp, _i, _ll, _ll] + [_i] * 5 +
                               [_f, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_status_name(status)}: {msg}")
        self.status = status


def _status_name(s: int) -> str:
    return {0: "MOE_OK", 1: "MOE_EINVAL", 2: "MOE_EUNSUPPORTED", 3: "MOE_EWORKSPACE", 4: "MOE_EHIP"}.get(s, str(s))


def lib() -> ctypes.CDLL:
    """Load libmoe_mi355x.so (built by `python -m sparse_expert_routing_sigmoid_amd.build`)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_expert_routing_sigmoid_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, lib().moe_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.numel():
            return None
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return t.data_ptr()
    return t


# The current stream's handle without a torch.cuda.Stream object around it
# (0.1 against 2.6 us, of the 6 that a small call takes on the host), where
# torch has the two functions for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return ctypes.c_void_p(_raw_stream(_raw_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.uint8:
        return MOE_E4M3
    raise ValueError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------ sizes --
def moe_route_workspace_bytes(T, d, Nr):
    return lib().moe_route_workspace_bytes(T, d, Nr)


def moe_permute_rows(T, K, Nr, Ns, tile_m):
    return lib().moe_permute_rows(T, K, Nr, Ns, tile_m)


def moe_permute_tiles_max(T, K, Nr, Ns, tile_m):
    return lib().moe_permute_tiles_max(T, K, Nr, Ns, tile_m)


def moe_permute_workspace_bytes(T, K, Nr, Ns):
    return lib().moe_permute_workspace_bytes(T, K, Nr, Ns)


def moe_gemm_workspace_bytes(T, K, Nr, Ns, d, I, tile_m, x_t, w_t):
    return lib().moe_gemm_workspace_bytes(T, K, Nr, Ns, d, I, tile_m, x_t, w_t)


def moe_gemm_train_workspace_bytes(T, K, Nr, Ns, d, I, tile_m):
    return lib().moe_gemm_train_workspace_bytes(T, K, Nr, Ns, d, I, tile_m)


def moe_gemm_backward_workspace_bytes(T, K, Nr, Ns, d, I, tile_m):
    return lib().moe_gemm_backward_workspace_bytes(T, K, Nr, Ns, d, I, tile_m)


def _nbytes(t):
    return t.numel() * t.element_size() if t is not None else 0


# ------------------------------------------------------------ entry points --
def moe_route(u, centroids, bias, K, topk_idx, topk_gate, topk_score, expert_load, ws, stream=None):
    T, d = u.shape
    Nr = centroids.shape[0]
    _check(lib().moe_route(_ptr(u), dtype_code(u), _ptr(centroids), _ptr(bias), T, d, Nr, K,
                           _ptr(topk_idx), _ptr(topk_gate), _ptr(topk_score), _ptr(expert_load),
                           _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def moe_permute(topk_idx, Nr, Ns, tile_m, seg_offset, row_token, inv_row, tile_map, n_tiles, ws, stream=None):
    T, K = topk_idx.shape
    _check(lib().moe_permute(_ptr(topk_idx), T, K, Nr, Ns, tile_m, _ptr(seg_offset), _ptr(row_token),
                             _ptr(inv_row), _ptr(tile_map), _ptr(n_tiles), _ptr(ws),
                             ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def moe_permute_noalloc(topk_idx, Nr, Ns, tile_m, seg_offset, row_token, inv_row, tile_map, n_tiles, stream=None):
    """moe_permute with the library's own scratch array: allocates nothing."""
    T, K = topk_idx.shape
    _check(lib().moe_permute_noalloc(_ptr(topk_idx), T, K, Nr, Ns, tile_m, _ptr(seg_offset), _ptr(row_token),
                                     _ptr(inv_row), _ptr(tile_map), _ptr(n_tiles), _stream(stream)))


def moe_expert_gemm(x, x_scale, w_t, w13, w13_scale, w2, w2_scale, T, K, Nr, Ns, d, I, tile_m,
                    seg_offset, row_token, tile_map, n_tiles, ws, y, x_t=None, stream=None):
    x_t = dtype_code(x) if x_t is None else x_t
    _check(lib().moe_expert_gemm(_ptr(x), x_t, _ptr(x_scale), w_t, _ptr(w13), _ptr(w13_scale), _ptr(w2),
                                 _ptr(w2_scale), T, K, Nr, Ns, d, I, tile_m, _ptr(seg_offset), _ptr(row_token),
                                 _ptr(tile_map), _ptr(n_tiles), _ptr(ws),
                                 ws.numel() * ws.element_size() if ws is not None else 0,
                                 _ptr(y), dtype_code(y), _stream(stream)))


def moe_gemm_combine_workspace_bytes(T, K, Nr, Ns, d, I, tile_m, x_t, w_t):
    return lib().moe_gemm_combine_workspace_bytes(T, K, Nr, Ns, d, I, tile_m, x_t, w_t)


def moe_expert_gemm_combine(x, x_scale, w_t, w13, w13_scale, w2, w2_scale, T, K, Nr, Ns, d, I, tile_m, seg_offset,
                            row_token, tile_map, n_tiles, inv_row, topk_gate, u, ws, out, flags=0, x_t=None,
                            stream=None):
    """Expert GEMMs with the combine fused into the down projection (fp32
    atomics; not bitwise reproducible); out [T, d] fp32."""
    x_t = dtype_code(x) if x_t is None else x_t
    _check(lib().moe_expert_gemm_combine(_ptr(x), x_t, _ptr(x_scale), w_t, _ptr(w13), _ptr(w13_scale), _ptr(w2),
                                         _ptr(w2_scale), T, K, Nr, Ns, d, I, tile_m, _ptr(seg_offset),
                                         _ptr(row_token), _ptr(tile_map), _ptr(n_tiles), _ptr(inv_row),
                                         _ptr(topk_gate), _ptr(u), dtype_code(u), flags, _ptr(ws), _nbytes(ws),
                                         _ptr(out), _stream(stream)))


def moe_expert_gemm_train(x, w13, w2, T, K, Nr, Ns, d, I, tile_m, seg_offset, row_token, tile_map, n_tiles,
                          ws, h, ab, y, stream=None):
    _check(lib().moe_expert_gemm_train(_ptr(x), _ptr(w13), _ptr(w2), T, K, Nr, Ns, d, I, tile_m, _ptr(seg_offset),
                                       _ptr(row_token), _ptr(tile_map), _ptr(n_tiles), _ptr(ws), _nbytes(ws),
                                       _ptr(h), _ptr(ab), _ptr(y), dtype_code(y), _stream(stream)))


def moe_combine_backward(grad_out, y, inv_row, topk_gate, topk_score, seg_offset, Nr, Ns, dy, dgate, dz, dz_row,
                         stream=None):
    T, d = grad_out.shape
    K = inv_row.shape[1]
    _check(lib().moe_combine_backward(_ptr(grad_out), dtype_code(grad_out), _ptr(y), dtype_code(y), _ptr(inv_row),
                                      _ptr(topk_gate), _ptr(topk_score), _ptr(seg_offset), T, d, K, Nr, Ns, _ptr(dy),
                                      _ptr(dgate), _ptr(dz), _ptr(dz_row), _stream(stream)))


def moe_expert_gemm_backward(x, w13, w2, h, ab, dy, T, K, Nr, Ns, d, I, tile_m, seg_offset, row_token, tile_map,
                             n_tiles, ws, dx, dw13, dw2, stream=None):
    _check(lib().moe_expert_gemm_backward(_ptr(x), _ptr(w13), _ptr(w2), _ptr(h), _ptr(ab), _ptr(dy), T, K, Nr, Ns,
                                          d, I, tile_m, _ptr(seg_offset), _ptr(row_token), _ptr(tile_map),
                                          _ptr(n_tiles), _ptr(ws), _nbytes(ws), _ptr(dx), _ptr(dw13), _ptr(dw2),
                                          dtype_code(dw13), _stream(stream)))


def moe_gemm_train_w8_workspace_bytes(T, K, Nr, Ns, d, I, tile_m):
    return lib().moe_gemm_train_w8_workspace_bytes(T, K, Nr, Ns, d, I, tile_m)


def moe_expert_gemm_train_w8(xq, xs, w8: "ExpertWeights", T, K, Nr, Ns, d, I, tile_m, seg_offset, row_token,
                             tile_map, n_tiles, ws, h, ab, y, stream=None):
    """The E4M3 expert GEMMs keeping h and [a | b] (bf16) for the backward;
    xq / xs: u in 1x128 E4M3 tiles (fp8_quantize_tiles)."""
    if w8.w_t != MOE_E4M3:
        raise ValueError("moe_expert_gemm_train_w8 needs E4M3 weights")
    _check(lib().moe_expert_gemm_train_w8(_ptr(xq), _ptr(xs), _ptr(w8.w13), _ptr(w8.w13_scale), _ptr(w8.w2),
                                          _ptr(w8.w2_scale), T, K, Nr, Ns, d, I, tile_m, _ptr(seg_offset),
                                          _ptr(row_token), _ptr(tile_map), _ptr(n_tiles), _ptr(ws), _nbytes(ws),
                                          _ptr(h), _ptr(ab), _ptr(y), dtype_code(y), _stream(stream)))


def moe_gemm_backward_w8_workspace_bytes(T, K, Nr, Ns, d, I, tile_m):
    return lib().moe_gemm_backward_w8_workspace_bytes(T, K, Nr, Ns, d, I, tile_m)


def moe_expert_gemm_backward_w8(x, w8: "ExpertWeights", h, ab, dy, T, K, Nr, Ns, d, I, tile_m, seg_offset, row_token,
                                tile_map, n_tiles, ws, dx, dw13, dw2, stream=None):
    """moe_expert_gemm_backward with the input-gradient products on E4M3
    operands; w8: the E4M3 expert weights (quantize_weights)."""
    if w8.w_t != MOE_E4M3:
        raise ValueError("moe_expert_gemm_backward_w8 needs E4M3 weights")
    _check(lib().moe_expert_gemm_backward_w8(_ptr(x), _ptr(w8.w13), _ptr(w8.w13_scale), _ptr(w8.w2),
                                             _ptr(w8.w2_scale), _ptr(h), _ptr(ab), _ptr(dy), T, K, Nr, Ns, d, I,
                                             tile_m, _ptr(seg_offset), _ptr(row_token), _ptr(tile_map),
                                             _ptr(n_tiles), _ptr(ws), _nbytes(ws), _ptr(dx), _ptr(dw13), _ptr(dw2),
                                             dtype_code(dw13), _stream(stream)))


def moe_gemm_backward_f8_workspace_bytes(T, K, Nr, Ns, d, I, tile_m):
    return lib().moe_gemm_backward_f8_workspace_bytes(T, K, Nr, Ns, d, I, tile_m)


def moe_expert_gemm_backward_f8(x, w8: "ExpertWeights", h, ab, dy, T, K, Nr, Ns, d, I, tile_m, seg_offset, row_token,
                                tile_map, n_tiles, ws, dx, dw13, dw2, stream=None):
    """moe_expert_gemm_backward_w8 with the weight-gradient products on E4M3
    operands too (runs of 128 rows along the tokens)."""
    if w8.w_t != MOE_E4M3:
        raise ValueError("moe_expert_gemm_backward_f8 needs E4M3 weights")
    _check(lib().moe_expert_gemm_backward_f8(_ptr(x), _ptr(w8.w13), _ptr(w8.w13_scale), _ptr(w8.w2),
                                             _ptr(w8.w2_scale), _ptr(h), _ptr(ab), _ptr(dy), T, K, Nr, Ns, d, I,
                                             tile_m, _ptr(seg_offset), _ptr(row_token), _ptr(tile_map),
                                             _ptr(n_tiles), _ptr(ws), _nbytes(ws), _ptr(dx), _ptr(dw13), _ptr(dw2),
                                             dtype_code(dw13), _stream(stream)))


def fp8_quantize_runs_max(P, n_seg):
    return lib().fp8_quantize_runs_max(P, n_seg)


def fp8_quantize_runs(x, row_token, gather, seg_offset, P, run_offset, q, scale, stream=None):
    """E4M3 along the rows of the permuted layout: each segment of
    seg_offset in runs of 128 rows, one power-of-two scale per run and
    column.  x [P, cols], or with gather [rows, cols] read at row_token."""
    rows, cols = x.shape
    _check(lib().fp8_quantize_runs(_ptr(x), dtype_code(x), rows, cols, _ptr(row_token), int(bool(gather)),
                                   _ptr(seg_offset), seg_offset.shape[0] - 1, P, _ptr(run_offset), _ptr(q),
                                   _ptr(scale), _stream(stream)))


def moe_route_backward(grad_out, dx, u, centroids, topk_idx, inv_row, dz, dz_row, seg_offset, row_token, Nr, Ns,
                       du, de, stream=None):
    T, d = u.shape
    K = topk_idx.shape[1]
    _check(lib().moe_route_backward(_ptr(grad_out), dtype_code(grad_out), _ptr(dx), _ptr(u), dtype_code(u),
                                    _ptr(centroids), _ptr(topk_idx), _ptr(inv_row), _ptr(dz), _ptr(dz_row),
                                    _ptr(seg_offset), _ptr(row_token), T, d, K, Nr, Ns, _ptr(du), dtype_code(du),
                                    _ptr(de), _stream(stream)))


def moe_combine(u, y, inv_row, topk_gate, seg_offset, Nr, Ns, out, flags=0, stream=None):
    T, d = u.shape
    K = inv_row.shape[1]
    _check(lib().moe_combine(_ptr(u), dtype_code(u), _ptr(y), dtype_code(y), _ptr(inv_row), _ptr(topk_gate),
                             _ptr(seg_offset), T, d, K, Nr, Ns, flags, _ptr(out), dtype_code(out), _stream(stream)))


def moe_bias_update(expert_load, total_assign, gamma, bias, stream=None):
    _check(lib().moe_bias_update(_ptr(expert_load), bias.shape[0], int(total_assign), float(gamma), _ptr(bias),
                                 _stream(stream)))


def fp8_quantize_tiles(x, tile_rows, q, scale, tile_cols=128, stream=None):
    """Quantise x viewed as [rows, cols] = [numel / last dim, last dim]."""
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    _check(lib().fp8_quantize_tiles(_ptr(x), dtype_code(x), rows, cols, tile_rows, tile_cols, _ptr(q), _ptr(scale),
                                    _stream(stream)))


def fp8_dequantize_tiles(q, scale, tile_rows, out, tile_cols=128, stream=None):
    """Values of E4M3 tiles (code x tile scale) into out (fp32 or bf16), q
    viewed as [numel / last dim, last dim]."""
    cols = q.shape[-1]
    rows = q.numel() // cols if cols else 0
    _check(lib().fp8_dequantize_tiles(_ptr(q), _ptr(scale), rows, cols, tile_rows, tile_cols, _ptr(out),
                                      dtype_code(out), _stream(stream)))


def _same(t, like, name, dtype=None):
    """t has `like`'s shape (and `dtype`): a kernel reads and writes that many elements of it."""
    if t is not None and (t.shape != like.shape or (dtype is not None and t.dtype != dtype)):
        raise ValueError(f"{name}: expected {tuple(like.shape)}{'' if dtype is None else f' {dtype}'}, "
                         f"got {tuple(t.shape)} {t.dtype}")


def _shape(t, shape, dtype, name):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def moe_rmsnorm(x, weight, eps, residual=None, r_out=None, u=None, q=None, q_scale=None, rstd=None, stream=None):
    """r = x + residual, u = r (mean r^2 + eps)^(-1/2) weight, in one pass
    over the rows of x [T, d]: writes r_out (of residual's dtype, or x's), u,
    u's 1x128 E4M3 tiles q / q_scale and rstd [T], each where given."""
    T, d = x.shape
    r_t = MOE_F32
    for t, name in ((residual, "residual"), (r_out, "r_out")):
        _same(t, x, name)
        if t is not None:
            r_t = dtype_code(t)
    if residual is not None and r_out is not None and residual.dtype != r_out.dtype:
        raise ValueError("r_out must have residual's dtype")
    _shape(weight, (d,), weight.dtype, "weight")
    _same(u, x, "u")
    _same(q, x, "q", torch.uint8)
    _shape(q_scale, (T, d // 128), torch.float32, "q_scale")
    _shape(rstd, (T,), torch.float32, "rstd")
    _check(lib().moe_rmsnorm(_ptr(x), dtype_code(x), _ptr(residual), r_t, _ptr(weight), dtype_code(weight), eps, T, d,
                             _ptr(r_out), _ptr(u), MOE_F32 if u is None else dtype_code(u), _ptr(q), _ptr(q_scale),
                             _ptr(rstd), _stream(stream)))


def moe_rmsnorm_backward_workspace_bytes(T, d):
    return lib().moe_rmsnorm_backward_workspace_bytes(T, d)


def moe_rmsnorm_backward(du, r, weight, rstd, dr, dx, dw, ws, stream=None):
    """Gradients of moe_rmsnorm: dx [T, d] (of x and of the residual; dr, the
    gradient along the residual stream, is added when given) and dw [d] fp32.
    r, dr and dx share a dtype."""
    T, d = r.shape
    _same(du, r, "du")
    _same(dr, r, "dr", r.dtype)
    _same(dx, r, "dx", r.dtype)
    _shape(weight, (d,), weight.dtype, "weight")
    _shape(rstd, (T,), torch.float32, "rstd")
    _shape(dw, (d,), torch.float32, "dw")
    _check(lib().moe_rmsnorm_backward(_ptr(du), dtype_code(du), _ptr(r), dtype_code(r), _ptr(weight),
                                      dtype_code(weight), _ptr(rstd), _ptr(dr), T, d, _ptr(dx), _ptr(dw), _ptr(ws),
                                      _nbytes(ws), _stream(stream)))


def fp4_quantize_groups(x, q, scale, stream=None):
    """E2M1 codes q [..., cols / 2] (uint8, two to a byte) and exponent bytes
    scale [..., cols / 32] of x [..., cols], one power of two per 32 columns."""
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    _shape(q, (*x.shape[:-1], cols // 2), torch.uint8, "q")
    _shape(scale, (*x.shape[:-1], cols // 32), torch.uint8, "scale")
    _check(lib().fp4_quantize_groups(_ptr(x), dtype_code(x), rows, cols, _ptr(q), _ptr(scale), _stream(stream)))


def fp4_dequantize_groups(q, scale, out, stream=None):
    """Values of E2M1 groups into out [..., cols] (fp32 or bf16)."""
    cols = out.shape[-1]
    rows = out.numel() // cols if cols else 0
    _shape(q, (*out.shape[:-1], cols // 2), torch.uint8, "q")
    _shape(scale, (*out.shape[:-1], cols // 32), torch.uint8, "scale")
    _check(lib().fp4_dequantize_groups(_ptr(q), _ptr(scale), rows, cols, _ptr(out), dtype_code(out), _stream(stream)))


def fp4_matvec_workspace_bytes(T, N, K):
    return lib().fp4_matvec_workspace_bytes(T, N, K)


def fp4_matvec(x, q, scale, y, ws=None, stream=None):
    """y [T, N] = x [T, K] W^T with the 4-bit W [N, K] of (q, scale)."""
    T, K = x.shape
    N = q.shape[0]
    _shape(q, (N, K // 2), torch.uint8, "q")
    _shape(scale, (N, K // 32), torch.uint8, "scale")
    _shape(y, (T, N), y.dtype, "y")
    _check(lib().fp4_matvec(_ptr(x), dtype_code(x), _ptr(q), _ptr(scale), T, N, K, _ptr(y), dtype_code(y), _ptr(ws),
                            _nbytes(ws), _stream(stream)))


def moe_layer_few_workspace_bytes(T, d, Nr, Ns, I, K, u_t):
    return lib().moe_layer_few_workspace_bytes(T, d, Nr, Ns, I, K, u_t)


def _rows(t, T, K, dtype, name):
    """t is [at least T, K]: the call writes its first T rows."""
    if t is not None and (t.dim() != 2 or t.shape[0] < T or t.shape[1] != K or t.dtype != dtype):
        raise ValueError(f"{name}: expected at least {(T, K)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def _few_weights(w: "ExpertWeights", E, d, I):
    """w holds E experts of width I in one of moe_layer_few's weight types."""
    store = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_E4M3: torch.uint8, MOE_E2M1: torch.uint8}
    if w.w_t not in store:
        raise ValueError(f"w_t: unknown weight type {w.w_t}")
    per_byte = 2 if w.w_t == MOE_E2M1 else 1
    _shape(w.w13, (E, 2 * I, d // per_byte), store[w.w_t], "w13")
    _shape(w.w2, (E, d, I // per_byte), store[w.w_t], "w2")
    if w.w_t in (MOE_E4M3, MOE_E2M1) and (w.w13_scale is None or w.w2_scale is None):
        raise ValueError("E4M3 and E2M1 weights need scales")
    if w.w_t == MOE_E4M3:
        _shape(w.w13_scale, (E, 2 * I // 128, d // 128), torch.float32, "w13_scale")
        _shape(w.w2_scale, (E, d // 128, I // 128), torch.float32, "w2_scale")
    if w.w_t == MOE_E2M1:
        _shape(w.w13_scale, (E, 2 * I, d // 32), torch.uint8, "w13_scale")
        _shape(w.w2_scale, (E, d, I // 32), torch.uint8, "w2_scale")


def moe_layer_few(u, centroids, bias, w: "ExpertWeights", Ns, I, K, resid, topk_idx, topk_gate, topk_score, expert_load,
                  ws, out, stream=None):
    """The whole layer for up to MOE_FEW_TOKENS tokens u [T, d]; resid [T, d]
    or None is added to out [T, d].  The first T rows of topk_idx, topk_gate
    and topk_score (or None) are written."""
    T, d = u.shape
    Nr = centroids.shape[0]
    _few_weights(w, Nr + Ns, d, I)
    _shape(centroids, (Nr, d), torch.float32, "centroids")
    _shape(bias, (Nr,), torch.float32, "bias")
    _same(resid, u, "resid")
    _rows(topk_idx, T, K, torch.int32, "topk_idx")
    _rows(topk_gate, T, K, torch.float32, "topk_gate")
    _rows(topk_score, T, K, torch.float32, "topk_score")
    _shape(expert_load, (Nr,), torch.int32, "expert_load")
    _same(out, u, "out")
    _layer_few(u, centroids, bias, w, Ns, I, K, resid, topk_idx, topk_gate, topk_score, expert_load, ws, out, stream)


def _layer_few(u, centroids, bias, w, Ns, I, K, resid, topk_idx, topk_gate, topk_score, expert_load, ws, out, stream):
    T, d = u.shape
    _check(lib().moe_layer_few(_ptr(u), dtype_code(u), _ptr(centroids), _ptr(bias), w.w_t, _ptr(w.w13),
                               _ptr(w.w13_scale), _ptr(w.w2), _ptr(w.w2_scale), T, d, centroids.shape[0], Ns, I, K,
                               _ptr(resid), MOE_F32 if resid is None else dtype_code(resid), _ptr(topk_idx),
                               _ptr(topk_gate), _ptr(topk_score), _ptr(expert_load), _ptr(ws), _nbytes(ws), _ptr(out),
                               dtype_code(out), _stream(stream)))


# ------------------------------------------------------ latent attention --
def _on_gpu(*tensors):
    """Every tensor given is on the current HIP device, whose stream the call goes to."""
    dev = _raw_device() if _raw_device is not None and torch.cuda.is_initialized() else torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}: every tensor must be on the current HIP device")


def _strided_rows(t, shape, name):
    """The row stride of bf16 rows t [rows, cols] whose columns are contiguous."""
    if t.shape != shape or t.dtype != torch.bfloat16:
        raise ValueError(f"{name}: expected {tuple(shape)} torch.bfloat16, got {tuple(t.shape)} {t.dtype}")
    rows, cols = shape
    down, across = t.stride()
    if rows and cols and ((across != 1 and cols > 1) or (rows > 1 and down < cols)):
        raise ValueError(f"{name}: columns must be contiguous and rows apart")
    return down if rows > 1 else max(cols, 8)


def _float_out(t, shape, name):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name}: expected fp32 or bf16, got {t.dtype}")
    _shape(t, shape, t.dtype, name)


def mla_pages_workspace_bytes(B):
    return lib().mla_pages_workspace_bytes(B)


def mla_pages_extend(seq_len, new_len, page_size, block_table, free_pages, n_free, seq_len_out, n_free_out, n_failed,
                     cu_new, slot, position, ws=None, stream=None):
    """Pages and slots of the new_len[b] tokens that a step adds to each
    request of seq_len[b] tokens.  block_table [B, W] gets the new pages, taken
    from the top of free_pages[:n_free]; slot and position [N] hold the new
    tokens' places, request by request, and -1 behind them; cu_new [B + 1] their
    offsets.  seq_len_out and n_free_out may be seq_len and n_free.  n_failed [1]
    counts requests that found no room: their tokens have slot -1."""
    B = seq_len.shape[0]
    i32 = torch.int32
    _shape(seq_len, (B,), i32, "seq_len")
    _shape(new_len, (B,), i32, "new_len")
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [B, W]")
    _shape(block_table, (B, block_table.shape[1]), i32, "block_table")
    _shape(free_pages, (free_pages.numel(),), i32, "free_pages")
    _shape(n_free, (1,), i32, "n_free")
    _shape(seq_len_out, (B,), i32, "seq_len_out")
    _shape(n_free_out, (1,), i32, "n_free_out")
    _shape(n_failed, (1,), i32, "n_failed")
    _shape(cu_new, (B + 1,), i32, "cu_new")
    _shape(slot, (slot.numel(),), i32, "slot")
    _shape(position, (slot.numel(),), i32, "position")
    _on_gpu(seq_len, new_len, block_table, free_pages, n_free, seq_len_out, n_free_out, n_failed, cu_new, slot,
            position, ws)
    _check(lib().mla_pages_extend(_ptr(seq_len), _ptr(new_len), B, page_size, _ptr(block_table), block_table.shape[1],
                                  _ptr(free_pages), free_pages.numel(), _ptr(n_free), _ptr(seq_len_out),
                                  _ptr(n_free_out), _ptr(n_failed), _ptr(cu_new), _ptr(slot), _ptr(position),
                                  slot.numel(), _ptr(ws), _nbytes(ws), _stream(stream)))


def mla_pages_release(done, seq_len, page_size, block_table, free_pages, n_free, stream=None):
    """The pages of the requests with done[b] != 0 go back on the stack
    free_pages[:n_free], and their lengths become 0 (in place)."""
    B = seq_len.shape[0]
    i32 = torch.int32
    _shape(seq_len, (B,), i32, "seq_len")
    _shape(done, (B,), i32, "done")
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [B, W]")
    _shape(block_table, (B, block_table.shape[1]), i32, "block_table")
    _shape(free_pages, (free_pages.numel(),), i32, "free_pages")
    _shape(n_free, (1,), i32, "n_free")
    _on_gpu(done, seq_len, block_table, free_pages, n_free)
    _check(lib().mla_pages_release(_ptr(done), _ptr(seq_len), B, page_size, _ptr(block_table), block_table.shape[1],
                                   _ptr(free_pages), free_pages.numel(), _ptr(n_free), _stream(stream)))


def mla_cache_write(latent, k_rope, slot, cache, stream=None):
    """Rows slot[t] of cache [..., dc + dr] become [latent[t], k_rope[t]]
    (bf16); tokens whose slot lies outside the cache are not written.  latent
    [T, dc] and k_rope [T, dr] may be column ranges of wider rows."""
    if latent.dim() != 2 or k_rope.dim() != 2:
        raise ValueError("latent and k_rope: expected [T, dc] and [T, dr]")
    T, dc, dr = latent.shape[0], latent.shape[1], k_rope.shape[1]
    ldc, ldr = _strided_rows(latent, (T, dc), "latent"), _strided_rows(k_rope, (T, dr), "k_rope")
    _shape(slot, (T,), torch.int32, "slot")
    if cache.dtype != torch.bfloat16 or cache.dim() < 2 or cache.shape[-1] != dc + dr:
        raise ValueError(f"cache: expected [..., {dc + dr}] bf16, got {tuple(cache.shape)} {cache.dtype}")
    _on_gpu(latent, k_rope, slot, cache)
    _check(lib().mla_cache_write(latent.data_ptr(), ldc, k_rope.data_ptr(), ldr, _ptr(slot), T, dc, dr, _ptr(cache),
                                 cache.numel() // (dc + dr), _stream(stream)))


def mla_decode_workspace_bytes(B, S, H, dn, dr, dv, dc, max_len):
    return lib().mla_decode_workspace_bytes(B, S, H, dn, dr, dv, dc, max_len)


def mla_decode(q, w_kv, cache, block_table, seq_len, S, max_len, scale, out, ws, stream=None):
    """Attention of the newest S tokens of each request over the paged cache
    [n_pages, page_size, dc + dr]: q [B S, H, dn + dr] -> out [B S, H, dv], with
    w_kv [H, dn + dv, dc] the projection of a latent to each head's key and
    value.  seq_len [B] counts the S tokens.  max_len: a bound on seq_len, by
    which the work is divided and ws is sized (mla_decode_workspace_bytes)."""
    if q.dim() != 3 or w_kv.dim() != 3 or cache.dim() != 3 or out.dim() != 3 or block_table.dim() != 2:
        raise ValueError("expected q [B S, H, dn + dr], w_kv [H, dn + dv, dc], cache [n_pages, page_size, dc + dr], "
                         "block_table [B, W] and out [B S, H, dv]")
    N, H, dqk = q.shape
    n_pages, page_size, width = cache.shape
    B, dv, dc = seq_len.shape[0], out.shape[2], w_kv.shape[2]
    dr = width - dc
    dn = dqk - dr
    bf16 = torch.bfloat16
    _shape(q, (B * S, H, dqk), bf16, "q")
    _shape(w_kv, (H, dn + dv, dc), bf16, "w_kv")
    _shape(cache, (n_pages, page_size, width), bf16, "cache")
    _shape(block_table, (B, block_table.shape[1]), torch.int32, "block_table")
    _shape(seq_len, (B,), torch.int32, "seq_len")
    _float_out(out, (N, H, dv), "out")
    _on_gpu(q, w_kv, cache, block_table, seq_len, out, ws)
    _check(lib().mla_decode(_ptr(q), _ptr(w_kv), _ptr(cache), n_pages, page_size, _ptr(block_table),
                            block_table.shape[1], _ptr(seq_len), B, S, H, dn, dr, dv, dc, max_len, scale, _ptr(out),
                            dtype_code(out), _ptr(ws), _nbytes(ws), _stream(stream)))


def _attention_shapes(q, kv, k_rope, cu_q, cu_k, out, lse):
    if q.dim() != 3 or kv.dim() != 3 or k_rope.dim() != 2 or out.dim() != 3 or cu_q.dim() != 1:
        raise ValueError("expected q [Tq, H, dn + dr], kv [Tk, H, dn + dv], k_rope [Tk, dr], out [Tq, H, dv] and "
                         "cu_q [B + 1]")
    Tq, H, dqk = q.shape
    Tk, dr, dv = kv.shape[0], k_rope.shape[1], out.shape[2]
    dn = dqk - dr
    B = cu_q.shape[0] - 1
    if B < 0:
        raise ValueError("cu_q: expected [B + 1]")
    bf16 = torch.bfloat16
    _shape(q, (Tq, H, dqk), bf16, "q")
    _shape(kv, (Tk, H, dn + dv), bf16, "kv")
    ldr = _strided_rows(k_rope, (Tk, dr), "k_rope")
    _shape(cu_q, (B + 1,), torch.int32, "cu_q")
    _shape(cu_k, (B + 1,), torch.int32, "cu_k")
    _float_out(out, (Tq, H, dv), "out")
    _shape(lse, (Tq, H), torch.float32, "lse")
    return B, Tq, Tk, H, dn, dr, dv, ldr


def mla_attention(q, kv, k_rope, cu_q, cu_k, causal, scale, out, lse=None, stream=None):
    """Attention over packed sequences: q [Tq, H, dn + dr] against the keys and
    values kv [Tk, H, dn + dv] and the rotary key k_rope [Tk, dr] that the heads
    share -> out [Tq, H, dv], and lse [Tq, H] (fp32) for the backward.  Sequence b
    has rows cu_q[b] .. cu_q[b + 1] - 1 and cu_k[b] .. cu_k[b + 1] - 1; causal:
    its last query sees all its keys."""
    B, Tq, Tk, H, dn, dr, dv, ldr = _attention_shapes(q, kv, k_rope, cu_q, cu_k, out, lse)
    _on_gpu(q, kv, k_rope, cu_q, cu_k, out, lse)
    _check(lib().mla_attention(_ptr(q), _ptr(kv), k_rope.data_ptr(), ldr, _ptr(cu_q), _ptr(cu_k), B, Tq, Tk, H, dn, dr,
                               dv, int(bool(causal)), scale, _ptr(out), dtype_code(out), _ptr(lse), _stream(stream)))


def mla_attention_backward_workspace_bytes(Tq, Tk, H, dr):
    return lib().mla_attention_backward_workspace_bytes(Tq, Tk, H, dr)


def mla_attention_backward(dout, q, kv, k_rope, out, lse, cu_q, cu_k, causal, scale, dq, dkv, dk_rope, ws, stream=None):
    """Gradients of mla_attention for dL/dout = dout (bf16): dq, dkv and
    dk_rope, of one dtype (fp32 or bf16), with out and lse as the forward left
    them.  dk_rope [Tk, dr] is summed over the heads."""
    B, Tq, Tk, H, dn, dr, dv, ldr = _attention_shapes(q, kv, k_rope, cu_q, cu_k, out, lse)
    if lse is None:
        raise ValueError("the backward needs the forward's lse")
    _shape(dout, (Tq, H, dv), torch.bfloat16, "dout")
    _float_out(dq, q.shape, "dq")
    _shape(dkv, kv.shape, dq.dtype, "dkv")
    _shape(dk_rope, (Tk, dr), dq.dtype, "dk_rope")
    _on_gpu(dout, q, kv, k_rope, out, lse, cu_q, cu_k, dq, dkv, dk_rope, ws)
    _check(lib().mla_attention_backward(_ptr(dout), _ptr(q), _ptr(kv), k_rope.data_ptr(), ldr, _ptr(out),
                                        dtype_code(out), _ptr(lse), _ptr(cu_q), _ptr(cu_k), B, Tq, Tk, H, dn, dr, dv,
                                        int(bool(causal)), scale, _ptr(dq), _ptr(dkv), _ptr(dk_rope), dtype_code(dq),
                                        _ptr(ws), _nbytes(ws), _stream(stream)))


# ------------------------------------------------------- layer plumbing --
@dataclass
class ExpertWeights:
    """Expert weights as the library reads them: W13 [E, 2I, d], W2 [E, d, I]
    (bf16/fp32 tensors, E4M3 codes (uint8) with fp32 block scales, or E2M1
    codes two to a byte (uint8) with an exponent byte (uint8) per 32 columns)."""
    w_t: int
    w13: torch.Tensor
    w2: torch.Tensor
    w13_scale: torch.Tensor | None = None
    w2_scale: torch.Tensor | None = None


def quantize_weights(w13: torch.Tensor, w2: torch.Tensor, stream=None) -> ExpertWeights:
    """E4M3 codes + 128x128 block scales of fp32/bf16 expert weights, made by
    fp8_quantize_tiles (one 128x128 block per scale)."""
    E, twoI, d = w13.shape
    I = w2.shape[2]
    q13 = torch.empty((E, twoI, d), dtype=torch.uint8, device=w13.device)
    s13 = torch.empty((E, twoI // 128, d // 128), dtype=torch.float32, device=w13.device)
    q2 = torch.empty((E, d, I), dtype=torch.uint8, device=w2.device)
    s2 = torch.empty((E, d // 128, I // 128), dtype=torch.float32, device=w2.device)
    fp8_quantize_tiles(w13, 128, q13, s13, stream=stream)
    fp8_quantize_tiles(w2, 128, q2, s2, stream=stream)
    return ExpertWeights(MOE_E4M3, q13, q2, s13, s2)


def quantize_weights_fp4(w13: torch.Tensor, w2: torch.Tensor, stream=None) -> ExpertWeights:
    """E2M1 codes and exponent bytes of fp32/bf16 expert weights, made by
    fp4_quantize_groups (for FewTokenLayer)."""
    def one(w):
        q = torch.empty((*w.shape[:-1], w.shape[-1] // 2), dtype=torch.uint8, device=w.device)
        s = torch.empty((*w.shape[:-1], w.shape[-1] // 32), dtype=torch.uint8, device=w.device)
        fp4_quantize_groups(w, q, s, stream)
        return q, s

    (q13, s13), (q2, s2) = one(w13), one(w2)
    return ExpertWeights(MOE_E2M1, q13, q2, s13, s2)


class FewTokenLayer:
    """One DeepSeekMoE layer forward for at most T <= MOE_FEW_TOKENS tokens
    (moe_layer_few): the serving form of MoeLayer for a few sequences or
    drafted tokens, with fp32, bf16, E4M3 or E2M1 expert weights.

    Holds the outputs and the workspace; calls on it must not overlap.  After
    forward() of n tokens, the first n rows of topk_idx, topk_gate, topk_score
    and out, and expert_load, are those of the call."""

    def __init__(self, T, d, Nr, Ns, I, K, act_dtype, weights: ExpertWeights, out_dtype=None, device="cuda"):
        self.T, self.d, self.Nr, self.Ns, self.I, self.K = T, d, Nr, Ns, I, K
        self.act_dtype, self.w = act_dtype, weights
        if not 0 <= T <= MOE_FEW_TOKENS:
            raise ValueError(f"T: at most {MOE_FEW_TOKENS} tokens")
        _few_weights(weights, Nr + Ns, d, I)
        dev = torch.device(device)
        self.topk_idx = torch.empty((T, K), dtype=torch.int32, device=dev)
        self.topk_gate = torch.empty((T, K), dtype=torch.float32, device=dev)
        self.topk_score = torch.empty((T, K), dtype=torch.float32, device=dev)
        self.expert_load = torch.empty((Nr,), dtype=torch.int32, device=dev)
        self.out = torch.empty((T, d), dtype=act_dtype if out_dtype is None else out_dtype, device=dev)
        u_t = MOE_BF16 if act_dtype == torch.bfloat16 else MOE_F32
        self.ws = torch.empty((max(moe_layer_few_workspace_bytes(T, d, Nr, Ns, I, K, u_t), 1),), dtype=torch.uint8,
                              device=dev)
        self.tokens = T  # of the last forward()

    def forward(self, u, centroids, bias, residual=None, flags=0, stream=None):
        """out [n, d] = residual + the experts' part for u [n, d], n <= T.
        residual None is u, as in the combine equation (a pre-norm block
        passes its stream); MOE_COMBINE_NO_RESIDUAL in flags adds nothing."""
        n = u.shape[0]
        if n > self.T or u.shape[1] != self.d or u.dtype != self.act_dtype:
            raise ValueError(f"u: expected at most [{self.T}, {self.d}] {self.act_dtype}, got {tuple(u.shape)} {u.dtype}")
        if flags & ~MOE_COMBINE_NO_RESIDUAL:
            raise ValueError("flags: only MOE_COMBINE_NO_RESIDUAL")
        _same(residual, u, "residual")
        _shape(centroids, (self.Nr, self.d), torch.float32, "centroids")
        _shape(bias, (self.Nr,), torch.float32, "bias")
        resid = None if flags else u if residual is None else residual
        out = self.out if n == self.T else self.out[:n]
        _layer_few(u, centroids, bias, self.w, self.Ns, self.I, self.K, resid, self.topk_idx, self.topk_gate,
                   self.topk_score, self.expert_load, self.ws, out, stream)
        self.tokens = n
        return out

    def update_bias(self, bias, tokens=None, gamma=0.001, stream=None):
        """End-of-step bias rule for the loads of the last call: by default
        forward()'s, of as many tokens as it had (the replay of a captured
        call is none: give its `tokens` where they may differ)."""
        moe_bias_update(self.expert_load, (self.tokens if tokens is None else tokens) * self.K, gamma, bias, stream)


class LatentCache:
    """The paged latent cache of up to B requests in `layers` layers, and latent
    attention over it: mla_pages_extend -> mla_cache_write -> mla_decode, and
    mla_pages_release when requests end.

    Holds the cache [layers, n_pages, page_size, dc + dr] (bf16), the block
    table, the lengths and the stack of free pages, all on the device, and the
    workspaces; calls on it must not overlap.  One extend() serves all layers of
    a step.  A captured step follows the lengths at its replays, with the number
    of rows that it was captured with (rows without a token have slot -1).

    H, dn, dv: the heads and their sizes, S: the most new tokens of a request in
    a decode() call, max_len: the longest request, max_tokens: the most rows of a
    step."""

    def __init__(self, n_pages, page_size, B, max_len, max_tokens, H, dn, dr, dv, dc, S=1, layers=1, device="cuda"):
        self.page_size, self.B, self.S, self.max_tokens = page_size, B, S, max_tokens
        self.H, self.dn, self.dr, self.dv, self.dc = H, dn, dr, dv, dc
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        width = max(-(-max_len // page_size), 1)
        self.max_len = width * page_size
        self.cache = torch.zeros((layers, n_pages, page_size, dc + dr), dtype=torch.bfloat16, device=dev)
        self.block_table = torch.zeros((B, width), **i32)
        self.seq_len = torch.zeros((B,), **i32)
        self.free_pages = torch.arange(n_pages - 1, -1, -1, **i32)
        self.n_free = torch.full((1,), n_pages, **i32)
        self.n_failed = torch.zeros((1,), **i32)
        self.cu_new = torch.zeros((B + 1,), **i32)
        self.slot, self.position = (torch.full((max_tokens,), -1, **i32) for _ in range(2))
        self.rows = 0                                              # of the last extend(): slots behind are older ones
        self.pages_ws = torch.empty((max(mla_pages_workspace_bytes(B), 1),), dtype=torch.uint8, device=dev)
        need = [mla_decode_workspace_bytes(B, i, H, dn, dr, dv, dc, self.max_len) for i in range(1, S + 1)]
        self.ws = torch.empty((max(need + [1]),), dtype=torch.uint8, device=dev)

    def extend(self, new_len, tokens=None, stream=None):
        """Pages and slots for new_len[b] (device int32 [B]) more tokens of each
        request, in `tokens` rows (max_tokens by default): returns (slot,
        position) of the rows.  Requests that found no room keep their length,
        and n_failed counts them."""
        tokens = self.max_tokens if tokens is None else tokens
        if not 0 <= tokens <= self.max_tokens:
            raise ValueError(f"tokens: at most {self.max_tokens}")
        slot, position = self.slot[:tokens], self.position[:tokens]
        mla_pages_extend(self.seq_len, new_len, self.page_size, self.block_table, self.free_pages, self.n_free,
                         self.seq_len, self.n_free, self.n_failed, self.cu_new, slot, position, self.pages_ws, stream)
        self.rows = tokens
        return slot, position

    def write(self, latent, k_rope, layer=0, stream=None):
        """Rows of the last extend() (the replay of a captured call is none)
        into a layer's cache: latent [n, dc], k_rope [n, dr], n at most its `tokens`."""
        n = latent.shape[0]
        if n > self.rows:
            raise ValueError(f"latent: {n} rows, of which the last extend() placed {self.rows}")
        mla_cache_write(latent, k_rope, self.slot[:n], self.cache[layer], stream)

    def decode(self, q, w_kv, scale, out, S=1, layer=0, stream=None):
        """Attention of the newest S tokens of each request: q [B S, H, dn + dr]
        -> out [B S, H, dv].  The rows of a request without tokens are zeros."""
        if not 1 <= S <= self.S:
            raise ValueError(f"S: at most {self.S}")
        if q.shape != (self.B * S, self.H, self.dn + self.dr) or w_kv.shape != (self.H, self.dn + self.dv, self.dc):
            raise ValueError(f"q {tuple(q.shape)} or w_kv {tuple(w_kv.shape)} does not fit the cache's sizes")
        mla_decode(q, w_kv, self.cache[layer], self.block_table, self.seq_len, S, self.max_len, scale, out, self.ws,
                   stream)
        return out

    def release(self, done, stream=None):
        """The pages of the requests with done[b] != 0 (device int32 [B]) are free again."""
        mla_pages_release(done, self.seq_len, self.page_size, self.block_table, self.free_pages, self.n_free, stream)


class MoeLayer:
    """Buffers and call order of one DeepSeekMoE layer forward.

    Allocates every output and workspace once (torch, on `device`) and runs
    moe_route -> moe_permute -> [fp8_quantize_tiles] -> moe_expert_gemm ->
    moe_combine, then moe_bias_update when a step ends.  No host
    synchronisation happens inside forward()."""

    def __init__(self, T, d, Nr, Ns, I, K, act_dtype, weights: ExpertWeights, x_fp8=False,
                 tile_m=32, out_dtype=None, device="cuda", train=False, grad_dtype=None, dgrad_weights=None,
                 fused_combine=False, wgrad_fp8=None):
        self.T, self.d, self.Nr, self.Ns, self.I, self.K = T, d, Nr, Ns, I, K
        self.tile_m, self.x_fp8, self.w = tile_m, x_fp8, weights
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        P = moe_permute_rows(T, K, Nr, Ns, tile_m)
        tiles = moe_permute_tiles_max(T, K, Nr, Ns, tile_m)
        self.P_max, self.tiles_max = P, tiles
        self.topk_idx = torch.empty((T, K), **i32)
        self.topk_gate = torch.empty((T, K), **f32)
        self.topk_score = torch.empty((T, K), **f32)
        self.expert_load = torch.empty((Nr,), **i32)
        self.route_ws = torch.empty((max(moe_route_workspace_bytes(T, d, Nr), 1),), dtype=torch.uint8, device=dev)
        self.seg_offset = torch.empty((Nr + Ns + 1,), **i32)
        self.row_token = torch.empty((P,), **i32)
        self.inv_row = torch.empty((T, K), **i32)
        self.tile_map = torch.empty((tiles, 4), **i32)
        self.n_tiles = torch.empty((1,), **i32)
        self.perm_ws = torch.empty((max(moe_permute_workspace_bytes(T, K, Nr, Ns), 1),), dtype=torch.uint8,
                                   device=dev)
        self.x_t = MOE_E4M3 if x_fp8 else (MOE_BF16 if act_dtype == torch.bfloat16 else MOE_F32)
        if x_fp8:
            self.xq = torch.empty((T, d), dtype=torch.uint8, device=dev)
            self.xs = torch.empty((T, d // 128), **f32)
        self.gemm_ws = torch.empty((max(moe_gemm_workspace_bytes(T, K, Nr, Ns, d, I, tile_m, self.x_t,
                                                                  weights.w_t), 1),),
                                   dtype=torch.uint8, device=dev)
        out_dtype = act_dtype if out_dtype is None else out_dtype
        self.fused = fused_combine
        if fused_combine:
            # moe_expert_gemm_combine: no y rows; the output is fp32
            self.fc_ws = torch.empty((max(moe_gemm_combine_workspace_bytes(T, K, Nr, Ns, d, I, tile_m, self.x_t,
                                                                           weights.w_t), 1),),
                                     dtype=torch.uint8, device=dev)
            self.out = torch.empty((T, d), dtype=torch.float32, device=dev)
        else:
            self.y = torch.empty((P, d), dtype=out_dtype, device=dev)
            self.out = torch.empty((T, d), dtype=out_dtype, device=dev)
        self.train = train
        if train:
            # the training forward keeps h and the pre-activations [a | b]
            # for the backward: bf16 activations with bf16 weights, or the
            # E4M3 path (x_fp8 with E4M3 weights, which the backward's
            # input-gradient products then use too)
            self.train_fp8 = x_fp8 and weights.w_t == MOE_E4M3
            if act_dtype != torch.bfloat16 or not (self.train_fp8 or (not x_fp8 and weights.w_t == MOE_BF16)):
                raise ValueError("training needs bf16 activations with bf16 weights, or x_fp8 with E4M3 weights")
            if self.train_fp8:
                if dgrad_weights is not None and dgrad_weights is not weights:
                    raise ValueError("the E4M3 training path uses its own weights for the backward")
                dgrad_weights = weights
            bf16 = dict(dtype=torch.bfloat16, device=dev)
            E = Nr + Ns
            self.h = torch.empty((P, I), **bf16)
            self.ab = torch.empty((P, 2 * I), **bf16)
            tws = moe_gemm_train_w8_workspace_bytes if self.train_fp8 else moe_gemm_train_workspace_bytes
            self.train_ws = torch.empty((max(tws(T, K, Nr, Ns, d, I, tile_m), 1),), dtype=torch.uint8, device=dev)
            gd = (torch.bfloat16 if self.train_fp8 else weights.w13.dtype) if grad_dtype is None else grad_dtype
            self.dy = torch.empty((P, d), **bf16)
            self.dx = torch.empty((P, d), **bf16)
            self.dgate = torch.empty((T, K), **f32)
            self.dz = torch.empty((T, K), **f32)
            self.dz_row = torch.empty((P,), **f32)
            # dgrad_weights: E4M3 copies of the weights (quantize_weights); the
            # backward then runs its input-gradient products on E4M3 operands
            self.dgrad_w = dgrad_weights
            # the E4M3 step's gate/up weight gradient takes Q(u), the operand
            # its forward multiplied (straight-through quantisers)
            self.xdq = torch.empty((T, d), **bf16) if self.train_fp8 else None
            if dgrad_weights is not None and dgrad_weights.w_t != MOE_E4M3:
                raise ValueError("dgrad_weights must be E4M3 weights")
            # wgrad_fp8: the weight gradients on E4M3 operands too
            # (moe_expert_gemm_backward_f8); the E4M3 training step's default
            self.wgrad_fp8 = self.train_fp8 if wgrad_fp8 is None else bool(wgrad_fp8)
            if self.wgrad_fp8 and not self.train_fp8:
                raise ValueError("wgrad_fp8 needs the E4M3 training path (x_fp8 with E4M3 weights)")
            if dgrad_weights is None:
                ws_fn = moe_gemm_backward_workspace_bytes
            else:
                ws_fn = moe_gemm_backward_f8_workspace_bytes if self.wgrad_fp8 else moe_gemm_backward_w8_workspace_bytes
            self.bwd_ws = torch.empty((max(ws_fn(T, K, Nr, Ns, d, I, tile_m), 1),), dtype=torch.uint8, device=dev)
            self.dw13 = torch.empty((E, 2 * I, d), dtype=gd, device=dev)
            self.dw2 = torch.empty((E, d, I), dtype=gd, device=dev)
            self.du = torch.empty((T, d), dtype=act_dtype, device=dev)
            self.de = torch.empty((Nr, d), **f32)

    def route(self, u, centroids, bias, stream=None):
        moe_route(u, centroids, bias, self.K, self.topk_idx, self.topk_gate, self.topk_score, self.expert_load,
                  self.route_ws, stream)

    def permute(self, stream=None):
        moe_permute(self.topk_idx, self.Nr, self.Ns, self.tile_m, self.seg_offset, self.row_token, self.inv_row,
                    self.tile_map, self.n_tiles, self.perm_ws, stream)

    def experts(self, u, stream=None, tiles_ready=False):
        w = self.w
        if self.x_fp8:
            if not tiles_ready:
                fp8_quantize_tiles(u, 1, self.xq, self.xs, stream=stream)
            x, xs = self.xq, self.xs
        else:
            x, xs = u, None
        if self.train:
            if self.train_fp8:
                moe_expert_gemm_train_w8(x, xs, w, self.T, self.K, self.Nr, self.Ns, self.d, self.I, self.tile_m,
                                         self.seg_offset, self.row_token, self.tile_map, self.n_tiles, self.train_ws,
                                         self.h, self.ab, self.y, stream)
            else:
                moe_expert_gemm_train(u, w.w13, w.w2, self.T, self.K, self.Nr, self.Ns, self.d, self.I, self.tile_m,
                                      self.seg_offset, self.row_token, self.tile_map, self.n_tiles, self.train_ws,
                                      self.h, self.ab, self.y, stream)
            return
        moe_expert_gemm(x, xs, w.w_t, w.w13, w.w13_scale, w.w2, w.w2_scale, self.T, self.K, self.Nr, self.Ns,
                        self.d, self.I, self.tile_m, self.seg_offset, self.row_token, self.tile_map, self.n_tiles,
                        self.gemm_ws, self.y, x_t=self.x_t, stream=stream)

    def combine(self, u, flags=0, out=None, stream=None):
        out = self.out if out is None else out
        moe_combine(u, self.y, self.inv_row, self.topk_gate, self.seg_offset, self.Nr, self.Ns, out, flags, stream)
        return out

    def experts_combine(self, u, flags=0, stream=None, tiles_ready=False):
        """Expert GEMMs with the combine fused into the down projection
        (moe_expert_gemm_combine); returns the fp32 layer output."""
        w = self.w
        if self.x_fp8:
            if not tiles_ready:
                fp8_quantize_tiles(u, 1, self.xq, self.xs, stream=stream)
            x, xs = self.xq, self.xs
        else:
            x, xs = u, None
        moe_expert_gemm_combine(x, xs, w.w_t, w.w13, w.w13_scale, w.w2, w.w2_scale, self.T, self.K, self.Nr, self.Ns,
                                self.d, self.I, self.tile_m, self.seg_offset, self.row_token, self.tile_map,
                                self.n_tiles, self.inv_row, self.topk_gate, u, self.fc_ws, self.out, flags,
                                x_t=self.x_t, stream=stream)
        return self.out

    def forward(self, u, centroids, bias, stream=None, tiles_ready=False):
        """tiles_ready (E4M3 activations): u's 1x128 tiles are in self.xq /
        self.xs already, written by moe_rmsnorm with u."""
        if tiles_ready and not self.x_fp8:
            raise ValueError("tiles_ready needs a layer with E4M3 activations (x_fp8)")
        self.route(u, centroids, bias, stream)
        self.permute(stream)
        if self.fused:
            return self.experts_combine(u, stream=stream, tiles_ready=tiles_ready)
        self.experts(u, stream, tiles_ready)
        return self.combine(u, stream=stream)

    def backward(self, grad_out, u, centroids, stream=None):
        """Gradients of the last training forward for dL/dh' = grad_out:
        returns (du, de, dW13, dW2); the bias gets none."""
        if not self.train:
            raise RuntimeError("backward needs a layer built with train=True")
        w = self.w
        moe_combine_backward(grad_out, self.y, self.inv_row, self.topk_gate, self.topk_score, self.seg_offset,
                             self.Nr, self.Ns, self.dy, self.dgate, self.dz, self.dz_row, stream)
        if self.dgrad_w is None:
            moe_expert_gemm_backward(u, w.w13, w.w2, self.h, self.ab, self.dy, self.T, self.K, self.Nr, self.Ns,
                                     self.d, self.I, self.tile_m, self.seg_offset, self.row_token, self.tile_map,
                                     self.n_tiles, self.bwd_ws, self.dx, self.dw13, self.dw2, stream)
        else:
            x = u
            if self.train_fp8:
                fp8_dequantize_tiles(self.xq, self.xs, 1, self.xdq, stream=stream)
                x = self.xdq
            bwd = moe_expert_gemm_backward_f8 if self.wgrad_fp8 else moe_expert_gemm_backward_w8
            bwd(x, self.dgrad_w, self.h, self.ab, self.dy, self.T, self.K, self.Nr, self.Ns, self.d, self.I,
                self.tile_m, self.seg_offset, self.row_token, self.tile_map, self.n_tiles, self.bwd_ws, self.dx,
                self.dw13, self.dw2, stream)
        moe_route_backward(grad_out, self.dx, u, centroids, self.topk_idx, self.inv_row, self.dz, self.dz_row,
                           self.seg_offset, self.row_token, self.Nr, self.Ns, self.du, self.de, stream)
        return self.du, self.de, self.dw13, self.dw2

    def update_bias(self, bias, gamma=0.001, stream=None):
        moe_bias_update(self.expert_load, self.T * self.K, gamma, bias, stream)


def moe_forward(u, centroids, bias, weights: ExpertWeights, K, Ns, update_bias=False, gamma=0.001, x_fp8=False,
                tile_m=32, out_dtype=None, stream=None):
    """One DeepSeekMoE layer forward in a single call: route, permute,
    [quantise u], expert GEMMs, combine, and optionally the end-of-step bias
    rule (the bias tensor is updated in place).  Allocates the layer's
    buffers on every call (MoeLayer keeps them across steps).  Returns
    (out, layer): the layer holds the routing, loads and layout of the call.

    u [T, d] (fp32/bf16), centroids [N_r, d] fp32, bias [N_r] fp32,
    weights: ExpertWeights of the N_r routed + Ns shared experts."""
    T, d = u.shape
    Nr = centroids.shape[0]
    I = weights.w2.shape[2]
    layer = MoeLayer(T, d, Nr, Ns, I, K, u.dtype, weights, x_fp8=x_fp8, tile_m=tile_m, out_dtype=out_dtype,
                     device=u.device)
    out = layer.forward(u, centroids, bias, stream)
    if update_bias:
        layer.update_bias(bias, gamma, stream)
    return out, layer
