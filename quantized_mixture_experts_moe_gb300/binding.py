"""Thin ctypes binding over libqmoe.so (declared in include/qmoe.h).

Argument marshalling only: every function passes device pointers of torch
tensors, the sizes and the current CUDA stream to the C entry point of the
same name and raises QmoeError on a non-zero status.  There is no fallback:
when the CUDA library is missing or fails to load, every call raises.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmoe.so")

SCHEME_ID = {"w4a16": 0, "mxfp4": 1, "w8a8": 2, "w4a8": 3}
DEV_BAD_EXPERT_ID = 1
DEV_WAIT_TIMEOUT = 2


class QmoeError(RuntimeError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("k", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32)]


class TileRule(ctypes.Structure):
    """qmoe_tile_rule: dims with these H, I, E, k (0 = any) and t_min <= T <= t_max use token tile nmax."""
    _fields_ = [("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("t_min", ctypes.c_int64), ("t_max", ctypes.c_int64), ("nmax", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Fp8Mat(ctypes.Structure):
    """qmoe_fp8_mat: E4M3 codes with row stride ld; the scale of (row r, block b) is s[(r // s_rows) * s_row + b * s_blk]."""
    _fields_ = [("q", ctypes.c_void_p), ("ld", ctypes.c_int64), ("s", ctypes.c_void_p), ("s_row", ctypes.c_int64),
                ("s_blk", ctypes.c_int64), ("s_rows", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_DP = ctypes.POINTER(Dims)
_MP = ctypes.POINTER(Fp8Mat)

# name -> (argtypes, restype)
SIGNATURES = {
    "qmoe_status_str": ([_i32], ctypes.c_char_p),
    "qmoe_version": ([], ctypes.c_char_p),
    "qmoe_workspace_bytes": ([_DP], _sz),
    "qmoe_align_sort": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_align_sort_static_scratch": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "qmoe_quant_act_mxfp8": ([_i64, _i64, _vp, _vp, _vp, _vp], _i32),
    "qmoe_quant_rows_int8_bf16": ([_i64, _i64, _vp, _vp, _vp, _vp], _i32),
    "qmoe_quant_rows_int8_f32": ([_i64, _i64, _vp, _vp, _vp, _vp], _i32),
    "qmoe_mx_scales_packed_bytes": ([_i64, _i64], _sz),
    "qmoe_fp4_weights_packed_bytes": ([_i64, _i64], _sz),
    "qmoe_prepack_fp4_weights": ([_i64, _i64, _vp, _vp, _vp], _i32),
    "qmoe_prepack_mx_scales": ([_i64, _i64, _vp, _vp, _vp], _i32),
    "qmoe_int4_weights_packed_bytes": ([_i64, _i64], _sz),
    "qmoe_prepack_int4_weights": ([_i64, _i64, _vp, _vp, _vp, _vp], _i32),
    "qmoe_w4a16_x_tiles_bytes": ([_DP], _sz),
    "qmoe_w4a16_h_tiles_bytes": ([_DP], _sz),
    "qmoe_w4a16_h16_tiles_bytes": ([_DP], _sz),
    "qmoe_w4a16_h_to_f16": ([_DP, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_permute_x_f16": ([_DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm1_swiglu_w4a16": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_mx_tiles_bytes": ([_DP, _i64], _sz),
    "qmoe_permute_quant_mxfp8": ([_DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm1_swiglu_mxfp4": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm1_swiglu_mxfp4_gather": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_mx_layer_gathers": ([_DP], _i32),
    "qmoe_forward_launches": ([_DP, _i32], _i32),
    "qmoe_w8a8_tiles_bytes": ([_DP, _i64], _sz),
    "qmoe_permute_quant_int8": ([_DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_quant_tiles_int8_f32": ([_DP, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm1_swiglu_w8a8": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm2_w4a16": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm2_mxfp4": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm2_w8a8": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_set_tile_rules": ([ctypes.POINTER(TileRule), _i32], _i32),
    "qmoe_tile_nmax": ([_DP], _i32),
    "qmoe_gemm1_swiglu_w4a8": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_gemm2_w4a8": ([_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmoe_combine": ([_DP, _vp, _vp, _vp, _vp, _vp], _i32),
    "qmoe_forward_workspace_bytes": ([_DP, _i32], _sz),
    "qmoe_norm_pre": ([_i64, _i64, _i32, _i32, _vp, _i64, _vp, _f32, _vp, _i64, _vp, _vp], _i32),
    "qmoe_norm_post": ([_i64, _i64, _i32, _i32, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _f32, _vp, _f32, _vp, _i64,
                        _vp, _i64, _vp, _vp, _vp], _i32),
    "qmoe_norm_bwd_workspace_bytes": ([_i64, _i64], _sz),
    "qmoe_norm_pre_backward": ([_i64, _i64, _i32, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp,
                                _sz, _vp], _i32),
    "qmoe_norm_post_backward": ([_i64, _i64, _i32, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _vp, _i64, _f32, _vp,
                                 _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _sz, _vp],
                                _i32),
    "qmoe_route_workspace_bytes": ([_i64, _i32], _sz),
    "qmoe_route_topk": ([_i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp,
                         _sz, _vp], _i32),
    "qmoe_route_topk_backward": ([_i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i32, _f32, _vp, _f32, _vp, _vp, _vp,
                                  _i64, _vp], _i32),
    "qmoe_fp8_quant_rows": ([_i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp], _i32),
    "qmoe_fp8_quant_cols": ([_i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp], _i32),
    "qmoe_fp8_quant_blocks": ([_i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp], _i32),
    "qmoe_fp8_matmul": ([_i64, _i64, _i64, _MP, _MP, _vp, _i32, _i64, _vp, _vp], _i32),
    "qmoe_fp8_linear_workspace_bytes": ([_i64, _i64], _sz),
    "qmoe_fp8_linear": ([_i64, _i64, _i64, _i32, _vp, _i64, _MP, _vp, _i32, _i64, _vp, _vp, _sz, _vp], _i32),
    "qmoe_moe_forward": ([_i32, _DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
}

_lib = None


def lib():
    """Load libqmoe.so (raises when it is missing: there is no CPU path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QmoeError(f"{LIB_PATH} is not built; run quantized_mixture_experts_moe_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        # the tuned token-tile table shipped beside the library (QMOE_TILE_TABLE: another
        # file, or "none" for the built-in rule alone)
        path = os.environ.get("QMOE_TILE_TABLE", TILE_TABLE_PATH)
        if path != "none" and os.path.exists(path):
            set_tile_rules(read_tile_table(path))
    return _lib


TILE_TABLE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "tile_table.csv")
TILE_TABLE_FIELDS = ("scheme", "H", "I", "E", "k", "t_min", "t_max", "nmax")


def read_tile_table(path):
    """Rules from a tile-table CSV (header row; one rule per line, first match wins).  The
    scheme column records what the row was measured on; the library's rule is per shape."""
    import csv

    with open(path) as f:
        rows = [r for r in csv.DictReader(line for line in f if not line.startswith("#"))]
    return [dict(H=int(r["H"]), I=int(r["I"]), E=int(r["E"]), k=int(r["k"]), t_min=int(r["t_min"]),
                 t_max=int(r["t_max"]), nmax=int(r["nmax"])) for r in rows]


def set_tile_rules(rules):
    """Replace the library's token-tile table (a list of dicts with H, I, E, k, t_min, t_max, nmax)."""
    arr = (TileRule * max(1, len(rules)))()
    for i, r in enumerate(rules):
        arr[i] = TileRule(r.get("H", 0), r.get("I", 0), r.get("E", 0), r.get("k", 0), r.get("t_min", 0),
                          r.get("t_max", 2**62), r["nmax"], 0)
    _check(lib().qmoe_set_tile_rules(arr, len(rules)), "qmoe_set_tile_rules")


def tile_nmax(d: Dims) -> int:
    """The token tile (16, 112 or 224) the library uses for dims d."""
    return int(lib().qmoe_tile_nmax(ctypes.byref(d)))


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise QmoeError("qmoe kernels take device tensors")
    if not t.is_contiguous():
        raise QmoeError("qmoe kernels take contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, name: str):
    if rc != 0:
        raise QmoeError(f"{name} failed: {rc} ({lib().qmoe_status_str(rc).decode()})")


def dims(T, k, H, I, E) -> Dims:
    return Dims(T, k, H, I, E)


def status_str(code: int) -> str:
    return lib().qmoe_status_str(code).decode()


def version() -> str:
    return lib().qmoe_version().decode()


def workspace_bytes(d: Dims) -> int:
    return int(lib().qmoe_workspace_bytes(ctypes.byref(d)))


def forward_workspace_bytes(d: Dims, scheme: str) -> int:
    return int(lib().qmoe_forward_workspace_bytes(ctypes.byref(d), SCHEME_ID[scheme]))


def qmoe_align_sort(d, topk_ids, counts, offsets, sorted_pair_ids, pair_slot, dev_status, ws, stream=None):
    rc = lib().qmoe_align_sort(ctypes.byref(d), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(sorted_pair_ids),
                               _ptr(pair_slot), _ptr(dev_status), _ptr(ws), ws.numel() * ws.element_size(),
                               _stream(stream))
    _check(rc, "qmoe_align_sort")


STATIC_SCRATCH_BYTES = 1 << 20


def qmoe_align_sort_static_scratch(d, topk_ids, counts, offsets, sorted_pair_ids, pair_slot, dev_status,
                                   stream=None):
    """The routing sort with the library's built-in scratch (no workspace)."""
    rc = lib().qmoe_align_sort_static_scratch(ctypes.byref(d), _ptr(topk_ids), _ptr(counts), _ptr(offsets),
                                              _ptr(sorted_pair_ids), _ptr(pair_slot), _ptr(dev_status),
                                              _stream(stream))
    _check(rc, "qmoe_align_sort_static_scratch")


def qmoe_quant_act_mxfp8(x_bf16, x_q, x_s, stream=None):
    rows, cols = x_bf16.shape
    _check(lib().qmoe_quant_act_mxfp8(rows, cols, _ptr(x_bf16), _ptr(x_q), _ptr(x_s), _stream(stream)),
           "qmoe_quant_act_mxfp8")


def qmoe_quant_rows_int8_bf16(x, q, s, stream=None):
    rows, cols = x.shape
    _check(lib().qmoe_quant_rows_int8_bf16(rows, cols, _ptr(x), _ptr(q), _ptr(s), _stream(stream)),
           "qmoe_quant_rows_int8_bf16")


def qmoe_quant_rows_int8_f32(x, q, s, stream=None):
    rows, cols = x.shape
    _check(lib().qmoe_quant_rows_int8_f32(rows, cols, _ptr(x), _ptr(q), _ptr(s), _stream(stream)),
           "qmoe_quant_rows_int8_f32")


def _ws(ws):
    return _ptr(ws), (0 if ws is None else ws.numel() * ws.element_size())


def mx_scales_packed_bytes(rows: int, K: int) -> int:
    return int(lib().qmoe_mx_scales_packed_bytes(rows, K))


def qmoe_prepack_mx_scales(s_rowmajor, s_packed, rows: int, K: int, stream=None):
    _check(lib().qmoe_prepack_mx_scales(rows, K, _ptr(s_rowmajor), _ptr(s_packed), _stream(stream)),
           "qmoe_prepack_mx_scales")


def fp4_weights_packed_bytes(rows: int, K: int) -> int:
    return int(lib().qmoe_fp4_weights_packed_bytes(rows, K))


def qmoe_prepack_fp4_weights(w_rowmajor, w_packed, rows: int, K: int, stream=None):
    _check(lib().qmoe_prepack_fp4_weights(rows, K, _ptr(w_rowmajor), _ptr(w_packed), _stream(stream)),
           "qmoe_prepack_fp4_weights")


def prepack_fp4_weights(w_rowmajor, K: int, stream=None):
    """Packed 4-bit weights [..., K/2] (rows = all leading dims) -> tile-major byte tensor."""
    rows = w_rowmajor.numel() // (K // 2)
    out = torch.empty(max(fp4_weights_packed_bytes(rows, K), 16), dtype=torch.uint8, device=w_rowmajor.device)
    qmoe_prepack_fp4_weights(w_rowmajor.contiguous(), out, rows, K, stream)
    return out


def prepack_mxfp4(w1, w1_s, w2, w2_s, H: int, I: int, stream=None):
    """All four MXFP4 weight tensors in the form the GEMMs take."""
    return (prepack_fp4_weights(w1, H, stream), prepack_mx_scales(w1_s, H, stream),
            prepack_fp4_weights(w2, I, stream), prepack_mx_scales(w2_s, I, stream))


def prepack_mx_scales(s_rowmajor, K: int, stream=None):
    """E8M0 scales [..., K/32] (rows = all leading dims) -> packed byte tensor."""
    rows = s_rowmajor.numel() // (K // 32)
    out = torch.empty(max(mx_scales_packed_bytes(rows, K), 16), dtype=torch.uint8, device=s_rowmajor.device)
    qmoe_prepack_mx_scales(s_rowmajor.contiguous(), out, rows, K, stream)
    return out


def int4_weights_packed_bytes(rows: int, K: int) -> int:
    return int(lib().qmoe_int4_weights_packed_bytes(rows, K))


def qmoe_prepack_int4_weights(w_rowmajor, s_fp16, packed, rows: int, K: int, stream=None):
    _check(lib().qmoe_prepack_int4_weights(rows, K, _ptr(w_rowmajor), _ptr(s_fp16), _ptr(packed), _stream(stream)),
           "qmoe_prepack_int4_weights")


def prepack_int4_weights(w_rowmajor, s_fp16, K: int, stream=None):
    """int4 codes [..., K/2] + fp16 scales [..., K/32] (rows = all leading dims) -> packed byte tensor."""
    rows = w_rowmajor.numel() // (K // 2)
    out = torch.empty(max(int4_weights_packed_bytes(rows, K), 16), dtype=torch.uint8, device=w_rowmajor.device)
    qmoe_prepack_int4_weights(w_rowmajor.contiguous(), s_fp16.contiguous(), out, rows, K, stream)
    return out


def prepack_w4a16(w1, w1_s, w2, w2_s, H: int, I: int, stream=None):
    """Both W4A16 weight tensors (codes with their scales) in the form the GEMMs take."""
    return prepack_int4_weights(w1, w1_s, H, stream), prepack_int4_weights(w2, w2_s, I, stream)


def w4a16_x_tiles_bytes(d: Dims) -> int:
    return int(lib().qmoe_w4a16_x_tiles_bytes(ctypes.byref(d)))


def w4a16_h_tiles_bytes(d: Dims) -> int:
    return int(lib().qmoe_w4a16_h_tiles_bytes(ctypes.byref(d)))


def w4a16_h16_tiles_bytes(d: Dims) -> int:
    return int(lib().qmoe_w4a16_h16_tiles_bytes(ctypes.byref(d)))


def qmoe_w4a16_h_to_f16(d, h_tiles, offsets, h16_tiles, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_w4a16_h_to_f16(ctypes.byref(d), _ptr(h_tiles), _ptr(offsets), _ptr(h16_tiles), wp, wn,
                                     _stream(stream)), "qmoe_w4a16_h_to_f16")


def qmoe_permute_x_f16(d, x, sorted_pair_ids, offsets, x_tiles, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_permute_x_f16(ctypes.byref(d), _ptr(x), _ptr(sorted_pair_ids), _ptr(offsets), _ptr(x_tiles),
                                    wp, wn, _stream(stream)), "qmoe_permute_x_f16")


def qmoe_gemm1_swiglu_w4a16(d, x_tiles, w1, offsets, h_tiles, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm1_swiglu_w4a16(ctypes.byref(d), _ptr(x_tiles), _ptr(w1), _ptr(offsets), _ptr(h_tiles),
                                         _ptr(status), wp, wn, _stream(stream)), "qmoe_gemm1_swiglu_w4a16")


def mx_tiles_bytes(d: Dims, K: int) -> int:
    return int(lib().qmoe_mx_tiles_bytes(ctypes.byref(d), K))


def qmoe_permute_quant_mxfp8(d, x, pair_slot, offsets, x_tiles, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_permute_quant_mxfp8(ctypes.byref(d), _ptr(x), _ptr(pair_slot), _ptr(offsets),
                                          _ptr(x_tiles), wp, wn, _stream(stream)), "qmoe_permute_quant_mxfp8")


def qmoe_gemm1_swiglu_mxfp4(d, x_tiles, w1, w1_s, offsets, h_tiles, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm1_swiglu_mxfp4(ctypes.byref(d), _ptr(x_tiles), _ptr(w1), _ptr(w1_s), _ptr(offsets),
                                         _ptr(h_tiles), _ptr(status), wp, wn, _stream(stream)),
           "qmoe_gemm1_swiglu_mxfp4")


def qmoe_gemm1_swiglu_mxfp4_gather(d, x_q, x_s, sorted_pair_ids, w1, w1_s, offsets, h_tiles, status, ws,
                                   stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm1_swiglu_mxfp4_gather(ctypes.byref(d), _ptr(x_q), _ptr(x_s), _ptr(sorted_pair_ids),
                                                _ptr(w1), _ptr(w1_s), _ptr(offsets), _ptr(h_tiles), _ptr(status),
                                                wp, wn, _stream(stream)),
           "qmoe_gemm1_swiglu_mxfp4_gather")


def forward_launches(d: Dims, scheme: str) -> int:
    return int(lib().qmoe_forward_launches(ctypes.byref(d), SCHEME_ID[scheme]))


def mx_layer_gathers(d: Dims) -> bool:
    return bool(lib().qmoe_mx_layer_gathers(ctypes.byref(d)))


def w8a8_tiles_bytes(d: Dims, K: int) -> int:
    return int(lib().qmoe_w8a8_tiles_bytes(ctypes.byref(d), K))


def qmoe_permute_quant_int8(d, x, sorted_pair_ids, offsets, x_tiles, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_permute_quant_int8(ctypes.byref(d), _ptr(x), _ptr(sorted_pair_ids), _ptr(offsets),
                                         _ptr(x_tiles), wp, wn, _stream(stream)), "qmoe_permute_quant_int8")


def qmoe_quant_tiles_int8_f32(d, h, offsets, h_tiles, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_quant_tiles_int8_f32(ctypes.byref(d), _ptr(h), _ptr(offsets), _ptr(h_tiles), wp, wn,
                                           _stream(stream)), "qmoe_quant_tiles_int8_f32")


def qmoe_gemm1_swiglu_w8a8(d, x_tiles, w1, w1_s, offsets, h, dbg_acc, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm1_swiglu_w8a8(ctypes.byref(d), _ptr(x_tiles), _ptr(w1), _ptr(w1_s), _ptr(offsets), _ptr(h),
                                        _ptr(dbg_acc), _ptr(status), wp, wn, _stream(stream)),
           "qmoe_gemm1_swiglu_w8a8")


def qmoe_gemm2_w4a16(d, h16_tiles, w2, offsets, y, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm2_w4a16(ctypes.byref(d), _ptr(h16_tiles), _ptr(w2), _ptr(offsets), _ptr(y), _ptr(status),
                                  wp, wn, _stream(stream)), "qmoe_gemm2_w4a16")


def qmoe_gemm2_mxfp4(d, h_tiles, w2, w2_s, offsets, y, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm2_mxfp4(ctypes.byref(d), _ptr(h_tiles), _ptr(w2), _ptr(w2_s), _ptr(offsets), _ptr(y),
                                  _ptr(status), wp, wn, _stream(stream)), "qmoe_gemm2_mxfp4")


def qmoe_gemm2_w8a8(d, h_tiles, w2, w2_s, offsets, y, dbg_acc, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm2_w8a8(ctypes.byref(d), _ptr(h_tiles), _ptr(w2), _ptr(w2_s), _ptr(offsets), _ptr(y),
                                 _ptr(dbg_acc), _ptr(status), wp, wn, _stream(stream)), "qmoe_gemm2_w8a8")


def qmoe_combine(d, y, topk_w, pair_slot, out, stream=None):
    _check(lib().qmoe_combine(ctypes.byref(d), _ptr(y), _ptr(topk_w), _ptr(pair_slot), _ptr(out), _stream(stream)),
           "qmoe_combine")


def qmoe_gemm1_swiglu_w4a8(d, x_tiles, w1, w1_s, offsets, h, dbg_acc, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm1_swiglu_w4a8(ctypes.byref(d), _ptr(x_tiles), _ptr(w1), _ptr(w1_s), _ptr(offsets), _ptr(h),
                                        _ptr(dbg_acc), _ptr(status), wp, wn, _stream(stream)),
           "qmoe_gemm1_swiglu_w4a8")


def qmoe_gemm2_w4a8(d, h_tiles, w2, w2_s, offsets, y, dbg_acc, status, ws, stream=None):
    wp, wn = _ws(ws)
    _check(lib().qmoe_gemm2_w4a8(ctypes.byref(d), _ptr(h_tiles), _ptr(w2), _ptr(w2_s), _ptr(offsets), _ptr(y),
                                 _ptr(dbg_acc), _ptr(status), wp, wn, _stream(stream)), "qmoe_gemm2_w4a8")


def qmoe_moe_forward(scheme, d, x, topk_ids, topk_w, w1, w1_s, w2, w2_s, out, dev_status, ws, stream=None):
    rc = lib().qmoe_moe_forward(SCHEME_ID[scheme], ctypes.byref(d), _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w1),
                                _ptr(w1_s), _ptr(w2), _ptr(w2_s), _ptr(out), _ptr(dev_status), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "qmoe_moe_forward")


# ------------------------------------------------------------------ conveniences (torch allocation only)

def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte-aligned byte workspace (torch allocations are 512-aligned)."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def moe_forward(scheme, x, topk_ids, topk_w, w1, w1_s, w2, w2_s, H=None, I=None, E=None, ws=None, stream=None):
    """Whole layer through qmoe_moe_forward; returns (out bf16-bits [T, H], dev_status)."""
    T, H_ = x.shape
    k = topk_ids.shape[1]
    E_ = w1.shape[0] if E is None else E
    I_ = (w1.shape[1] // 2) if I is None else I
    d = dims(T, k, H_, I_, E_)
    if ws is None:
        ws = alloc_workspace(forward_workspace_bytes(d, scheme), x.device)
    out = torch.empty((T, H_), dtype=torch.int16, device=x.device)
    status = torch.zeros(1, dtype=torch.int32, device=x.device)
    qmoe_moe_forward(scheme, d, x, topk_ids, topk_w, w1, w1_s, w2, w2_s, out, status, ws, stream)
    return out, status


# ------------------------------------------------------------------ around the experts: norms, routing, FP8 products
#
# These take tensors of torch's float32, bfloat16 and float16 (int16 tensors
# are bf16 bits, as above) whose last axis is contiguous; rows may be strided.
# They allocate their outputs, run on the current stream (or on the one that
# the keyword `stream` names, on which their outputs then belong) and raise QmoeError for what the library refuses and ValueError for tensors whose
# shapes or types do not go together.

GATE_NONE, GATE_ROW, GATE_COL, GATE_FULL = 0, 1, 2, 3
FP8_BLOCK = 128

_F32, _U8, _I32 = torch.float32, torch.uint8, torch.int32
_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.int16: 1, torch.float16: 2}

# These calls are made for single tokens too, where the kernels take a few
# microseconds: the checks below cost one comparison each, messages are built
# only to be raised, and the stream is asked for by device index.
_empty = torch.empty
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent from builds without CUDA


def _dtype(dtype) -> int:
    try:
        return _DTYPE[dtype]
    except KeyError:
        raise ValueError(f"expected float32, bfloat16 or float16, got {dtype}") from None


def _here(t):
    """The current stream of the device of tensor t."""
    i = t.get_device()
    if i < 0:
        raise QmoeError("qmoe kernels take device tensors")
    return _raw_stream(i)


def _rows(t, T, H):
    """(pointer, row stride) of a [T, H] device tensor with contiguous rows."""
    if t.shape != (T, H):
        raise ValueError(f"expected a tensor of shape {[T, H]}, got {list(t.shape)}")
    if not t.is_cuda:
        raise QmoeError("qmoe kernels take device tensors")
    ld, step = t.stride()
    if step != 1 and H > 1:
        raise QmoeError("qmoe kernels take rows of contiguous columns")
    if ld < H:
        if T > 1:
            raise QmoeError("qmoe kernels take rows that do not overlap")
        ld = H
    return t.data_ptr(), ld


def _vec(t, n, dtype=_F32):
    """Pointer of a contiguous device tensor of n values (None: NULL)."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n:
        raise ValueError(f"expected {n} values of {dtype}, got {list(t.shape)} of {t.dtype}")
    if not t.is_cuda:
        raise QmoeError("qmoe kernels take device tensors")
    if not t.is_contiguous():
        raise QmoeError("qmoe kernels take contiguous tensors")
    return t.data_ptr()


def _at(t):
    return None if t is None else t.data_ptr()


def _on_stream(fn):
    """Runs a call that was given a stream as the current stream's, so that what it allocates (outputs, workspaces, codes)
    belongs to the stream that uses it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _ws_for(nbytes, ws, device):
    """(pointer, bytes, tensor) of a workspace: the caller's, or a new one."""
    if ws is None:
        ws = _empty(max(nbytes, 256), dtype=_U8, device=device)
        return ws.data_ptr(), max(nbytes, 256), ws
    return _ptr(ws), ws.numel() * ws.element_size(), ws


@_on_stream
def norm_pre(x, w, eps=1e-6, out_dtype=None):
    """n = x / rms(x) * w for rows x [T, H], w fp32 [H]; returns (n, rstd fp32 [T]).  n has x's type, or a 16-bit
    out_dtype beside fp32 x."""
    T, H = x.shape
    dev, dtype = x.device, x.dtype
    if out_dtype is None:
        out_dtype = dtype
    xp, ldx = _rows(x, T, H)
    n = _empty((T, H), dtype=out_dtype, device=dev)
    rstd = _empty((T,), dtype=_F32, device=dev)
    rc = lib().qmoe_norm_pre(T, H, _dtype(dtype), _dtype(out_dtype), xp, ldx, _vec(w, H), eps, n.data_ptr(), H,
                             rstd.data_ptr(), _here(x))
    if rc:
        _check(rc, "qmoe_norm_pre")
    return n, rstd


@_on_stream
def norm_pre_backward(dn, x, rstd, w, dres=None, ws=None):
    """Gradients of norm_pre: (dx [T, H] in x's type, dw fp32 [H]); dres (x's type) is added to dx."""
    T, H = x.shape
    dev, dtype = x.device, x.dtype
    xp, ldx = _rows(x, T, H)
    dnp, lddn = _rows(dn, T, H)
    drp, lddr = None, 0
    if dres is not None:
        if dres.dtype != dtype:
            raise ValueError("dres has x's type")
        drp, lddr = _rows(dres, T, H)
    dx = _empty((T, H), dtype=dtype, device=dev)
    dw = _empty((H,), dtype=_F32, device=dev)
    L = lib()
    wp, wn, ws = _ws_for(L.qmoe_norm_bwd_workspace_bytes(T, H), ws, dev)
    rc = L.qmoe_norm_pre_backward(T, H, _dtype(dtype), _dtype(dn.dtype), dnp, lddn, xp, ldx, _vec(rstd, T), _vec(w, H), drp,
                                  lddr, dx.data_ptr(), H, dw.data_ptr(), wp, wn, _here(x))
    if rc:
        _check(rc, "qmoe_norm_pre_backward")
    return dx, dw


def _gate(gate, T, H, block_dtype):
    """(mode, pointer, row stride) of a gate: None; one fp32 value for each row, [T, 1] or [T]; one fp32 value for each
    column, [1, H] or [H]; or [T, H] of the block's type.  A 1-D gate of T == H values is one for each row: give a column
    gate as [1, H] where the number of rows may be anything."""
    if gate is None:
        return GATE_NONE, None, 0
    shape = tuple(gate.shape)
    if shape == (T,) or shape == (T, 1) and gate.dtype == _F32:
        return GATE_ROW, _vec(gate, T), 0
    if shape == (T, H) and gate.dtype == block_dtype:
        return (GATE_FULL, *_rows(gate, T, H))
    if shape == (H,) or shape == (1, H):
        return GATE_COL, _vec(gate, H), 0
    raise ValueError(f"a gate is fp32 [T, 1], [T], [1, H] or [H], or [T, H] of the block's type; got {list(shape)} of {gate.dtype}")


@_on_stream
def norm_post(r, y, w=None, gate=None, alpha=1.0, w_next=None, eps=1e-6):
    """out = r + alpha * gate * (y / rms(y) * w) for rows r, y [T, H] (w None: y itself), and n = out / rms(out) * w_next
    where w_next is given.  Returns (out, n, rstd, rstd_next), None for what is not computed.  out has r's type, n y's.
    gate: None, fp32 [T, 1] or [T] (one for each row), fp32 [1, H] or [H] (one for each column; [H] is taken as [T]
    where T == H), or [T, H] of y's type."""
    T, H = y.shape
    dev, st, bt = y.device, r.dtype, y.dtype
    rp, ldr = _rows(r, T, H)
    yp, ldy = _rows(y, T, H)
    mode, gp, ldg = _gate(gate, T, H, bt)
    out = _empty((T, H), dtype=st, device=dev)
    n = rstd = rstd_next = None
    if w is not None:
        rstd = _empty((T,), dtype=_F32, device=dev)
    if w_next is not None:
        n = _empty((T, H), dtype=bt, device=dev)
        rstd_next = _empty((T,), dtype=_F32, device=dev)
    rc = lib().qmoe_norm_post(T, H, _dtype(st), _dtype(bt), rp, ldr, yp, ldy, _vec(w, H), mode, gp, ldg, alpha,
                              _vec(w_next, H), eps, out.data_ptr(), H, _at(n), H, _at(rstd), _at(rstd_next), _here(y))
    if rc:
        _check(rc, "qmoe_norm_post")
    return out, n, rstd, rstd_next


@_on_stream
def norm_post_backward(dout, y, w=None, rstd=None, gate=None, alpha=1.0, dn=None, out=None, w_next=None, rstd_next=None,
                       ws=None):
    """Gradients of norm_post from dout (the stream's; None: 0) and dn (of n; None: 0): (dr, dy, dw, dgate, dw_next), None
    for what has no input.  y, w, gate, alpha, w_next as in the forward call, out, rstd, rstd_next as it returned them."""
    T, H = y.shape
    dev, bt = y.device, y.dtype
    if dout is None and dn is None:
        raise ValueError("norm_post_backward needs dout or dn")
    if w is not None and rstd is None:
        raise ValueError("w needs rstd")
    dop, lddo, dnp, lddn, op, ldo, wnp, rnp = None, 0, None, 0, None, 0, None, None
    dw = dw_next = dgate = None
    if dn is not None:
        if out is None or w_next is None or rstd_next is None:
            raise ValueError("dn needs out, w_next and rstd_next")
        if dn.dtype != bt or dout is not None and out.dtype != dout.dtype:
            raise ValueError("dn has y's type, and out dout's")
        dnp, lddn = _rows(dn, T, H)
        op, ldo = _rows(out, T, H)
        wnp, rnp = _vec(w_next, H), _vec(rstd_next, T)
        dw_next = _empty((H,), dtype=_F32, device=dev)
    if dout is not None:
        dop, lddo = _rows(dout, T, H)
    st = out.dtype if dout is None else dout.dtype
    yp, ldy = _rows(y, T, H)
    mode, gp, ldg = _gate(gate, T, H, bt)
    dr = _empty((T, H), dtype=st, device=dev)
    dy = _empty((T, H), dtype=bt, device=dev)
    if w is not None:
        dw = _empty((H,), dtype=_F32, device=dev)
    if gate is not None:
        dgate = _empty(gate.shape, dtype=gate.dtype, device=dev)
    if T == 0:  # no rows (and no pointers to tell what was given): the sums are zero
        return dr, dy, *(t if t is None else t.zero_() for t in (dw, dgate, dw_next))
    L = lib()
    wp, wn, ws = _ws_for(L.qmoe_norm_bwd_workspace_bytes(T, H), ws, dev)
    rc = L.qmoe_norm_post_backward(T, H, _dtype(st), _dtype(bt), dop, lddo, yp, ldy, _vec(w, H),
                                   None if w is None else _vec(rstd, T), mode, gp, ldg, alpha, dnp, lddn, op, ldo, wnp, rnp,
                                   dr.data_ptr(), H, dy.data_ptr(), H, _at(dw), _at(dgate), H, _at(dw_next), wp, wn, _here(y))
    if rc:
        _check(rc, "qmoe_norm_post_backward")
    return dr, dy, dw, dgate, dw_next


class Routing:
    """What route_topk returns, and what its gradient takes: ids int32 [T, k], w fp32 [T, k], lse fp32 [T]; with coef also
    counts int32 [E + 1] (the last is the number of routed tokens), probs fp32 [E], loss fp32 [1] (else None); and the
    call's renorm, scale and coef."""
    __slots__ = ("ids", "w", "lse", "counts", "probs", "loss", "renorm", "scale", "coef")

    def __init__(self, ids, w, lse, counts, probs, loss, renorm, scale, coef):
        self.ids, self.w, self.lse, self.counts, self.probs, self.loss = ids, w, lse, counts, probs, loss
        self.renorm, self.scale, self.coef = renorm, scale, coef


@_on_stream
def route_topk(logits, k, bias=None, mask=None, renorm=True, scale=1.0, coef=None, ws=None) -> Routing:
    """The k experts of largest logit + bias of each row of logits [T, E] and their weights; with coef also the balance
    loss and the per-expert counts.  mask (bool or uint8 [T]): rows where it is 0 are routed nowhere (ids -1)."""
    T, E = logits.shape
    dev = logits.device
    lp, ld = _rows(logits, T, E)
    if mask is not None and mask.dtype == torch.bool:
        mask = mask.view(_U8)
    ids = _empty((T, k), dtype=_I32, device=dev)
    w = _empty((T, k), dtype=_F32, device=dev)
    lse = _empty((T,), dtype=_F32, device=dev)
    L = lib()
    if coef is None:
        counts = probs = loss = None
        rc = L.qmoe_route_topk(T, E, k, _dtype(logits.dtype), lp, ld, _vec(bias, E), _vec(mask, T, _U8), renorm, scale,
                               ids.data_ptr(), w.data_ptr(), lse.data_ptr(), 0.0, None, None, None, None, 0, _here(logits))
    else:
        counts = _empty((E + 1,), dtype=_I32, device=dev)
        probs = _empty((E,), dtype=_F32, device=dev)
        loss = _empty((1,), dtype=_F32, device=dev)
        wp, wn, ws = _ws_for(L.qmoe_route_workspace_bytes(T, E), ws, dev)
        rc = L.qmoe_route_topk(T, E, k, _dtype(logits.dtype), lp, ld, _vec(bias, E), _vec(mask, T, _U8), renorm, scale,
                               ids.data_ptr(), w.data_ptr(), lse.data_ptr(), coef, counts.data_ptr(), probs.data_ptr(),
                               loss.data_ptr(), wp, wn, _here(logits))
    if rc:
        _check(rc, "qmoe_route_topk")
    return Routing(ids, w, lse, counts, probs, loss, renorm, scale, coef)


@_on_stream
def route_topk_backward(logits, routing: Routing, dw=None, dloss=None):
    """dlogits (the logits' type) from dw fp32 [T, k] and / or dloss fp32 [1]."""
    T, E = logits.shape
    k = routing.ids.shape[1]
    if dw is None and dloss is None:
        raise ValueError("route_topk_backward needs dw or dloss")
    if dloss is not None and routing.coef is None:
        raise ValueError("dloss needs a routing made with coef")
    lp, ld = _rows(logits, T, E)
    dlogits = _empty((T, E), dtype=logits.dtype, device=logits.device)
    if T == 0:
        return dlogits
    rc = lib().qmoe_route_topk_backward(T, E, k, _dtype(logits.dtype), lp, ld, _vec(routing.ids, T * k, _I32),
                                        _vec(routing.w, T * k), _vec(routing.lse, T), routing.renorm, routing.scale,
                                        _vec(dw, T * k), routing.coef or 0.0, _vec(routing.counts, E + 1, _I32),
                                        _vec(dloss, 1), dlogits.data_ptr(), E, _here(logits))
    if rc:
        _check(rc, "qmoe_route_topk_backward")
    return dlogits


def _blocks(n):
    return (n + 127) // 128


def _up16(n):
    return (n + 15) // 16 * 16


def _codes(rows, cols, device):
    """Uninitialised E4M3 codes [rows, cols] whose rows start on 16-byte boundaries."""
    return _empty((rows, _up16(cols)), dtype=torch.float8_e4m3fn, device=device)[:, :cols]


@_on_stream
def fp8_quant_rows(x):
    """E4M3 codes of x [T, K] (float8_e4m3fn) and their scales [T, ceil(K / 128)], one for each 128 of a row."""
    T, K = x.shape
    xp, ldx = _rows(x, T, K)
    q = _codes(T, K, x.device)
    s = _empty((_blocks(K), T), dtype=_F32, device=x.device)
    rc = lib().qmoe_fp8_quant_rows(T, K, _dtype(x.dtype), xp, ldx, q.data_ptr(), _up16(K), s.data_ptr(), _here(x))
    if rc:
        _check(rc, "qmoe_fp8_quant_rows")
    return q, s.t()


@_on_stream
def fp8_quant_cols(x, rows_too=False):
    """E4M3 codes of x [T, K] transposed, [K, T], and their scales [K, ceil(T / 128)], one for each 128 of a column of x;
    with rows_too (qt, st, q, s), what fp8_quant_rows gives from the same read of x."""
    T, K = x.shape
    xp, ldx = _rows(x, T, K)
    qt = _codes(K, T, x.device)
    st = _empty((_blocks(T), K), dtype=_F32, device=x.device)
    q = s = None
    if rows_too:
        q = _codes(T, K, x.device)
        s = _empty((_blocks(K), T), dtype=_F32, device=x.device)
    rc = lib().qmoe_fp8_quant_cols(T, K, _dtype(x.dtype), xp, ldx, qt.data_ptr(), _up16(T), st.data_ptr(), _at(q), _up16(K),
                                   _at(s), _here(x))
    if rc:
        _check(rc, "qmoe_fp8_quant_cols")
    return (qt, st.t(), q, s.t()) if rows_too else (qt, st.t())


@_on_stream
def fp8_quant_blocks(w, transposed=False):
    """E4M3 codes of w [N, K] and their scales [ceil(N / 128), ceil(K / 128)], one for each 128 x 128 block; with
    transposed also the codes as [K, N] (their scales are the transposed scales)."""
    N, K = w.shape
    wp, ldw = _rows(w, N, K)
    q = _codes(N, K, w.device)
    qt = _codes(K, N, w.device) if transposed else None
    s = _empty((_blocks(N), _blocks(K)), dtype=_F32, device=w.device)
    rc = lib().qmoe_fp8_quant_blocks(N, K, _dtype(w.dtype), wp, ldw, q.data_ptr(), _up16(K), _at(qt), _up16(N), s.data_ptr(),
                                     _here(w))
    if rc:
        _check(rc, "qmoe_fp8_quant_blocks")
    return (q, s, qt) if transposed else (q, s)


def _fp8_mat(q, s):
    rows, K = q.shape
    if q.dtype != torch.float8_e4m3fn and q.dtype != _U8:
        raise ValueError(f"expected float8_e4m3fn or uint8 codes, got {q.dtype}")
    blocks = (K + 127) // 128
    tall = 1
    if s.shape != (rows, blocks):
        tall = FP8_BLOCK
        if s.shape != (_blocks(rows), blocks):
            raise ValueError(f"expected scales [{rows} or {_blocks(rows)}, {blocks}], got {list(s.shape)}")
    if s.dtype != _F32:
        raise ValueError(f"expected fp32 scales, got {s.dtype}")
    if not s.is_cuda:
        raise QmoeError("qmoe kernels take device tensors")
    qp, ld = _rows(q, rows, K)
    if rows == 1:
        ld = _up16(ld)  # the stride of a single row is not used
    s_row, s_blk = s.stride()
    return Fp8Mat(qp, ld, s.data_ptr(), s_row, s_blk, tall, 0)


_status_words = {}


def status_word(device):
    """The int32 device word where the FP8 products report a wait that ran out (QMOE_DEV_WAIT_TIMEOUT) unless a call is
    given its own: one for each device, zero until then."""
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    if index not in _status_words:
        _status_words[index] = torch.zeros(1, dtype=_I32, device=f"cuda:{index}")
        torch.cuda.synchronize(index)  # seen by every stream
    return _status_words[index]


def _status(dev_status, t):
    if dev_status is None:
        dev_status = _status_words.get(t.get_device())
        if dev_status is None:
            dev_status = status_word(t.device)
    return _vec(dev_status, 1, _I32)


@_on_stream
def fp8_matmul(a_q, a_s, b_q, b_s, out_dtype=torch.bfloat16, dev_status=None):
    """c [M, N] = a b^T of E4M3 codes a_q [M, K], b_q [N, K] with fp32 scales [rows or ceil(rows / 128), ceil(K / 128)] of
    any strides."""
    M, K = a_q.shape
    N = b_q.shape[0]
    if b_q.shape[1] != K:
        raise ValueError(f"reduction lengths {K} and {b_q.shape[1]} differ")
    a, b = _fp8_mat(a_q, a_s), _fp8_mat(b_q, b_s)
    c = _empty((M, N), dtype=out_dtype, device=a_q.device)
    rc = lib().qmoe_fp8_matmul(M, N, K, ctypes.byref(a), ctypes.byref(b), c.data_ptr(), _dtype(out_dtype), N,
                               _status(dev_status, a_q), _here(a_q))
    if rc:
        _check(rc, "qmoe_fp8_matmul")
    return c


@_on_stream
def fp8_linear(x, w_q, w_s, out_dtype=None, dev_status=None, ws=None):
    """y = x w^T for x [T, K], quantised on the way (fp8_quant_rows), and a quantised weight w_q [N, K], w_s."""
    T, K = x.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError(f"reduction lengths {K} and {w_q.shape[1]} differ")
    dev, dtype = x.device, x.dtype
    if out_dtype is None:
        out_dtype = dtype
    xp, ldx = _rows(x, T, K)
    w = _fp8_mat(w_q, w_s)
    y = _empty((T, N), dtype=out_dtype, device=dev)
    L = lib()
    wp, wn, ws = _ws_for(L.qmoe_fp8_linear_workspace_bytes(T, K), ws, dev)
    rc = L.qmoe_fp8_linear(T, N, K, _dtype(dtype), xp, ldx, ctypes.byref(w), y.data_ptr(), _dtype(out_dtype), N,
                           _status(dev_status, x), wp, wn, _here(x))
    if rc:
        _check(rc, "qmoe_fp8_linear")
    return y


@_on_stream
def fp8_linear_backward(dy, x, wt_q, w_s, dev_status=None):
    """Gradients of y = x w^T: (dx = dy w in dy's type, dw = dy^T x in fp32).  dy and x are quantised along the axis that
    each product sums; wt_q [K, N] are the weight's transposed codes and w_s its scales (fp8_quant_blocks)."""
    T, N = dy.shape
    K = x.shape[1]
    if x.shape[0] != T or wt_q.shape != (K, N):
        raise ValueError("dy [T, N], x [T, K] and wt_q [K, N] do not go together")
    if T == 0:
        return _empty((0, K), dtype=dy.dtype, device=dy.device), torch.zeros((N, K), dtype=_F32, device=dy.device)
    dyt_q, dyt_s, dy_q, dy_s = fp8_quant_cols(dy, rows_too=True)
    xt_q, xt_s = fp8_quant_cols(x)
    dx = fp8_matmul(dy_q, dy_s, wt_q, w_s.t(), out_dtype=dy.dtype, dev_status=dev_status)
    dw = fp8_matmul(dyt_q, dyt_s, xt_q, xt_s, out_dtype=_F32, dev_status=dev_status)
    return dx, dw
