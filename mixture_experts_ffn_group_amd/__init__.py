"""MI355X (gfx950) sparse-MoE expert FFN: Python binding of libmoe_ffn.so.

Every step of the layer runs in the library's HIP kernels; this module only
checks tensor dtypes/devices, allocates outputs with torch on the input's
device and passes raw pointers and torch's current HIP stream. Names follow
the C ABI in include/moe_ffn.h:

    route, permute, grouped_gemm, grouped_gemm_wgrad, combine, combine_bwd,
    ffn_fwd, ffn_bwd
    route_scored, route_scored_bwd: routing by scores, groups and a balance bias
    ckpt_quantize, ckpt_dequantize, swiglu_bwd_ckpt, grouped_gemm_wgrad_ckpt:
    activations kept in 8 bits between the passes
    ffn_fwd_routed, ffn_bwd_ckpt: the layer on a given routing, and its
    backward from the 8-bit saved set
    ffn_fwd_few, ffn_fwd_few_mx: the layer for a few tokens (a decode step)
    norm, norm_bwd, block_out, block_out_bwd: the norms around the layer, with
    the gate and the residual sum

Tensors: bf16 activations/weights, fp32 router weights/logits/top-k weights,
int32 indices, all contiguous and on one CUDA (HIP) device.
"""
from __future__ import annotations

import ctypes as C
import functools
import operator
import struct

import torch

from . import _lib
from ._lib import (MOE_EPI_NONE, MOE_EPI_SWIGLU, MOE_EPI_SWIGLU_BWD, MOE_NN, MOE_NT, MoeError,  # noqa: F401
                   MoeGemmRows, MoeSaved, MoeShape)

__all__ = ["route", "permute", "grouped_gemm", "grouped_gemm_wgrad", "combine", "combine_bwd", "ffn_fwd", "ffn_bwd",
           "route_scored", "route_scored_bwd", "ckpt_quantize", "ckpt_dequantize", "swiglu_bwd_ckpt",
           "grouped_gemm_wgrad_ckpt", "ffn_fwd_routed", "ffn_bwd_ckpt",
           "ffn_fwd_few", "ffn_fwd_few_mx", "norm", "norm_bwd", "block_out", "block_out_bwd", "query_support", "workspace_bytes", "MoeError"]

_EPI = {"none": MOE_EPI_NONE, "swiglu": MOE_EPI_SWIGLU, "swiglu_bwd": MOE_EPI_SWIGLU_BWD}
_OP = {"nn": MOE_NN, "nt": MOE_NT}


def _ptr(t: torch.Tensor | None):
    return None if t is None else C.c_void_p(t.data_ptr())


# The current stream's handle straight from torch, where it offers that (0.1 us; building a Stream object to
# read it from costs 1.8 us, half a kernel launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device):
    if _raw_stream is not None and dev.index is not None:
        return C.c_void_p(_raw_stream(dev.index))
    return C.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, name, dtype, device=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def query_support(T: int, emb: int, mlp: int, E: int, k: int) -> None:
    """Raise MoeError if the layer kernels do not support this shape."""
    s = _lib.shape(T, emb, mlp, E, k)
    _lib.check(_lib.lib().moe_query_support(C.byref(s)), "moe_query_support")


def workspace_bytes(T: int, emb: int, mlp: int, E: int, k: int, backward: bool = False,
                    recompute_h: bool = False) -> int:
    s = _lib.shape(T, emb, mlp, E, k)
    return int(_lib.lib().moe_workspace_bytes(C.byref(s), (2 if recompute_h else 1) if backward else 0))


def route(k: int, x: torch.Tensor | None = None, wr: torch.Tensor | None = None, bias: torch.Tensor | None = None,
          logits: torch.Tensor | None = None):
    """(topk_idx [T,k] int32, topk_w [T,k] fp32). Either x [T,emb] bf16 + wr [emb,E] fp32 (+ bias [E]),
    or logits [T,E] fp32."""
    if logits is not None:
        _need(logits, "logits", torch.float32)
        dev = logits.device
        T, E = logits.shape
        emb = 64
    else:
        _need(x, "x", torch.bfloat16)
        dev = x.device
        _need(wr, "wr", torch.float32, dev)
        _need(bias, "bias", torch.float32, dev)
        T, emb = x.shape
        E = wr.shape[1]
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    s = _lib.shape(T, emb, 64, E, k)
    _lib.check(_lib.lib().moe_route(C.byref(s), _ptr(x), _ptr(wr), _ptr(bias), _ptr(logits), _ptr(idx), _ptr(w),
                                    _stream(dev)), "moe_route")
    return idx, w


def permute(x: torch.Tensor, topk_idx: torch.Tensor, E: int, rows: bool = True, noalloc: bool = False) -> dict:
    """Expert-sorted gather: dict of group_sizes [E], group_offsets [E+1], sorted_slot [S], slot_row [S]
    (int32) and xs [S, emb] bf16. rows=False builds the index only (no xs). noalloc=True calls
    moe_permute_noalloc, which takes no workspace (the library's fixed per-GPU scratch)."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(topk_idx, "topk_idx", torch.int32, dev)
    T, emb = x.shape
    k = topk_idx.shape[1]
    S = T * k
    s = _lib.shape(T, emb, 64, E, k)
    out = dict(group_sizes=torch.empty(E, dtype=torch.int32, device=dev),
               group_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               sorted_slot=torch.empty(S, dtype=torch.int32, device=dev),
               slot_row=torch.empty(S, dtype=torch.int32, device=dev),
               xs=torch.empty((S, emb), dtype=torch.bfloat16, device=dev) if rows else None)
    if noalloc:
        _lib.check(_lib.lib().moe_permute_noalloc(C.byref(s), _ptr(x), _ptr(topk_idx), _ptr(out["group_sizes"]),
                                                  _ptr(out["group_offsets"]), _ptr(out["sorted_slot"]),
                                                  _ptr(out["slot_row"]), _ptr(out["xs"]), _stream(dev)),
                   "moe_permute_noalloc")
        return out
    ws_n = int(_lib.lib().moe_permute_workspace_bytes(C.byref(s)))
    ws = torch.empty(max(ws_n, 16), dtype=torch.uint8, device=dev)
    _lib.check(_lib.lib().moe_permute(C.byref(s), _ptr(x), _ptr(topk_idx), _ptr(out["group_sizes"]),
                                      _ptr(out["group_offsets"]), _ptr(out["sorted_slot"]), _ptr(out["slot_row"]),
                                      _ptr(out["xs"]), _ptr(ws), ws.numel(), _stream(dev)), "moe_permute")
    return out


def grouped_gemm(A: torch.Tensor, B: torch.Tensor, group_offsets: torch.Tensor, op: str = "nn",
                 epilogue: str = "none", aux_in: torch.Tensor | None = None, save_h: bool = False,
                 out: torch.Tensor | None = None, row_slot: torch.Tensor | None = None, slot_div: int = 1,
                 slot_scale: torch.Tensor | None = None, M: int | None = None, grid: int = 0):
    """Ragged grouped GEMM (see moe_grouped_gemm). Returns C, or (C, h) with save_h (SwiGLU, h in fp32).

    row_slot [M] int32 (optional): output row r reads A row row_slot[r] // slot_div (A is not permuted).
    slot_scale (optional, fp32): per-row scale, indexed by row_slot[r] (or r).
    grid: workgroups of the persistent grid (0 = one per compute unit; see moe_grouped_gemm_grid)."""
    _need(A, "A", torch.bfloat16)
    dev = A.device
    _need(B, "B", torch.bfloat16, dev)
    _need(group_offsets, "group_offsets", torch.int32, dev)
    _need(aux_in, "aux_in", torch.float32, dev)
    _need(row_slot, "row_slot", torch.int32, dev)
    _need(slot_scale, "slot_scale", torch.float32, dev)
    K = A.shape[1]
    if M is None:
        M = row_slot.numel() if row_slot is not None else A.shape[0]
    E = B.shape[0]
    N = B.shape[2] if op == "nn" else B.shape[1]
    _lib.need_32_bits(E | K | N | slot_div | grid, "E, K, N, slot_div and grid")
    epi = _EPI[epilogue]
    width = N if epi == MOE_EPI_NONE else (N // 2 if epi == MOE_EPI_SWIGLU else 2 * N)
    C_ = out if out is not None else torch.empty((M, width), dtype=torch.bfloat16, device=dev)
    _need(C_, "out", torch.bfloat16, dev)
    h = torch.empty((M, N), dtype=torch.float32, device=dev) if (save_h and epi == MOE_EPI_SWIGLU) else None
    rows = None
    if row_slot is not None or slot_scale is not None:
        n_slots = A.shape[0] * slot_div if row_slot is not None else 0
        rows = C.byref(MoeGemmRows(None if row_slot is None else row_slot.data_ptr(), n_slots, slot_div,
                                   None if slot_scale is None else slot_scale.data_ptr()))
    _lib.check(_lib.lib().moe_grouped_gemm_grid(_OP[op], epi, _ptr(A), _ptr(B), _ptr(aux_in), _ptr(h),
                                                _ptr(group_offsets), E, M, K, N, rows, _ptr(C_), grid, _stream(dev)),
               "moe_grouped_gemm")
    return (C_, h) if save_h else C_


def grouped_gemm_wgrad(A: torch.Tensor, D: torch.Tensor, group_offsets: torch.Tensor, E: int,
                       grid: int = 0) -> torch.Tensor:
    """C [E, P, Q] = per-group A^T D (grid as in grouped_gemm)."""
    _need(A, "A", torch.bfloat16)
    dev = A.device
    _need(D, "D", torch.bfloat16, dev)
    _need(group_offsets, "group_offsets", torch.int32, dev)
    M, P = A.shape
    Q = D.shape[1]
    _lib.need_32_bits(E | P | Q | grid, "E, P, Q and grid")
    C_ = torch.empty((E, P, Q), dtype=torch.bfloat16, device=dev)
    _lib.check(_lib.lib().moe_grouped_gemm_wgrad_grid(_ptr(A), _ptr(D), _ptr(group_offsets), E, M, P, Q, _ptr(C_),
                                                      grid, _stream(dev)), "moe_grouped_gemm_wgrad")
    return C_


_SCHED = {"gemm": _lib.MOE_SCHED_GEMM, "swiglu": _lib.MOE_SCHED_GEMM_SWIGLU, "wgrad": _lib.MOE_SCHED_WGRAD}


def tile_schedule(kind: str, group_offsets, M: int, N: int, grid: int, Q: int = 0):
    """Host-side tile list of a persistent grouped GEMM (moe_tile_schedule): int32 array [n, 7] of
    (workgroup, turn, expert, row0, row1, col0, col1). group_offsets: host integer array [E + 1]."""
    import numpy as np

    off = np.ascontiguousarray(group_offsets, dtype=np.int32)
    E = len(off) - 1
    _lib.need_32_bits(N | Q | grid, "N, Q and grid")
    count = C.c_int64(0)
    f = _lib.lib().moe_tile_schedule
    _lib.check(f(_SCHED[kind], off.ctypes.data, E, M, N, Q, grid, None, 0, C.byref(count)), "moe_tile_schedule")
    out = np.empty((count.value, 7), np.int32)
    _lib.check(f(_SCHED[kind], off.ctypes.data, E, M, N, Q, grid, out.ctypes.data if count.value else None,
                 count.value, C.byref(count)), "moe_tile_schedule")
    return out


def combine(ys: torch.Tensor, slot_row: torch.Tensor, topk_w: torch.Tensor | None, T: int, k: int) -> torch.Tensor:
    """y [T, emb] = sum_j topk_w[t,j] ys[slot_row[t*k+j]] (unit weights when topk_w is None)."""
    _need(ys, "ys", torch.bfloat16)
    dev = ys.device
    _need(slot_row, "slot_row", torch.int32, dev)
    _need(topk_w, "topk_w", torch.float32, dev)
    emb = ys.shape[1]
    y = torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    s = _lib.shape(T, emb, 64, max(k, 1), k)
    _lib.check(_lib.lib().moe_combine(C.byref(s), _ptr(ys), _ptr(slot_row), _ptr(topk_w), _ptr(y), _stream(dev)),
               "moe_combine")
    return y


def combine_bwd(dy: torch.Tensor, ys: torch.Tensor | None, slot_row: torch.Tensor, topk_w: torch.Tensor, k: int):
    """(dys [S, emb] bf16, dtopk_w [T, k] fp32 or None when ys is None)."""
    _need(dy, "dy", torch.bfloat16)
    dev = dy.device
    _need(ys, "ys", torch.bfloat16, dev)
    _need(slot_row, "slot_row", torch.int32, dev)
    _need(topk_w, "topk_w", torch.float32, dev)
    T, emb = dy.shape
    dys = torch.empty((T * k, emb), dtype=torch.bfloat16, device=dev)
    dw = torch.empty((T, k), dtype=torch.float32, device=dev) if ys is not None else None
    s = _lib.shape(T, emb, 64, max(k, 1), k)
    _lib.check(_lib.lib().moe_combine_bwd(C.byref(s), _ptr(dy), _ptr(ys), _ptr(slot_row), _ptr(topk_w), _ptr(dys),
                                          _ptr(dw), _stream(dev)), "moe_combine_bwd")
    return dys, dw


_SAVED_NAMES = ("topk_idx", "topk_w", "group_sizes", "group_offsets", "sorted_slot", "slot_row", "xs", "h", "a", "o")


def alloc_saved(T: int, emb: int, mlp: int, E: int, k: int, device, keep_h: bool = True) -> dict:
    """Buffers of one forward pass for the backward; keep_h=False leaves h out (the backward recomputes it)."""
    S = T * k
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    return dict(topk_idx=torch.empty((T, k), dtype=i32, device=device),
                topk_w=torch.empty((T, k), dtype=f32, device=device),
                group_sizes=torch.empty(E, dtype=i32, device=device),
                group_offsets=torch.empty(E + 1, dtype=i32, device=device),
                sorted_slot=torch.empty(S, dtype=i32, device=device),
                slot_row=torch.empty(S, dtype=i32, device=device),
                xs=torch.empty((S, emb), dtype=bf, device=device),
                h=torch.empty((S, 2 * mlp), dtype=f32, device=device) if keep_h else None,
                a=torch.empty((S, mlp), dtype=bf, device=device),
                o=torch.empty((S, emb), dtype=bf, device=device))


def _saved_struct(saved: dict) -> MoeSaved:
    return MoeSaved(*[0 if saved[n] is None else saved[n].data_ptr() for n in _SAVED_NAMES])


def route_bwd(x: torch.Tensor, wr: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
              dtopk_w: torch.Tensor, sorted_slot: torch.Tensor, group_offsets: torch.Tensor,
              dx: torch.Tensor | None = None, want_dbias: bool = True) -> dict:
    """Router gradients with the picks held fixed (see moe_route_bwd): dict(dwr [emb, E] fp32, dbias [E] fp32
    or None). dx (bf16 [T, emb], optional) is updated in place: dx += dlogits . wr^T."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    for t, n, d in ((wr, "wr", torch.float32), (topk_idx, "topk_idx", torch.int32), (topk_w, "topk_w", torch.float32),
                    (dtopk_w, "dtopk_w", torch.float32), (sorted_slot, "sorted_slot", torch.int32),
                    (group_offsets, "group_offsets", torch.int32), (dx, "dx", torch.bfloat16)):
        _need(t, n, d, dev)
    T, emb = x.shape
    E = wr.shape[1]
    k = topk_idx.shape[1]
    s = _lib.shape(T, emb, 64, E, k)
    ws_n = int(_lib.lib().moe_route_bwd_workspace_bytes(C.byref(s)))
    if ws_n == 0:
        _lib.check(_lib.lib().moe_query_support(C.byref(s)), "route_bwd")
    ws = torch.empty(ws_n, dtype=torch.uint8, device=dev)
    dwr = torch.empty((emb, E), dtype=torch.float32, device=dev)
    dbias = torch.empty(E, dtype=torch.float32, device=dev) if want_dbias else None
    _lib.check(_lib.lib().moe_route_bwd(C.byref(s), _ptr(x), _ptr(wr), _ptr(topk_idx), _ptr(topk_w), _ptr(dtopk_w),
                                        _ptr(sorted_slot), _ptr(group_offsets), _ptr(dwr), _ptr(dbias), _ptr(dx),
                                        _ptr(ws), ws.numel(), _stream(dev)), "moe_route_bwd")
    return dict(dwr=dwr, dbias=dbias)


def ffn_fwd(x: torch.Tensor, wi: torch.Tensor, wo: torch.Tensor, k: int, wr: torch.Tensor | None = None,
            bias: torch.Tensor | None = None, logits: torch.Tensor | None = None, save: bool = False,
            workspace: torch.Tensor | None = None, out: torch.Tensor | None = None, keep_h: bool = True):
    """MoE FFN forward. Returns (y [T, emb] bf16, saved dict or None). With save and keep_h=False the
    saved set has no h, and ffn_bwd recomputes it."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    for t, n, d in ((wi, "wi", torch.bfloat16), (wo, "wo", torch.bfloat16), (wr, "wr", torch.float32),
                    (bias, "bias", torch.float32), (logits, "logits", torch.float32)):
        _need(t, n, d, dev)
    T, emb = x.shape
    E, _, n2 = wi.shape
    mlp = n2 // 2
    s = _lib.shape(T, emb, mlp, E, k)
    ws_n = int(_lib.lib().moe_workspace_bytes(C.byref(s), 0))
    if ws_n == 0:
        _lib.check(_lib.lib().moe_query_support(C.byref(s)), "ffn_fwd")
    ws = workspace if workspace is not None and workspace.numel() >= ws_n else \
        torch.empty(ws_n, dtype=torch.uint8, device=dev)
    y = out if out is not None else torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    saved = alloc_saved(T, emb, mlp, E, k, dev, keep_h=keep_h) if save else None
    sv = C.byref(_saved_struct(saved)) if save else None
    _lib.check(_lib.lib().moe_ffn_fwd(C.byref(s), _ptr(x), _ptr(wr), _ptr(bias), _ptr(logits), _ptr(wi), _ptr(wo),
                                      _ptr(y), sv, _ptr(ws), ws.numel(), _stream(dev)), "moe_ffn_fwd")
    return y, saved


def ffn_bwd(dy: torch.Tensor, saved: dict, wi: torch.Tensor, wo: torch.Tensor, k: int,
            need=("dx", "dwi", "dwo", "dtopk_w"), workspace: torch.Tensor | None = None) -> dict:
    """MoE FFN backward with the routing held fixed; returns the requested gradients."""
    _need(dy, "dy", torch.bfloat16)
    dev = dy.device
    _need(wi, "wi", torch.bfloat16, dev)
    _need(wo, "wo", torch.bfloat16, dev)
    T, emb = dy.shape
    E, _, n2 = wi.shape
    mlp = n2 // 2
    s = _lib.shape(T, emb, mlp, E, k)
    ws_n = int(_lib.lib().moe_workspace_bytes(C.byref(s), 2 if saved.get("h") is None else 1))
    if ws_n == 0:
        _lib.check(_lib.lib().moe_query_support(C.byref(s)), "ffn_bwd")
    ws = workspace if workspace is not None and workspace.numel() >= ws_n else \
        torch.empty(ws_n, dtype=torch.uint8, device=dev)
    g = {}
    if "dx" in need:
        g["dx"] = torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    if "dwi" in need:
        g["dwi"] = torch.empty((E, emb, 2 * mlp), dtype=torch.bfloat16, device=dev)
    if "dwo" in need:
        g["dwo"] = torch.empty((E, mlp, emb), dtype=torch.bfloat16, device=dev)
    if "dtopk_w" in need:
        g["dtopk_w"] = torch.empty((T, k), dtype=torch.float32, device=dev)
    _lib.check(_lib.lib().moe_ffn_bwd(C.byref(s), _ptr(dy), C.byref(_saved_struct(saved)), _ptr(wi), _ptr(wo),
                                      _ptr(g.get("dx")), _ptr(g.get("dwi")), _ptr(g.get("dwo")),
                                      _ptr(g.get("dtopk_w")), _ptr(ws), ws.numel(), _stream(dev)), "moe_ffn_bwd")
    return g


def mx_quantize_rows(src: torch.Tensor, row_index: torch.Tensor | None = None, row_div: int = 1,
                     rows: int | None = None):
    """MXFP8 of rows of src [R, K] bf16 (see moe_mx_quantize_rows): (codes [M, K] uint8, scales [K/64, M, 4]
    uint8). With row_index, output row r is source row row_index[r] // row_div."""
    _need(src, "src", torch.bfloat16)
    dev = src.device
    _need(row_index, "row_index", torch.int32, dev)
    R, K = src.shape
    _lib.need_32_bits(K | row_div, "a row's length and row_div")
    M = rows if rows is not None else (row_index.numel() if row_index is not None else R)
    codes = torch.empty((M, K), dtype=torch.uint8, device=dev)
    scales = torch.empty((K // 64, M, 4), dtype=torch.uint8, device=dev)
    _lib.check(_lib.lib().moe_mx_quantize_rows(_ptr(src), R, K, _ptr(row_index), row_div, M, _ptr(codes),
                                               _ptr(scales), _stream(dev)), "moe_mx_quantize_rows")
    return codes, scales


def mx_quantize_weight(w: torch.Tensor):
    """MXFP8 of expert weights w [E, K, N] bf16 along K, transposed (see moe_mx_quantize_weight):
    (codes [E, N, K] uint8, scales [E, K/64, N, 4] uint8)."""
    _need(w, "w", torch.bfloat16)
    E, K, N = w.shape
    _lib.need_32_bits(E | K | N, "E, K and N")
    codes = torch.empty((E, N, K), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, K // 64, N, 4), dtype=torch.uint8, device=w.device)
    _lib.check(_lib.lib().moe_mx_quantize_weight(_ptr(w), E, K, N, _ptr(codes), _ptr(scales), _stream(w.device)),
               "moe_mx_quantize_weight")
    return codes, scales


def grouped_gemm_mx(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                    group_offsets: torch.Tensor, epilogue: str = "none", out: torch.Tensor | None = None,
                    row_slot: torch.Tensor | None = None, slot_div: int = 1, rows: int | None = None,
                    mx_out: bool = False, bf16_out: bool = True):
    """Grouped GEMM on MXFP8 operands (see moe_grouped_gemm_mx): a_codes [a_rows, K] with a_scales
    [K/64, a_rows, 4] from mx_quantize_rows, b_codes [E, N, K] with b_scales [E, K/64, N, 4] from
    mx_quantize_weight. With row_slot, output row r reads A row row_slot[r] // slot_div (rows = number of
    output rows, default row_slot's length). Returns C [M, N] bf16, or [M, N/2] for epilogue "swiglu"; with
    mx_out (SwiGLU only) returns (C or None, codes [M, N/2], scales [N/128, M, 4]) of the MXFP8 output."""
    dev = a_codes.device
    for t, n in ((a_codes, "a_codes"), (a_scales, "a_scales"), (b_codes, "b_codes"), (b_scales, "b_scales")):
        _need(t, n, torch.uint8, dev)
    _need(group_offsets, "group_offsets", torch.int32, dev)
    _need(row_slot, "row_slot", torch.int32, dev)
    a_rows, K = a_codes.shape
    M = a_rows if row_slot is None else (rows if rows is not None else row_slot.numel())
    E, N, _ = b_codes.shape
    _lib.need_32_bits(E | K | N | slot_div, "E, K, N and slot_div")
    epi = {"none": 0, "swiglu": 1}[epilogue]
    width = N if epi == 0 else N // 2
    C_ = (out if out is not None else torch.empty((M, width), dtype=torch.bfloat16, device=dev)) if bf16_out \
        else None
    cq = torch.empty((M, width), dtype=torch.uint8, device=dev) if mx_out else None
    cqs = torch.zeros((width // 64, M, 4), dtype=torch.uint8, device=dev) if mx_out else None
    _lib.check(_lib.lib().moe_grouped_gemm_mx(epi, _ptr(a_codes), _ptr(a_scales), a_rows, _ptr(row_slot), slot_div,
                                              _ptr(b_codes), _ptr(b_scales), _ptr(group_offsets), E, M, K, N,
                                              _ptr(C_), _ptr(cq), _ptr(cqs), _stream(dev)),
               "moe_grouped_gemm_mx")
    return (C_, cq, cqs) if mx_out else C_


def mx_quantize_expert_weights(wi: torch.Tensor, wo: torch.Tensor) -> dict:
    """Weight preparation for ffn_fwd_mx: the MXFP8 codes and scales of wi and wo along their K."""
    wic, wis = mx_quantize_weight(wi)
    woc, wos = mx_quantize_weight(wo)
    return dict(wi_codes=wic, wi_scales=wis, wo_codes=woc, wo_scales=wos, mlp=wi.shape[2] // 2)


def ffn_fwd_mx(x: torch.Tensor, wq: dict, k: int, wr: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               logits: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """MoE FFN forward with MXFP8 grouped GEMMs (see moe_ffn_fwd_mx); wq from mx_quantize_expert_weights."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    for t, n, d in ((wr, "wr", torch.float32), (bias, "bias", torch.float32), (logits, "logits", torch.float32)):
        _need(t, n, d, dev)
    T, emb = x.shape
    E = wq["wi_codes"].shape[0]
    mlp = wq["mlp"]
    s = _lib.shape(T, emb, mlp, E, k)
    ws_n = int(_lib.lib().moe_workspace_bytes_mx(C.byref(s)))
    if ws_n == 0:
        _lib.check(_lib.lib().moe_query_support(C.byref(s)), "ffn_fwd_mx")
        raise _lib.MoeError(_lib.MOE_ERR_UNSUPPORTED, "ffn_fwd_mx", "mlp must be a multiple of 64")
    ws = workspace if workspace is not None and workspace.numel() >= ws_n else \
        torch.empty(ws_n, dtype=torch.uint8, device=dev)
    y = out if out is not None else torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    _lib.check(_lib.lib().moe_ffn_fwd_mx(C.byref(s), _ptr(x), _ptr(wr), _ptr(bias), _ptr(logits),
                                         _ptr(wq["wi_codes"]), _ptr(wq["wi_scales"]), _ptr(wq["wo_codes"]),
                                         _ptr(wq["wo_scales"]), _ptr(y), _ptr(ws), ws.numel(), _stream(dev)),
               "moe_ffn_fwd_mx")
    return y


_SCORE = {"softmax": _lib.MOE_SCORE_SOFTMAX, "sigmoid": _lib.MOE_SCORE_SIGMOID}
_TYPE = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16}


def _need_like(t, name, shape, dtype, device):
    """_need, with the shape checked too (the kernels index by the sizes they are given)."""
    if t is None or (type(t) is torch.Tensor and t.dtype is dtype and t.device == device and t.is_contiguous()
                     and t.shape == shape):
        return
    _need(t, name, dtype, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_typed(t, name, ndim):
    """A contiguous float32 or bfloat16 device tensor of ndim dimensions; returns its MOE_* type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    ty = _TYPE.get(t.dtype)
    if ty is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    if not (t.is_cuda and t.is_contiguous()):
        _need(t, name, t.dtype)
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    return ty


def _need_rank2(t, name, dtype, device):
    _need(t, name, dtype, device)
    if t is None or t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {None if t is None else tuple(t.shape)}")


@functools.lru_cache(maxsize=None)
def _entry(fn):
    return getattr(_lib.lib(), fn)


def _call(fn, dev, *args):
    """Library call `fn` on dev's current stream, with dev current: tensors pass as pointers, None as NULL."""
    i = dev.index
    if i != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(fn, dev, *args)
    stream = _raw_stream(i) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    status = _entry(fn)(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args], stream)
    if status != _lib.MOE_OK:
        _lib.check(status, fn)


def _call_raw(fn, dev, *args):
    """_call with pointers for tensors already: the short way for the calls of a decode step."""
    i = dev.index
    if i != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call_raw(fn, dev, *args)
    stream = _raw_stream(i) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    status = _entry(fn)(*args, stream)
    if status != _lib.MOE_OK:
        _lib.check(status, fn)


def _at(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=256)
def _route_shape(T, E, k):
    return C.byref(_lib.shape(T, 64, 64, E, k))


@functools.lru_cache(maxsize=256)
def _router(score, n_group, topk_group, group_top, renorm, scale):
    if score not in _SCORE:
        raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}")
    _lib.need_32_bits(n_group | topk_group | group_top, "n_group, topk_group and group_top")
    return C.byref(_lib.MoeRouter(_SCORE[score], n_group, topk_group, group_top, renorm, scale))


def route_scored(k: int, logits: torch.Tensor, balance_bias: torch.Tensor | None = None, score: str = "softmax",
                 n_group: int = 1, topk_group: int = 1, group_top: int = 1, renorm: bool = True,
                 scale: float = 1.0):
    """Routing by scores (see moe_route_scored): (topk_idx [T, k] int32, topk_w [T, k] fp32) of logits [T, E]
    fp32 or bf16. balance_bias [E] fp32 steers the choice and leaves the weights alone; with topk_group < n_group
    the picks come from the topk_group groups of the largest sums of their group_top best choice values."""
    ty = _need_typed(logits, "logits", 2)
    dev = logits.device
    T, E = logits.shape
    _need_like(balance_bias, "balance_bias", (E,), torch.float32, dev)
    # plain numbers, as the structures below are kept by value
    k = operator.index(k)
    r = _router(score, operator.index(n_group), operator.index(topk_group), operator.index(group_top), bool(renorm),
                float(scale))
    s = _route_shape(T, E, k)
    kk = k if k > 0 else 0  # a k <= 0 is the library's to refuse
    idx = torch.empty((T, kk), dtype=torch.int32, device=dev)
    w = torch.empty((T, kk), dtype=torch.float32, device=dev)
    _call("moe_route_scored", dev, s, r, logits, ty, balance_bias, idx, w)
    return idx, w


def route_scored_bwd(logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, dtopk_w: torch.Tensor,
                     score: str = "softmax", renorm: bool = True, scale: float = 1.0) -> torch.Tensor:
    """dlogits [T, E], of the logits' type, from the gradient of route_scored's weights (moe_route_scored_bwd);
    score, renorm and scale as in the forward."""
    ty = _need_typed(logits, "logits", 2)
    dev = logits.device
    T, E = logits.shape
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        _need_rank2(topk_idx, "topk_idx", torch.int32, dev)
    shape = (T, topk_idx.shape[1])
    _need_like(topk_idx, "topk_idx", shape, torch.int32, dev)
    _need_like(topk_w, "topk_w", shape, torch.float32, dev)
    _need_like(dtopk_w, "dtopk_w", shape, torch.float32, dev)
    k = shape[1]
    d = torch.empty_like(logits)
    _call("moe_route_scored_bwd", dev, _route_shape(T, E, k), _router(score, 1, 1, 1, bool(renorm), float(scale)), logits, ty,
          topk_idx, topk_w, dtopk_w, d)
    return d


def ckpt_quantize(src: torch.Tensor):
    """8-bit checkpoint of rows src [M, K] fp32 or bf16 (see moe_ckpt_quantize): (codes [M, K] int8,
    scales [M, K/32] uint8). K must be a multiple of 32."""
    ty = _need_typed(src, "src", 2)
    dev = src.device
    M, K = src.shape
    _lib.need_32_bits(K, "a row's length")
    codes = torch.empty((M, K), dtype=torch.int8, device=dev)
    scales = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
    _call("moe_ckpt_quantize", dev, src, ty, M, K, codes, scales)
    return codes, scales


def _need_ckpt(codes, scales, name, dev):
    """An 8-bit checkpoint: codes [M, K] and scales [M, K/32] of one device."""
    _need_rank2(codes, f"{name}codes", torch.int8, dev)
    M, K = codes.shape
    if scales is None:
        raise ValueError(f"{name}scales is missing")
    _need_like(scales, f"{name}scales", (M, K // 32), torch.uint8, codes.device)


def ckpt_dequantize(codes: torch.Tensor, scales: torch.Tensor, row_index: torch.Tensor | None = None,
                    row_div: int = 1, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Values of an 8-bit checkpoint as rows [M, K] of dtype (bf16 holds them exactly); with row_index [M] int32,
    row r is checkpoint row row_index[r] // row_div (see moe_ckpt_dequantize)."""
    _need_ckpt(codes, scales, "", None)
    dev = codes.device
    if dtype not in _TYPE:
        raise TypeError(f"dtype must be torch.float32 or torch.bfloat16, got {dtype}")
    R, K = codes.shape
    _lib.need_32_bits(K | row_div, "a row's length and row_div")
    M = R
    if row_index is not None:
        M = row_index.numel()
        _need_like(row_index, "row_index", (M,), torch.int32, dev)
    dst = torch.empty((M, K), dtype=dtype, device=dev)
    _call("moe_ckpt_dequantize", dev, codes, scales, R, K, row_index, row_div, M, dst, _TYPE[dtype])
    return dst


def swiglu_bwd_ckpt(da: torch.Tensor, h_codes: torch.Tensor, h_scales: torch.Tensor,
                    row_slot: torch.Tensor | None = None, slot_scale: torch.Tensor | None = None,
                    want_a: bool = True, want_dscale: bool = True):
    """SwiGLU backward from an 8-bit h (see moe_swiglu_bwd_ckpt): (dh [M, 2*mlp] bf16, a [M, mlp] bf16 or None,
    dslot_scale [M] fp32 or None) from da [M, mlp] bf16; row_slot [M] int32 maps rows to entries of slot_scale [M]
    and dslot_scale."""
    _need_rank2(da, "da", torch.bfloat16, None)
    dev = da.device
    M, mlp = da.shape
    _lib.need_32_bits(mlp, "mlp")
    if h_codes is None or h_scales is None:
        raise ValueError("h_codes or h_scales is missing")
    _need_like(h_codes, "h_codes", (M, 2 * mlp), torch.int8, dev)
    _need_like(h_scales, "h_scales", (M, mlp // 16), torch.uint8, dev)
    _need_like(row_slot, "row_slot", (M,), torch.int32, dev)
    _need_like(slot_scale, "slot_scale", (M,), torch.float32, dev)
    dh = torch.empty((M, 2 * mlp), dtype=torch.bfloat16, device=dev)
    a = torch.empty_like(da) if want_a else None
    ds = torch.empty(M, dtype=torch.float32, device=dev) if want_dscale else None
    _call("moe_swiglu_bwd_ckpt", dev, M, mlp, da, h_codes, h_scales, row_slot, slot_scale, dh, a, ds)
    return dh, a, ds


def grouped_gemm_wgrad_ckpt(a_codes: torch.Tensor, a_scales: torch.Tensor, D: torch.Tensor,
                            group_offsets: torch.Tensor, E: int, row_slot: torch.Tensor | None = None,
                            slot_div: int = 1, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C [E, P, Q] = per-group X^T D with X an 8-bit checkpoint [R, P] (see moe_grouped_gemm_wgrad_ckpt); with
    row_slot [M] int32, row r of the product reads X row row_slot[r] // slot_div. workspace: uint8, by default a new
    one of moe_wgrad_ckpt_workspace_bytes; a smaller one only cuts fewer long groups."""
    _need_ckpt(a_codes, a_scales, "a_", None)
    dev = a_codes.device
    _need_rank2(D, "D", torch.bfloat16, dev)
    M, Q = D.shape
    R, P = a_codes.shape
    _lib.need_32_bits(E | P | Q | slot_div, "E, P, Q and slot_div")
    _need_like(row_slot, "row_slot", (M,), torch.int32, dev)
    if group_offsets is None:
        raise ValueError("group_offsets is missing")
    _need_like(group_offsets, "group_offsets", (E + 1,), torch.int32, dev)
    ws = _workspace(workspace, int(_lib.lib().moe_wgrad_ckpt_workspace_bytes(E, M, P, Q)), dev)
    C_ = torch.empty((max(E, 0), P, Q), dtype=torch.bfloat16, device=dev)
    _call("moe_grouped_gemm_wgrad_ckpt", dev, a_codes, a_scales, R, row_slot, slot_div, D, group_offsets, E, M, P, Q,
          C_, ws, ws.numel())
    return C_


_SAVED8_NAMES = ("group_sizes", "group_offsets", "sorted_slot", "slot_row", "x_codes", "x_scales", "h_codes",
                 "h_scales")


def alloc_saved8(T: int, emb: int, mlp: int, E: int, k: int, device) -> dict:
    """Buffers of one forward pass in 8 bits, for ffn_bwd_ckpt."""
    S = T * k
    i32, i8, u8 = torch.int32, torch.int8, torch.uint8
    return dict(group_sizes=torch.empty(E, dtype=i32, device=device),
                group_offsets=torch.empty(E + 1, dtype=i32, device=device),
                sorted_slot=torch.empty(S, dtype=i32, device=device),
                slot_row=torch.empty(S, dtype=i32, device=device),
                x_codes=torch.empty((T, emb), dtype=i8, device=device),
                x_scales=torch.empty((T, emb // 32), dtype=u8, device=device),
                h_codes=torch.empty((S, 2 * mlp), dtype=i8, device=device),
                h_scales=torch.empty((S, mlp // 16), dtype=u8, device=device))


def _layer_sizes(wi, wo, emb, dev):
    """(E, mlp) of a layer's weights wi [E, emb, 2*mlp], wo [E, mlp, emb]."""
    _need(wi, "wi", torch.bfloat16, dev)
    if wi is None or wi.dim() != 3 or wi.shape[1] != emb or wi.shape[2] % 2:
        raise ValueError(f"wi must have shape [E, {emb}, 2*mlp], got {None if wi is None else tuple(wi.shape)}")
    E, mlp = wi.shape[0], wi.shape[2] // 2
    if wo is None:
        raise ValueError("wo is missing")
    _need_like(wo, "wo", (E, mlp, emb), torch.bfloat16, dev)
    return E, mlp


def _workspace(workspace, n, dev):
    """The caller's workspace, checked, or a new one of n bytes."""
    if workspace is None:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    return workspace


def ffn_fwd_routed(x: torch.Tensor, wi: torch.Tensor, wo: torch.Tensor, topk_idx: torch.Tensor,
                   topk_w: torch.Tensor, save: str | None = None, keep_h: bool = True,
                   workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """MoE FFN forward on a given routing (route, route_scored, or the caller's own): (y [T, emb] bf16, saved dict
    or None). save: None, "full" (the set ffn_bwd takes; keep_h as in ffn_fwd) or "int8" (the set ffn_bwd_ckpt
    takes); a set holds topk_idx and topk_w themselves, not copies. workspace: uint8 of at least workspace_bytes_routed(...) bytes."""
    if save not in (None, "full", "int8"):
        raise ValueError(f'save must be None, "full" or "int8", got {save!r}')
    _need_rank2(x, "x", torch.bfloat16, None)
    dev = x.device
    T, emb = x.shape
    E, mlp = _layer_sizes(wi, wo, emb, dev)
    _need_rank2(topk_idx, "topk_idx", torch.int32, dev)
    k = topk_idx.shape[1]
    for t, n, d in ((topk_idx, "topk_idx", torch.int32), (topk_w, "topk_w", torch.float32)):
        if t is None:
            raise ValueError(f"{n} is missing")
        _need_like(t, n, (T, k), d, dev)
    _need_like(out, "out", (T, emb), torch.bfloat16, dev)
    s = _lib.shape(T, emb, mlp, E, k)
    _lib.check(_lib.lib().moe_query_support(C.byref(s)), "ffn_fwd_routed")
    ws = _workspace(workspace, int(_lib.lib().moe_workspace_bytes_routed(C.byref(s), 0)), dev)
    y = out if out is not None else torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    saved = full = int8 = None
    if save == "full":
        saved = alloc_saved(T, emb, mlp, E, k, dev, keep_h=keep_h)
        saved["topk_idx"], saved["topk_w"] = topk_idx, topk_w
        full = C.byref(_saved_struct(saved))
    elif save == "int8":
        saved = alloc_saved8(T, emb, mlp, E, k, dev)
        saved["topk_idx"], saved["topk_w"] = topk_idx, topk_w
        int8 = C.byref(_lib.MoeSaved8(*[saved[n].data_ptr() for n in _SAVED8_NAMES]))
    _call("moe_ffn_fwd_routed", dev, C.byref(s), x, topk_idx, topk_w, wi, wo, y, full, int8, ws, ws.numel())
    return y, saved


def ffn_bwd_ckpt(dy: torch.Tensor, saved: dict, wi: torch.Tensor, wo: torch.Tensor,
                 need=("dx", "dwi", "dwo", "dtopk_w"), workspace: torch.Tensor | None = None) -> dict:
    """MoE FFN backward from the 8-bit set of ffn_fwd_routed(save="int8"), the routing held fixed; returns the
    requested gradients, as ffn_bwd does. workspace: uint8 of at least workspace_bytes_routed(..., backward=True)
    bytes."""
    _need_rank2(dy, "dy", torch.bfloat16, None)
    dev = dy.device
    T, emb = dy.shape
    E, mlp = _layer_sizes(wi, wo, emb, dev)
    _need_rank2(saved["topk_w"], "topk_w", torch.float32, dev)
    k = saved["topk_w"].shape[1]
    S = T * k
    s = _lib.shape(T, emb, mlp, E, k)
    _lib.check(_lib.lib().moe_query_support(C.byref(s)), "ffn_bwd_ckpt")
    for n, shape, d in (("topk_w", (T, k), torch.float32), ("group_sizes", (E,), torch.int32),
                        ("group_offsets", (E + 1,), torch.int32), ("sorted_slot", (S,), torch.int32),
                        ("slot_row", (S,), torch.int32), ("x_codes", (T, emb), torch.int8),
                        ("x_scales", (T, emb // 32), torch.uint8), ("h_codes", (S, 2 * mlp), torch.int8),
                        ("h_scales", (S, mlp // 16), torch.uint8)):
        _need_like(saved[n], n, shape, d, dev)
    g = {}
    if "dx" in need:
        g["dx"] = torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    if "dwi" in need:
        g["dwi"] = torch.empty((E, emb, 2 * mlp), dtype=torch.bfloat16, device=dev)
    if "dwo" in need:
        g["dwo"] = torch.empty((E, mlp, emb), dtype=torch.bfloat16, device=dev)
    if "dtopk_w" in need:
        g["dtopk_w"] = torch.empty((T, k), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, int(_lib.lib().moe_workspace_bytes_routed(C.byref(s), 1)), dev)
    _call("moe_ffn_bwd_ckpt", dev, C.byref(s), dy, saved["topk_w"],
          C.byref(_lib.MoeSaved8(*[saved[n].data_ptr() for n in _SAVED8_NAMES])), wi, wo, g.get("dx"), g.get("dwi"),
          g.get("dwo"), g.get("dtopk_w"), ws, ws.numel())
    return g


def workspace_bytes_routed(T: int, emb: int, mlp: int, E: int, k: int, backward: bool = False) -> int:
    """Workspace bytes of ffn_fwd_routed, or of ffn_bwd_ckpt with backward."""
    s = _lib.shape(T, emb, mlp, E, k)
    return int(_lib.lib().moe_workspace_bytes_routed(C.byref(s), int(backward)))


FEW_MAX_TOKENS = 64  # most tokens of ffn_fwd_few and ffn_fwd_few_mx


@functools.lru_cache(maxsize=256)
def _few_plan(T, emb, mlp, E, k):
    """The shape structure and the workspace bytes of a few-token call."""
    s = _lib.shape(T, emb, mlp, E, k)
    n = int(_lib.lib().moe_workspace_bytes_few(C.byref(s)))
    return C.byref(s), n


def workspace_bytes_few(T: int, emb: int, mlp: int, E: int, k: int) -> int:
    """Workspace bytes of ffn_fwd_few and ffn_fwd_few_mx (0: unsupported shape)."""
    return _few_plan(T, emb, mlp, E, k)[1]


def _few(fn, x, weights, mlp, E, k, wr, bias, topk_idx, topk_w, workspace, out):
    dev = x.device
    T, emb = x.shape
    if wr is not None:
        if topk_idx is not None or topk_w is not None:
            raise ValueError("either wr or topk_idx and topk_w must be given, not both")
        if k is None:
            raise ValueError("k is missing")
        k = operator.index(k)
        _need_like(wr, "wr", (emb, E), torch.float32, dev)
        _need_like(bias, "bias", (E,), torch.float32, dev)
        topk_idx = torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev)
        topk_w = torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev)
    else:
        if topk_idx is None or topk_w is None:
            raise ValueError("wr, or topk_idx and topk_w, must be given")
        if bias is not None:
            raise ValueError("bias is the router's: with topk_idx and topk_w it must be None")
        _need_rank2(topk_idx, "topk_idx", torch.int32, dev)
        if k is not None and k != topk_idx.shape[1]:
            raise ValueError(f"k is {k}, topk_idx has {topk_idx.shape[1]} picks")
        k = topk_idx.shape[1]
        _need_like(topk_idx, "topk_idx", (T, k), torch.int32, dev)
        _need_like(topk_w, "topk_w", (T, k), torch.float32, dev)
    _need_like(out, "out", (T, emb), torch.bfloat16, dev)
    s, n = _few_plan(T, emb, mlp, E, k)
    ws = _workspace(workspace, n, dev)
    y = out if out is not None else torch.empty((T, emb), dtype=torch.bfloat16, device=dev)
    _call_raw(fn, dev, s, x.data_ptr(), _at(wr), _at(bias), topk_idx.data_ptr(), topk_w.data_ptr(),
              *[w.data_ptr() for w in weights], y.data_ptr(), ws.data_ptr(), ws.numel())
    return y, topk_idx, topk_w


def ffn_fwd_few(x: torch.Tensor, wi: torch.Tensor, wo: torch.Tensor, k: int | None = None,
                wr: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The whole layer for a few tokens, at most FEW_MAX_TOKENS (see moe_ffn_fwd_few): (y [T, emb] bf16, topk_idx
    [T, k] int32, topk_w [T, k] fp32). Either k and wr [emb, E] fp32 (+ bias [E] fp32), or a routing topk_idx,
    topk_w, which then comes back as it is. workspace: uint8 of at least workspace_bytes_few(...) bytes."""
    _need_rank2(x, "x", torch.bfloat16, None)
    E, mlp = _layer_sizes(wi, wo, x.shape[1], x.device)
    return _few("moe_ffn_fwd_few", x, (wi, wo), mlp, E, k, wr, bias, topk_idx, topk_w, workspace, out)


def ffn_fwd_few_mx(x: torch.Tensor, wq: dict, k: int | None = None, wr: torch.Tensor | None = None,
                   bias: torch.Tensor | None = None, topk_idx: torch.Tensor | None = None,
                   topk_w: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   out: torch.Tensor | None = None):
    """ffn_fwd_few on MXFP8 weights wq from mx_quantize_expert_weights (see moe_ffn_fwd_few_mx): x and the SwiGLU
    output are not quantized."""
    _need_rank2(x, "x", torch.bfloat16, None)
    dev, emb, mlp = x.device, x.shape[1], operator.index(wq["mlp"])
    _need(wq["wi_codes"], "wi_codes", torch.uint8, dev)
    E = wq["wi_codes"].shape[0]
    for n, shape in (("wi_codes", (E, 2 * mlp, emb)), ("wi_scales", (E, emb // 64, 2 * mlp, 4)),
                     ("wo_codes", (E, emb, mlp)), ("wo_scales", (E, mlp // 64, emb, 4))):
        if wq[n] is None:
            raise ValueError(f"{n} is missing")
        _need_like(wq[n], n, shape, torch.uint8, dev)
    return _few("moe_ffn_fwd_few_mx", x, (wq["wi_codes"], wq["wi_scales"], wq["wo_codes"], wq["wo_scales"]), mlp, E, k,
                wr, bias, topk_idx, topk_w, workspace, out)


def _weight_type(t, name, emb, dev):
    """MOE_* type of a norm's weight [emb] (fp32 without one)."""
    if t is None:
        return _lib.MOE_F32
    if type(t) is torch.Tensor and t.device == dev and t.is_contiguous() and t.shape == (emb,):
        ty = _TYPE.get(t.dtype)
        if ty is not None:
            return ty
    ty = _need_typed(t, name, 1)
    _need_like(t, name, (emb,), t.dtype, dev)
    return ty


def _bf16_like(t):
    return torch.empty_like(t) if t.dtype is torch.bfloat16 else torch.empty_like(t, dtype=torch.bfloat16)


def norm(x: torch.Tensor, weight: torch.Tensor | None = None, offset: float = 0.0, eps: float = 1e-6,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * (offset + weight) over rows [T, emb] fp32 or bf16, as bf16 (see moe_norm);
    weight [emb] fp32 or bf16, or None."""
    ty = _need_typed(x, "x", 2)
    dev = x.device
    T, emb = x.shape
    _lib.need_32_bits(emb, "emb")
    wt = _weight_type(weight, "weight", emb, dev)
    _need_like(out, "out", (T, emb), torch.bfloat16, dev)
    y = out if out is not None else _bf16_like(x)
    _call_raw("moe_norm", dev, T, emb, x.data_ptr(), ty, _at(weight), wt, offset, eps, y.data_ptr())
    return y


def norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None = None, offset: float = 0.0,
             eps: float = 1e-6, dres: torch.Tensor | None = None, want_dweight: bool = True,
             workspace: torch.Tensor | None = None):
    """Gradients of norm from dy [T, emb] bf16 (see moe_norm_bwd): (dx of x's type, dweight [emb] fp32 or None).
    dres, of x's type, is the gradient that reaches x on the residual stream: it is added."""
    ty = _need_typed(x, "x", 2)
    dev = x.device
    T, emb = x.shape
    _lib.need_32_bits(emb, "emb")
    wt = _weight_type(weight, "weight", emb, dev)
    if dy is None:
        raise ValueError("dy is missing")
    _need_like(dy, "dy", (T, emb), torch.bfloat16, dev)
    _need_like(dres, "dres", (T, emb), x.dtype, dev)
    dx = torch.empty_like(x)
    dw = ws = None
    if weight is not None and want_dweight:
        dw = torch.empty(emb, dtype=torch.float32, device=dev)
        ws = _workspace(workspace, int(_lib.lib().moe_norm_bwd_workspace_bytes(T, emb)), dev)
    _call("moe_norm_bwd", dev, T, emb, dy, x, ty, weight, wt, offset, eps, dres, dx, dw, ws,
          0 if ws is None else ws.numel())
    return dx, dw


_BLOCK = struct.Struct("@5i4f3P")  # moe_block_t (packed: a third of the time that filling a ctypes structure takes)


def _block(x_type, T, emb, dev, post_norm, post_weight, gate, scale, res_scale, next_weight, offset, eps):
    """The structure of a block_out call, and the gate's mode."""
    _lib.need_32_bits(emb, "emb")
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight without post_norm")
    wt = _weight_type(post_weight, "post_weight", emb, dev)
    nt = _weight_type(next_weight, "next_weight", emb, dev)
    if post_weight is not None and next_weight is not None and wt != nt:
        raise TypeError("post_weight and next_weight must have one type")
    mode, gt = _lib.MOE_GATE_NONE, _lib.MOE_F32
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch.Tensor")
        gt = _need_typed(gate, "gate", 1 if gate.dim() == 1 else 2)
        shape = tuple(gate.shape)
        mode = {(emb,): _lib.MOE_GATE_CHANNEL, (T, 1): _lib.MOE_GATE_TOKEN, (T, emb): _lib.MOE_GATE_FULL}.get(shape)
        if mode is None:
            raise ValueError(f"gate must have shape ({emb},), ({T}, 1) or ({T}, {emb}), got {shape}")
        _need_like(gate, "gate", shape, gate.dtype, dev)
    return _BLOCK.pack(x_type, nt if post_weight is None else wt, mode, gt, 1 if post_norm else 0, offset, eps, scale,
                       res_scale, 0 if post_weight is None else post_weight.data_ptr(),
                       0 if next_weight is None else next_weight.data_ptr(), 0 if gate is None else gate.data_ptr()), mode


def block_out(res: torch.Tensor, y: torch.Tensor | None = None, ys: torch.Tensor | None = None,
              slot_row: torch.Tensor | None = None, topk_w: torch.Tensor | None = None, post_norm: bool = False,
              post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
              res_scale: float = 1.0, next_norm: bool = False, next_weight: torch.Tensor | None = None,
              offset: float = 0.0, eps: float = 1e-6, want_y: bool = False, out: torch.Tensor | None = None) -> dict:
    """What follows the layer in a block (see moe_block_out): dict(out = res_scale * res + scale * gate * z, of res's
    type; xn = norm(out) bf16 with next_norm, else None; y bf16 with want_y, else None), z = norm(y) with post_norm,
    else y. The layer's output is y [T, emb] bf16, or the weighted sum of its expert rows ys [T*k, emb] through
    slot_row [T*k] and topk_w [T, k] (as combine). gate: [emb], [T, 1] or [T, emb], fp32 or bf16. out may be res."""
    ty = _need_typed(res, "res", 2)
    dev = res.device
    T, emb = res.shape
    if next_weight is not None and not next_norm:
        raise ValueError("next_weight without next_norm")
    b, _ = _block(ty, T, emb, dev, post_norm, post_weight, gate, float(scale), float(res_scale), next_weight,
                  float(offset), float(eps))
    k = 0
    if y is not None:
        if ys is not None or slot_row is not None or topk_w is not None or want_y:
            raise ValueError("either y or ys, slot_row and topk_w must be given, not both (nor want_y with y)")
        _need_like(y, "y", (T, emb), torch.bfloat16, dev)
    else:
        if ys is None or slot_row is None or topk_w is None:
            raise ValueError("y, or ys, slot_row and topk_w, must be given")
        _need_rank2(topk_w, "topk_w", torch.float32, dev)
        k = topk_w.shape[1]
        _need_like(topk_w, "topk_w", (T, k), torch.float32, dev)
        _need_like(ys, "ys", (T * k, emb), torch.bfloat16, dev)
        _need_like(slot_row, "slot_row", (T * k,), torch.int32, dev)
    _need_like(out, "out", (T, emb), res.dtype, dev)
    o = out if out is not None else torch.empty_like(res)
    xn = _bf16_like(res) if next_norm else None
    yo = _bf16_like(res) if want_y else None
    _call_raw("moe_block_out", dev, T, emb, b, res.data_ptr(), _at(y), k, _at(ys), _at(slot_row), _at(topk_w),
              o.data_ptr(), _at(xn), _at(yo))
    return dict(out=o, xn=xn, y=yo)


def block_out_bwd(dout: torch.Tensor | None, y: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  dxn: torch.Tensor | None = None, post_norm: bool = False, post_weight: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, scale: float = 1.0, res_scale: float = 1.0,
                  next_norm: bool = False, next_weight: torch.Tensor | None = None, offset: float = 0.0,
                  eps: float = 1e-6, need=("dres", "dy", "dpost_weight", "dgate", "dnext_weight"),
                  workspace: torch.Tensor | None = None) -> dict:
    """Gradients of block_out (see moe_block_out_bwd) from dout (of the residual's type, or None) and, with next_norm,
    dxn [T, emb] bf16 at the stored out: dict of dres, dy, dpost_weight, dgate, dnext_weight, None where not needed or
    not there. y as given to, or returned by, block_out. dgate: fp32 for a gate [emb] or [T, 1], else the gate's
    type."""
    lead = out if out is not None else dout
    if lead is None:
        raise ValueError("dout, or dxn and out, must be given")
    ty = _need_typed(lead, "dout" if out is None else "out", 2)
    dev = lead.device
    T, emb = lead.shape
    if next_norm != (dxn is not None) or next_norm != (out is not None):
        raise ValueError("next_norm goes with dxn and out")
    if next_weight is not None and not next_norm:
        raise ValueError("next_weight without next_norm")
    b, mode = _block(ty, T, emb, dev, post_norm, post_weight, gate, float(scale), float(res_scale), next_weight,
                     float(offset), float(eps))
    _need_like(dout, "dout", (T, emb), lead.dtype, dev)
    _need_like(dxn, "dxn", (T, emb), torch.bfloat16, dev)
    if y is None and (post_norm or gate is not None):
        raise ValueError("y is missing")
    _need_like(y, "y", (T, emb), torch.bfloat16, dev)

    def new(name, have, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev) if have and name in need else None

    f32 = torch.float32
    dres = new("dres", True, (T, emb), lead.dtype)
    dy = new("dy", True, (T, emb), torch.bfloat16)
    dpw = new("dpost_weight", post_weight is not None, (emb,), f32)
    dnw = new("dnext_weight", next_weight is not None, (emb,), f32)
    dgate = None
    if gate is not None:
        dgate = new("dgate", True, tuple(gate.shape), gate.dtype if mode == _lib.MOE_GATE_FULL else f32)
    ws = None
    if dpw is not None or dnw is not None or (dgate is not None and mode == _lib.MOE_GATE_CHANNEL):
        ws = _workspace(workspace, int(_lib.lib().moe_block_out_bwd_workspace_bytes(T, emb)), dev)
    _call("moe_block_out_bwd", dev, T, emb, b, dout, y, out, dxn, dres, dy, dpw, dnw, dgate, ws,
          0 if ws is None else ws.numel())
    return dict(dres=dres, dy=dy, dpost_weight=dpw, dgate=dgate, dnext_weight=dnw)
