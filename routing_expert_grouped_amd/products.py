"""Ragged grouped products and int8 products (the C entry points of the same names in
include/moe.h): out[r] = rows[src(r)] W[e] over the experts' row ranges of a schedule, its two
gradients, and the int8 forms with a scale per token and per weight column.

``shape`` is make_gemm_shape(R, K, N, E): R routed rows, expert matrices [K][N], E experts.
``offsets`` [E + 1] int32 and ``perm`` [R] int32 are those of moe_permute; with perm, the rows are
the T tokens and routed row r reads token perm[r] // k. Rows of an output outside every expert's
range (dropped assignments) are left as they were.
"""
from __future__ import annotations

import ctypes
from ctypes import byref

import torch

from ._launch import ELT, Launch, elt16
from ._lib import MoeError, MoeGemmShape, check, load

__all__ = ["make_gemm_shape", "moe_grouped_gemm", "moe_grouped_gemm_dgrad",
           "moe_grouped_gemm_wgrad_workspace_bytes", "moe_grouped_gemm_wgrad", "moe_int8_pitch", "moe_quantize_int8",
           "moe_int8_weight_bytes", "moe_int8_pack_weights", "moe_int8_prepare_weights",
           "moe_gemm_int8", "moe_grouped_gemm_int8"]


def make_gemm_shape(R: int, K: int, N: int, E: int = 1) -> MoeGemmShape:
    return MoeGemmShape(R, K, N, E)


def _out_dtype(dtype, allowed):
    if dtype not in allowed:
        raise ValueError(f"out_dtype {dtype}, expected one of {allowed}")
    return dtype


def _gather(L, perm, k, R):
    """(row_src pointer, row_div) of the gather arguments."""
    if perm is None:
        if k != 1:
            raise ValueError("k without perm")
        return None, 1
    if k < 1:
        raise ValueError(f"k {k}, expected at least 1")
    return L.dense(perm, "perm", torch.int32, R), k


def _rows_product(fn, name, shape, rows, w, offsets, perm, k, out, out_dtype, stream, cin, cout):
    dt = elt16(rows, name)
    R, K, N, E = shape.R, shape.K, shape.N, shape.E
    L = Launch(rows.device, stream)
    with L:
        if out is None:
            out_dtype = _out_dtype(rows.dtype if out_dtype is None else out_dtype,
                                   (rows.dtype, torch.float32))
            out = L.empty(R, cout, dtype=out_dtype)
        else:
            _out_dtype(out.dtype, (rows.dtype, torch.float32))
        src, div = _gather(L, perm, k, R)
        rp, ld, n = L.rows(rows, name, rows.dtype, cin, None if perm is not None else R)
        op, old, _ = L.rows(out, "out", out.dtype, cout, R)
        check(fn, getattr(load(), fn)(
            byref(shape), dt, rp, ld, src, div, n, L.dense(w, "w", rows.dtype, E, K, N),
            L.dense(offsets, "offsets", torch.int32, E + 1), op, old, ELT[out.dtype], L.handle))
    return out


def moe_grouped_gemm(shape, rows, w, offsets, perm=None, k: int = 1, out=None, out_dtype=None,
                     stream=None):
    """out[r] = rows[src(r)] w[e]. rows [R][K] (or the tokens [T][K] with perm and k) bfloat16 or
    float16, w [E][K][N]; out [R][N] of rows' type or float32. Rows of `rows` and `out` may be
    slices of wider tensors. Returns out."""
    return _rows_product("moe_grouped_gemm", "rows", shape, rows, w, offsets, perm, k, out,
                         out_dtype, stream, shape.K, shape.N)


def moe_grouped_gemm_dgrad(shape, dy, w, offsets, perm=None, k: int = 1, out=None, out_dtype=None,
                           stream=None):
    """dx[r] = dy[src(r)] w[e]^T, the gradient of moe_grouped_gemm's routed rows [R][K] from dy
    [R][N]. (With weights [E][out][in], "y = x W^T", this is their forward product: shape
    make_gemm_shape(R, out, in, E), dy the inputs.) Returns dx."""
    return _rows_product("moe_grouped_gemm_dgrad", "dy", shape, dy, w, offsets, perm, k, out,
                         out_dtype, stream, shape.N, shape.K)


def moe_grouped_gemm_wgrad_workspace_bytes(shape) -> int:
    return load().moe_grouped_gemm_wgrad_workspace_bytes(byref(shape))


def moe_grouped_gemm_wgrad(shape, rows, dy, offsets, perm=None, k: int = 1, dw=None,
                           dw_dtype=torch.float32, ws=None, stream=None):
    """dw[e] = sum over the expert's rows of rows[src(r)]^T dy[r], [E][K][N] in float32 or the
    operands' type; an expert without rows gets zeros. Returns dw."""
    dt = elt16(rows, "rows")
    R, K, N, E = shape.R, shape.K, shape.N, shape.E
    nws = moe_grouped_gemm_wgrad_workspace_bytes(shape)
    if nws == 0:
        raise MoeError("moe_grouped_gemm_wgrad_workspace_bytes", 1, "shape rejected")
    L = Launch(rows.device, stream)
    with L:
        ws = L.empty(nws, dtype=torch.uint8) if ws is None else ws
        if dw is None:
            dw = L.empty(E, K, N, dtype=_out_dtype(dw_dtype, (rows.dtype, torch.float32)))
        else:
            _out_dtype(dw.dtype, (rows.dtype, torch.float32))
        src, div = _gather(L, perm, k, R)
        rp, ld, n = L.rows(rows, "rows", rows.dtype, K, None if perm is not None else R)
        dp, dld, _ = L.rows(dy, "dy", rows.dtype, N, R)
        check("moe_grouped_gemm_wgrad", load().moe_grouped_gemm_wgrad(
            byref(shape), dt, rp, ld, src, div, n, dp, dld,
            L.dense(offsets, "offsets", torch.int32, E + 1),
            L.dense(dw, "dw", dw.dtype, E, K, N), ELT[dw.dtype], L.buffer(ws, "ws", nws),
            L.handle))
    return dw


def moe_int8_pitch(K: int) -> int:
    """Bytes between int8 code rows of width K."""
    return load().moe_int8_pitch(K)


def moe_quantize_int8(x, swiglu: bool = False, codes=None, scales=None, stream=None):
    """Int8 codes and a scale per row of x [R][K] (bfloat16 or float16), or of silu(G) * U for
    x = [G | U] [R][2K] with swiglu. Returns (codes [R][moe_int8_pitch(K)] int8, scales [R])."""
    dt = elt16(x, "x")
    if x.dim() != 2 or (swiglu and x.shape[1] % 2):
        raise ValueError(f"x: shape {tuple(x.shape)}, expected "
                         f"{'(rows, 2 K)' if swiglu else '(rows, K)'}")
    R, K = x.shape[0], x.shape[1] // (2 if swiglu else 1)
    L = Launch(x.device, stream)
    pitch = (K + 127) // 128 * 128
    with L:
        codes = L.empty(R, pitch, dtype=torch.int8) if codes is None else codes
        scales = L.empty(R, dtype=torch.float32) if scales is None else scales
        xp, ld, _ = L.rows(x, "x", x.dtype, x.shape[1])
        check("moe_quantize_int8", load().moe_quantize_int8(
            R, K, dt, xp, ld, int(bool(swiglu)), L.dense(codes, "codes", torch.int8, R, pitch),
            L.dense(scales, "scales", torch.float32, R), L.handle))
    return codes, scales


def moe_int8_weight_bytes(shape) -> int:
    return load().moe_int8_weight_bytes(byref(shape))


def _packed_bytes(shape):
    n = moe_int8_weight_bytes(shape)
    if n == 0:
        raise MoeError("moe_int8_weight_bytes", 1, "shape rejected")
    return n


def moe_int8_pack_weights(shape, w_codes, packed=None, stream=None):
    """Int8 weights [E][N][K] in the layout the int8 products read (done once per weight)."""
    n = _packed_bytes(shape)
    L = Launch(w_codes.device, stream)
    with L:
        packed = L.empty(n, dtype=torch.uint8) if packed is None else packed
        check("moe_int8_pack_weights", load().moe_int8_pack_weights(
            byref(shape), L.dense(w_codes, "w_codes", torch.int8, shape.E, shape.N, shape.K),
            L.buffer(packed, "packed", n), L.handle))
    return packed


def moe_int8_prepare_weights(shape, w, packed=None, w_scales=None, stream=None):
    """Weights [E][K][N] bfloat16 quantised per column and packed. Returns (packed, w_scales
    [E][N])."""
    n = _packed_bytes(shape)
    L = Launch(w.device, stream)
    with L:
        packed = L.empty(n, dtype=torch.uint8) if packed is None else packed
        w_scales = L.empty(shape.E, shape.N, dtype=torch.float32) if w_scales is None else w_scales
        check("moe_int8_prepare_weights", load().moe_int8_prepare_weights(
            byref(shape), L.dense(w, "w", torch.bfloat16, shape.E, shape.K, shape.N),
            L.buffer(packed, "packed", n),
            L.dense(w_scales, "w_scales", torch.float32, shape.E, shape.N), L.handle))
    return packed, w_scales


def _int8_product(shape, codes, scales, packed, w_scales, offsets, perm, k, bias, out, out_dtype,
                  stream):
    R, K, N, E = shape.R, shape.K, shape.N, shape.E
    nbytes = _packed_bytes(shape)
    L = Launch(codes.device, stream)
    with L:
        allowed = (torch.bfloat16, torch.float16, torch.float32)
        if out is None:
            out = L.empty(R, N, dtype=_out_dtype(out_dtype, allowed))
        else:
            _out_dtype(out.dtype, allowed)
        src, div = _gather(L, perm, k, R)
        n = codes.shape[0] if codes.dim() == 2 and perm is not None else R
        cp = L.dense(codes, "codes", torch.int8, n, (K + 127) // 128 * 128)
        sp = L.dense(scales, "scales", torch.float32, n)
        op, old, _ = L.rows(out, "out", out.dtype, N, R)
        pp = L.buffer(packed, "packed", nbytes)
        wp = L.dense(w_scales, "w_scales", torch.float32, E, N)
        bp = L.dense(bias, "bias", torch.float32, E, N)
        if offsets is None:
            check("moe_gemm_int8", load().moe_gemm_int8(
                byref(shape), cp, sp, pp, wp, bp, op, old, ELT[out.dtype], L.handle))
        else:
            check("moe_grouped_gemm_int8", load().moe_grouped_gemm_int8(
                byref(shape), cp, sp, src, div, n,
                L.dense(offsets, "offsets", torch.int32, E + 1), pp, wp, bp, op, old,
                ELT[out.dtype], L.handle))
    return out


def moe_gemm_int8(shape, codes, scales, packed, w_scales, bias=None, out=None,
                  out_dtype=torch.bfloat16, stream=None):
    """out[r][n] = (codes[r] . q[n]) scales[r] w_scales[0][n] + bias[0][n]: codes and scales from
    moe_quantize_int8 or a norm, packed weights of one expert (shape.E = 1). Returns out [R][N]."""
    return _int8_product(shape, codes, scales, packed, w_scales, None, None, 1, bias, out,
                         out_dtype, stream)


def moe_grouped_gemm_int8(shape, codes, scales, packed, w_scales, offsets, perm=None, k: int = 1,
                          bias=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """The int8 product of each expert over its routed rows; with perm and k the codes are those of
    the T tokens, each quantised once. w_scales and bias [E][N]. Returns out [R][N]."""
    if offsets is None:
        raise ValueError("offsets: need the schedule's offsets")
    return _int8_product(shape, codes, scales, packed, w_scales, offsets, perm, k, bias, out,
                         out_dtype, stream)
