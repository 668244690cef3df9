"""Norms before and after a block, with the block's gate and residual scale, and their gradients
(the C entry points of the same names in include/moe.h). Tokens [T][h] bfloat16 or float16; norm
weights and channel gates [h] of the same type (None: ones); token gates and reciprocal norms [T]
float32.
"""
from __future__ import annotations

import torch

from ._launch import Launch, elt16
from ._lib import MoeError, check, load

__all__ = ["moe_pre_norm", "moe_pre_norm_int8", "moe_post_norm",
           "moe_norm_backward_workspace_bytes", "moe_pre_norm_backward",
           "moe_post_norm_backward"]


def _tokens(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (T, h)")
    return t.shape[0], t.shape[1], elt16(t, name)


def _int8_out(L, T, h, codes, scales):
    pitch = (h + 127) // 128 * 128
    codes = L.empty(T, pitch, dtype=torch.int8) if codes is None else codes
    scales = L.empty(T, dtype=torch.float32) if scales is None else scales
    return (codes, scales, L.dense(codes, "codes", torch.int8, T, pitch),
            L.dense(scales, "scales", torch.float32, T))


def _kept(L, T, save, t):
    """A reciprocal-norm output: allocated when a backward pass will follow."""
    return L.empty(T, dtype=torch.float32) if t is None and save else t


def moe_pre_norm(x, w=None, eps: float = 1e-6, z=None, rstd=None, save: bool = False, stream=None):
    """z = x rstd w, rstd = (mean x^2 + eps)^(-1/2). Returns (z, rstd); rstd is None unless save
    (what moe_pre_norm_backward reads)."""
    T, h, dt = _tokens(x, "x")
    L = Launch(x.device, stream)
    with L:
        z = L.empty(T, h, dtype=x.dtype) if z is None else z
        rstd = _kept(L, T, save, rstd)
        check("moe_pre_norm", load().moe_pre_norm(
            T, h, dt, L.dense(x, "x", x.dtype, T, h), L.dense(w, "w", x.dtype, h), eps,
            L.dense(z, "z", x.dtype, T, h), None, None,
            L.dense(rstd, "rstd", torch.float32, T), L.handle))
    return z, rstd


def moe_pre_norm_int8(x, w=None, eps: float = 1e-6, z=None, codes=None, scales=None, rstd=None,
                      save: bool = False, stream=None):
    """The pre-norm as the int8 rows that the int8 products read (and as z too, if a buffer for it
    is given: a router reads 16-bit tokens). Returns (codes, scales, rstd)."""
    T, h, dt = _tokens(x, "x")
    L = Launch(x.device, stream)
    with L:
        codes, scales, cp, sp = _int8_out(L, T, h, codes, scales)
        rstd = _kept(L, T, save, rstd)
        check("moe_pre_norm", load().moe_pre_norm(
            T, h, dt, L.dense(x, "x", x.dtype, T, h), L.dense(w, "w", x.dtype, h), eps,
            L.dense(z, "z", x.dtype, T, h), cp, sp, L.dense(rstd, "rstd", torch.float32, T),
            L.handle))
    return codes, scales, rstd


def moe_post_norm(res, y, w=None, gate=None, token_gate=None, res_scale: float = 1.0, w_next=None,
                  eps: float = 1e-6, next_norm: bool = False, next_int8: bool = False, u=None,
                  z=None, codes=None, scales=None, rstd=None, rstd_next=None, save: bool = False,
                  stream=None):
    """u = res_scale res + (y rstd w) gate token_gate; with w_next (or next_norm) also the next
    block's pre-norm z of u, with next_int8 its int8 form. Returns (u, z, rstd, rstd_next), z being
    None without a next norm and (codes, scales) with next_int8; the reciprocal norms are None
    unless save."""
    T, h, dt = _tokens(res, "res")
    L = Launch(res.device, stream)
    nxt = next_norm or next_int8 or w_next is not None or z is not None
    with L:
        u = L.empty(T, h, dtype=res.dtype) if u is None else u
        rstd = _kept(L, T, save, rstd)
        cp = sp = None
        if nxt:
            rstd_next = _kept(L, T, save, rstd_next)
            if next_int8:
                codes, scales, cp, sp = _int8_out(L, T, h, codes, scales)
            elif z is None:
                z = L.empty(T, h, dtype=res.dtype)
        check("moe_post_norm", load().moe_post_norm(
            T, h, dt, L.dense(res, "res", res.dtype, T, h), L.dense(y, "y", res.dtype, T, h),
            L.dense(w, "w", res.dtype, h), L.dense(gate, "gate", res.dtype, h),
            L.dense(token_gate, "token_gate", torch.float32, T), res_scale, eps,
            L.dense(u, "u", res.dtype, T, h), L.dense(rstd, "rstd", torch.float32, T),
            L.dense(w_next, "w_next", res.dtype, h), L.dense(z, "z", res.dtype, T, h), cp, sp,
            L.dense(rstd_next, "rstd_next", torch.float32, T), L.handle))
    return u, (codes, scales) if next_int8 else z, rstd, rstd_next


def moe_norm_backward_workspace_bytes(T: int, h: int) -> int:
    return load().moe_norm_backward_workspace_bytes(T, h)


def _workspace(L, T, h, ws):
    n = moe_norm_backward_workspace_bytes(T, h)
    if n == 0:
        raise MoeError("moe_norm_backward_workspace_bytes", 2, "shape rejected")
    ws = L.empty(n, dtype=torch.uint8) if ws is None else ws
    return ws, L.buffer(ws, "ws", n)


def moe_pre_norm_backward(dz, x, rstd, w=None, d_res=None, dx=None, dw=None, ws=None, stream=None):
    """dx = d_res + the gradient of x through z = x rstd w, and dw [h] float32 (None without w).
    rstd from moe_pre_norm(save=True). Returns (dx, dw)."""
    T, h, dt = _tokens(dz, "dz")
    L = Launch(dz.device, stream)
    with L:
        dx = L.empty(T, h, dtype=dz.dtype) if dx is None else dx
        if dw is None and w is not None:
            dw = L.empty(h, dtype=torch.float32)
        ws, wsp = _workspace(L, T, h, ws)
        check("moe_pre_norm_backward", load().moe_pre_norm_backward(
            T, h, dt, L.dense(dz, "dz", dz.dtype, T, h), L.dense(x, "x", dz.dtype, T, h),
            L.dense(rstd, "rstd", torch.float32, T), L.dense(w, "w", dz.dtype, h),
            L.dense(d_res, "d_res", dz.dtype, T, h), L.dense(dx, "dx", dz.dtype, T, h),
            L.dense(dw, "dw", torch.float32, h), wsp, L.handle))
    return dx, dw


def moe_post_norm_backward(du, y, rstd, w=None, gate=None, token_gate=None, res_scale: float = 1.0,
                           dz=None, u=None, rstd_next=None, w_next=None, out=None, ws=None,
                           stream=None):
    """Gradients of moe_post_norm from du and/or dz (with dz also the stored u, rstd_next and
    w_next). Returns a dict: dres, dy, and dw, dgate, dw_next [h], dtoken_gate [T] in float32 for
    each of w, gate, w_next, token_gate that was given (else None). `out` may hold buffers for any
    of them."""
    T, h, dt = _tokens(y, "y")
    L = Launch(y.device, stream)
    f4 = torch.float32
    o = dict(out or {})
    with L:
        for name in ("dres", "dy"):
            if o.get(name) is None:
                o[name] = L.empty(T, h, dtype=y.dtype)
        for name, ref, n in (("dw", w, h), ("dgate", gate, h), ("dtoken_gate", token_gate, T),
                             ("dw_next", w_next, h)):
            if o.get(name) is None:
                o[name] = L.empty(n, dtype=f4) if ref is not None else None
        ws, wsp = _workspace(L, T, h, ws)
        check("moe_post_norm_backward", load().moe_post_norm_backward(
            T, h, dt, L.dense(du, "du", y.dtype, T, h), L.dense(y, "y", y.dtype, T, h),
            L.dense(rstd, "rstd", f4, T), L.dense(w, "w", y.dtype, h),
            L.dense(gate, "gate", y.dtype, h), L.dense(token_gate, "token_gate", f4, T), res_scale,
            L.dense(dz, "dz", y.dtype, T, h), L.dense(u, "u", y.dtype, T, h),
            L.dense(rstd_next, "rstd_next", f4, T), L.dense(w_next, "w_next", y.dtype, h),
            L.dense(o["dres"], "dres", y.dtype, T, h), L.dense(o["dy"], "dy", y.dtype, T, h),
            L.dense(o["dw"], "dw", f4, h), L.dense(o["dgate"], "dgate", f4, h),
            L.dense(o["dtoken_gate"], "dtoken_gate", f4, T),
            L.dense(o["dw_next"], "dw_next", f4, h), wsp, L.handle))
    return o
