"""Plain 64-bit forms of the ragged products, the int8 products and the block norms, on the CPU,
with the error bounds that the GPU tests allow.

Bounds. A product of two 16-bit values is exact in float32, and a float32 sum of n terms is within
n 2^-23 of the sum of their magnitudes in any order, also where the matrix core truncates instead
of rounding an addition (2^-24 for a rounded one). The last rounding adds half a step of the output type
relative to the value (and half a subnormal step of float16 near zero).
"""
import numpy as np
import torch

F8 = torch.float64
EPS24 = 2.0 ** -24


def half_step(dtype, ref):
    """Half a step of dtype at ref, elementwise (an upper bound), and the subnormal floor."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def f8(t):
    return t.detach().cpu().to(F8)


def segments(offsets):
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def grouped(rows, w, offsets, src=None, trans=False):
    """(out, magnitude) of out[r] = rows[src[r]] W[e] in 64 bits; rows outside every expert NaN."""
    rows, w = f8(rows), f8(w)
    R = len(src) if src is not None else rows.shape[0]
    out = torch.full((R, w.shape[1] if trans else w.shape[2]), float("nan"), dtype=F8)
    mag = torch.zeros_like(out)
    for e, a, b in segments(offsets):
        if a == b:
            continue
        x = rows[src[a:b]] if src is not None else rows[a:b]
        we = w[e].t() if trans else w[e]
        out[a:b] = x @ we
        mag[a:b] = x.abs() @ we.abs()
    return out, mag


def wgrad(rows, dy, offsets, src=None):
    rows, dy = f8(rows), f8(dy)
    E = len(offsets) - 1
    out = torch.zeros(E, rows.shape[1], dy.shape[1], dtype=F8)
    mag = torch.zeros_like(out)
    for e, a, b in segments(offsets):
        if a == b:
            continue
        x = rows[src[a:b]] if src is not None else rows[a:b]
        out[e] = x.t() @ dy[a:b]
        mag[e] = x.abs().t() @ dy[a:b].abs()
    return out, mag


def product_bound(ref, mag, n, dtype):
    return half_step(dtype, ref) * (1 + 2.0 ** -8) + n * 2 * EPS24 * mag


def quantise(p):
    """(codes, amax) of float64 rows."""
    amax = p.abs().max(dim=1).values
    safe = torch.where(amax == 0, torch.ones_like(amax), amax)
    return torch.round(127.0 * p / safe[:, None]), amax  # torch.round: ties to even


def scale32(amax):
    """amax / 127 in one float32 rounding."""
    return torch.from_numpy(amax.numpy().astype(np.float32) / np.float32(127.0))


def rstd(x, eps):
    return 1.0 / torch.sqrt((x * x).mean(dim=1) + float(np.float32(eps)))


def rstd_rel(h):
    """Relative error of a float32 reciprocal norm: half that of a sum of h squares, and the
    mean, root, eps and quotient roundings."""
    return (h + 8) * EPS24


def vec(w, h):
    return torch.ones(h, dtype=F8) if w is None else f8(w)


def post_norm(res, y, w, gate, tau, scale, eps):
    """(u, rstd, magnitude)."""
    res, y = f8(res), f8(y)
    T, h = res.shape
    r = rstd(y, eps)
    t = torch.ones(T, dtype=F8) if tau is None else f8(tau)
    v = y * (r * t)[:, None] * (vec(w, h) * vec(gate, h))[None]
    u = float(np.float32(scale)) * res + v
    return u, r, (float(np.float32(scale)) * res).abs() + v.abs()


def norm_grads(dz, x, r, w):
    """(gradient of x through z = x r w, gradient of w, and the magnitudes of both)."""
    n = x * r[:, None]
    q = dz * w[None]
    dx = r[:, None] * (q - n * (q * n).mean(1, keepdim=True))
    mag = r[:, None].abs() * (q.abs() + n.abs() * (q * n).abs().mean(1, keepdim=True))
    return dx, (dz * n).sum(0), mag, (dz * n).abs().sum(0)


def post_norm_grads(du, y, r, w, gate, tau, scale, dz=None, u=None, r_next=None, w_next=None):
    """Every gradient of post_norm (r, r_next taken as given), with a magnitude for each."""
    y, r = f8(y), f8(r)
    T, h = y.shape
    w8, g8 = vec(w, h), vec(gate, h)
    t = (torch.ones(T, dtype=F8) if tau is None else f8(tau))[:, None]
    s = float(np.float32(scale))
    G = torch.zeros(T, h, dtype=F8) if du is None else f8(du)
    M = G.abs()
    o = {}
    if dz is not None:
        dx, dwn, mx, mwn = norm_grads(f8(dz), f8(u), f8(r_next), vec(w_next, h))
        G, M = G + dx, M + mx
        o["dw_next"] = (dwn, mwn)
    n = y * r[:, None]
    dn, dm = G * w8 * g8 * t, M * (w8 * g8 * t).abs()
    o["dres"] = (s * G, abs(s) * M)
    o["dy"] = (r[:, None] * (dn - n * (dn * n).mean(1, keepdim=True)),
               r[:, None].abs() * (dm + n.abs() * (dm * n.abs()).mean(1, keepdim=True)))
    o["dtoken_gate"] = ((G * n * w8 * g8).sum(1), (M * (n * w8 * g8).abs()).sum(1))
    A, MA = (G * n * t).sum(0), (M * (n * t).abs()).sum(0)
    o["dw"] = (A * g8, MA * g8.abs())
    o["dgate"] = (A * w8, MA * w8.abs())
    return o
