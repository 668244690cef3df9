"""GPU parity of the block norms against their plain 64-bit forms, within the bounds of
tests/_plain_ops.py, and the run of the norms, the int8 products and the expert layer's schedule and
combine together."""
import pytest

from tests import _plain_ops as P
from tests._gpu_helpers import note, poisoned, require_gpu, torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 2.0 ** -20
WIDTHS = [1, 3, 8, 100, 511, 512, 520, 1000, 1025, 2048, 2056, 4096, 4099, 6144, 7168, 8191, 8192,
          9000, 16384]


def _rand(g, *shape, dtype=BF, scale=1.0, mean=0.0):
    return (mean + torch.randn(*shape, generator=g) * scale).to(dtype)


def _close(got, ref, bound, what):
    got = P.f8(got)
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, bad.nonzero()[0].tolist(), got[bad][0].item(),
                           ref[bad][0].item(), bound[bad][0].item())


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("h", WIDTHS)
def test_pre_norm(h, dtype):
    G = require_gpu()
    T = 5
    g = torch.Generator().manual_seed(h)
    x, w = _rand(g, T, h, dtype=dtype, scale=2.0), _rand(g, h, dtype=dtype, mean=1.0, scale=0.2)
    x[1] = 0  # a row of zeros: rstd = eps^(-1/2), z = 0, int8 scale 0
    x[2] *= 2.0 ** -12
    for wt in (w, None):
        note(f"pre_norm h={h} {dtype} w={wt is not None}")
        xd, wd = _cuda(x, wt)
        z, r = G.moe_pre_norm(xd, wd, EPS, z=poisoned((T, h), dtype), save=True)
        rr = P.rstd(P.f8(x), EPS)
        _close(r, rr, rr * P.rstd_rel(h), "rstd")
        ref = P.f8(x) * rr[:, None] * P.vec(wt, h)
        _close(z, ref, P.half_step(dtype, ref) * (1 + 2.0 ** -8) +
               ref.abs() * (P.rstd_rel(h) + 2 * P.EPS24), "z")
        pitch = (h + 127) // 128 * 128
        z2 = poisoned((T, h), dtype)
        codes, scales, _ = G.moe_pre_norm_int8(xd, wd, EPS, z=z2,
                                               codes=poisoned((T, pitch), torch.int8))
        assert torch.equal(z2, z)
        c, amax = P.quantise(P.f8(x) * P.vec(wt, h))
        got = codes.cpu()
        assert (got[:, h:] == 0).all()
        if dtype == BF:  # 127 x w is exact in float32
            assert torch.equal(got[:, :h].to(P.F8), c)
        else:            # 127 x w rounds once: a code may fall on the other side of a border
            assert ((got[:, :h].to(P.F8) - c).abs() <= 1).all()
            assert ((got[:, :h].to(P.F8) != c).sum() <= 1 + c.numel() // 1000)
        sref = amax * rr / 127
        _close(scales, sref, sref * (P.rstd_rel(h) + 3 * P.EPS24), "scales")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("h", WIDTHS)
def test_post_norm(h, dtype):
    G = require_gpu()
    T, a = 6, 0.7
    g = torch.Generator().manual_seed(h + 1)
    res, y = _rand(g, T, h, dtype=dtype), _rand(g, T, h, dtype=dtype, scale=0.5)
    y[2] = 0
    w, gate, wn = (_rand(g, h, dtype=dtype, mean=1.0, scale=0.3) for _ in range(3))
    tau = torch.rand(T, generator=g)
    tau[3] = 0.0
    for opts in ((w, gate, tau, wn), (None, None, None, None), (w, None, tau, None)):
        w_, g_, t_, n_ = opts
        note(f"post_norm h={h} {dtype} {[o is not None for o in opts]}")
        rd, yd, wd, gd, td, nd = _cuda(res, y, w_, g_, t_, n_)
        u, z, r, rn = G.moe_post_norm(rd, yd, wd, gate=gd, token_gate=td, res_scale=a, w_next=nd,
                                      eps=EPS, next_norm=True, u=poisoned((T, h), dtype),
                                      z=poisoned((T, h), dtype), save=True)
        ref, rr, mag = P.post_norm(res, y, w_, g_, t_, a, EPS)
        _close(r, rr, rr * P.rstd_rel(h), "rstd")
        _close(u, ref, P.half_step(dtype, ref) * (1 + 2.0 ** -8) +
               mag * (P.rstd_rel(h) + 6 * P.EPS24), "u")
        # the next norm is that of the stored u, bit for bit
        z1, r1 = G.moe_pre_norm(u, nd, EPS, save=True)
        assert torch.equal(z, z1) and torch.equal(rn, r1)
        u2, none, _, _ = G.moe_post_norm(rd, yd, wd, gate=gd, token_gate=td, res_scale=a, eps=EPS)
        assert none is None and torch.equal(u, u2)
        u3, (c3, s3), _, _ = G.moe_post_norm(rd, yd, wd, gate=gd, token_gate=td, res_scale=a,
                                             w_next=nd, eps=EPS, next_int8=True)
        c1, s1, _ = G.moe_pre_norm_int8(u, nd, EPS)
        assert torch.equal(u3, u) and torch.equal(c3, c1) and torch.equal(s3, s1)


def _grad_bound(ref, mag, n, dtype):
    """float32 sums of n terms of the magnitudes, with a few roundings per term."""
    return P.half_step(dtype, ref) * (1 + 2.0 ** -8) + mag * (n + 32) * P.EPS24


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,h", [(1, 1), (3, 100), (5, 512), (700, 130), (9, 1024), (4, 2056),
                                 (600, 72), (6, 4096), (3, 6144), (2, 8191), (3, 16384)])
def test_norm_backward(T, h, dtype):
    G = require_gpu()
    g = torch.Generator().manual_seed(T + h)
    y, u = _rand(g, T, h, dtype=dtype, scale=0.5), _rand(g, T, h, dtype=dtype)
    du, dz = _rand(g, T, h, dtype=dtype), _rand(g, T, h, dtype=dtype)
    w, gate, wn = (_rand(g, h, dtype=dtype, mean=1.0, scale=0.3) for _ in range(3))
    tau = torch.rand(T, generator=g)
    r, rn = P.rstd(P.f8(y), EPS).float(), P.rstd(P.f8(u), EPS).float()
    # the norm before a block
    for d_res, wt in ((du, wn), (None, wn), (None, None)):
        note(f"pre_norm_backward T={T} h={h} {dtype} d_res={d_res is not None}")
        dzd, ud, rnd, wd, dd = _cuda(dz, u, rn, wt, d_res)
        dx, dw = G.moe_pre_norm_backward(dzd, ud, rnd, wd, d_res=dd, dx=poisoned((T, h), dtype))
        ref, rw, mag, mw = P.norm_grads(P.f8(dz), P.f8(u), P.f8(rn), P.vec(wt, h))
        if d_res is not None:
            ref, mag = ref + P.f8(du), mag + P.f8(du).abs()
        _close(dx, ref, _grad_bound(ref, mag, h, dtype), "dx")
        if wt is None:
            assert dw is None
        else:
            _close(dw, rw, _grad_bound(rw, mw, T, F32), "dw")
    # the norm after a block, alone and with the next norm
    for full in (True, False):
        for opt in (True, False):
            note(f"post_norm_backward T={T} h={h} {dtype} next={full} gates={opt}")
            w_, g_, t_ = (w, gate, tau) if opt else (None, None, None)
            nxt = dict(dz=dz, u=u, rstd_next=rn, w_next=wn if opt else None) if full else {}
            dur = du if opt or not full else None
            got = G.moe_post_norm_backward(
                *_cuda(dur, y, r, w_), gate=_cuda(g_)[0], token_gate=_cuda(t_)[0], res_scale=0.7,
                **{n: _cuda(v)[0] for n, v in nxt.items()},
                out={"dres": poisoned((T, h), dtype), "dy": poisoned((T, h), dtype)})
            want = P.post_norm_grads(dur, y, r, w_, g_, t_, 0.7, nxt.get("dz"), nxt.get("u"),
                                     nxt.get("rstd_next"), nxt.get("w_next"))
            for name, given in (("dres", True), ("dy", True), ("dw", opt), ("dgate", opt),
                                ("dtoken_gate", opt), ("dw_next", opt and full)):
                if not given:
                    assert got[name] is None, name
                    continue
                ref, mag = want[name]
                n = T + 2 * h if name in ("dw", "dgate") else (T if name == "dw_next" else 2 * h)
                _close(got[name], ref, _grad_bound(ref, mag, n, got[name].dtype), name)


def test_no_tokens():
    G = require_gpu()
    h = 96
    e = torch.empty(0, h, dtype=BF, device="cuda")
    r = torch.empty(0, device="cuda")
    w = torch.ones(h, dtype=BF, device="cuda")
    assert G.moe_pre_norm(e, w)[0].shape == (0, h)
    assert G.moe_post_norm(e, e, w, w_next=w)[1].shape == (0, h)
    dx, dw = G.moe_pre_norm_backward(e, e, r, w, dw=poisoned((h,), F32))
    assert dx.shape == (0, h) and (dw == 0).all()
    o = G.moe_post_norm_backward(e, e, r, w, gate=w, dz=e, u=e, rstd_next=r, w_next=w,
                                 out={n: poisoned((h,), F32) for n in ("dw", "dgate", "dw_next")})
    assert all((o[n] == 0).all() for n in ("dw", "dgate", "dw_next"))


def test_not_finite_rows_stay_apart():
    G = require_gpu()
    g = torch.Generator().manual_seed(8)
    x = _rand(g, 6, 700)
    x[1, 5], x[4, 6] = float("nan"), float("inf")
    z, _ = G.moe_pre_norm(x.cuda())
    ok = torch.isfinite(z).all(dim=1).cpu().tolist()
    assert ok == [True, False, True, True, False, True]
    _, scales, _ = G.moe_pre_norm_int8(x.cuda())
    assert torch.isfinite(scales).cpu().tolist() == ok


def test_graph_replays_and_determinism():
    G = require_gpu()
    g = torch.Generator().manual_seed(12)
    T, h = 300, 1000
    xs = [_rand(g, T, h).cuda() for _ in range(3)]
    y, du = _rand(g, T, h).cuda(), _rand(g, T, h).cuda()
    w, gate, wn = (_rand(g, h, mean=1.0, scale=0.2).cuda() for _ in range(3))

    def step(x):
        u, z, r, rn = G.moe_post_norm(x, y, w, gate=gate, w_next=wn, save=True)
        o = G.moe_post_norm_backward(du, y, r, w, gate=gate, dz=z, u=u, rstd_next=rn, w_next=wn)
        return [u, z] + [o[n] for n in ("dres", "dy", "dw", "dgate", "dw_next")]

    want = [[t.clone() for t in step(x)] for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        step(xs[2 - i])


def test_int8_layer_run():
    """A whole int8 expert layer between its norms, as one would serve it: pre-norm (16-bit tokens
    for the router, int8 rows for the experts), route, schedule, gate|up product gathered through
    perm, SwiGLU + quantise, down product, combine, post-norm with the next pre-norm."""
    G = require_gpu()
    T, h, m, E, k = 70, 256, 128, 8, 2
    g = torch.Generator().manual_seed(21)
    x = _rand(g, T, h)
    w1, w2, w3 = (_rand(g, h, mean=1.0, scale=0.1) for _ in range(3))
    gate = _rand(g, h, mean=0.5, scale=0.1)
    wr = _rand(g, E, h, scale=h ** -0.5)
    wg = _rand(g, E, h, 2 * m, scale=h ** -0.5)
    wd = _rand(g, E, m, h, scale=m ** -0.5)
    R = T * k
    s1, s2 = G.make_gemm_shape(R, h, 2 * m, E), G.make_gemm_shape(R, m, h, E)
    p1, ws1 = G.moe_int8_prepare_weights(s1, wg.cuda())
    p2, ws2 = G.moe_int8_prepare_weights(s2, wd.cuda())
    sh = G.make_shape(T, h, m, E, k)

    z = torch.empty(T, h, dtype=BF, device="cuda")
    codes, scales, _ = G.moe_pre_norm_int8(x.cuda(), w1.cuda(), z=z)
    _, idx, tw = G.moe_route(sh, z, wr.cuda())
    o = G.moe_permute(sh, "bf16", idx, z)
    gu = G.moe_grouped_gemm_int8(s1, codes, scales, p1, ws1, o["offsets"], perm=o["perm"], k=k)
    hc, hs = G.moe_quantize_int8(gu, swiglu=True)
    rows = G.moe_grouped_gemm_int8(s2, hc, hs, p2, ws2, o["offsets"])
    y = G.moe_combine(sh, rows, o["inv"], tw)
    u, zn, _, _ = G.moe_post_norm(x.cuda(), y, w2.cuda(), gate=gate.cuda(), res_scale=0.9,
                                  w_next=w3.cuda())

    # the same in 64 bits from the unquantised weights, on the routing found above: the int8 steps
    # (half a step of 1/127 of each row's and column's largest value) leave a relative error of
    # about 1% per product; 5% of the largest value bounds the layer
    f = P.f8
    zz = f(x) * P.rstd(f(x), 1e-6)[:, None] * f(w1)
    yy = torch.zeros(T, h, dtype=P.F8)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            a = zz[t] @ f(wg[e])
            hh = a[:m] / (1 + torch.exp(-a[:m])) * a[m:]
            yy[t] += float(tw[t, j]) * (hh @ f(wd[e]))
    assert (f(y) - yy).abs().max() <= 0.05 * yy.abs().max()
    ur, _, _ = P.post_norm(x, y, w2, gate, None, 0.9, 1e-6)
    _close(u, ur, P.half_step(BF, ur) * 1.01 + ur.abs().max() * 300 * P.EPS24, "u")
    zr = f(u) * P.rstd(f(u), 1e-6)[:, None] * f(w3)
    _close(zn, zr, P.half_step(BF, zr) * 1.01 + zr.abs() * 300 * P.EPS24, "z")


def test_training_step_run():
    """One expert matrix between the norms in training: forward and every gradient, each step
    against its 64-bit form on the values the step before it produced."""
    G = require_gpu()
    T, h, E, k = 90, 200, 5, 2
    R = T * k
    g = torch.Generator().manual_seed(22)
    x, du = _rand(g, T, h), _rand(g, T, h)
    w1, w2 = (_rand(g, h, mean=1.0, scale=0.1) for _ in range(2))
    W = _rand(g, E, h, h, scale=h ** -0.5)
    assign = torch.randint(0, E, (R,), generator=g)
    perm = torch.argsort(assign, stable=True)
    off = [0] + torch.bincount(assign, minlength=E).cumsum(0).tolist()
    pd, od = perm.to(torch.int32).cuda(), torch.tensor(off, dtype=torch.int32).cuda()
    src = perm // k
    sh = G.make_gemm_shape(R, h, h, E)
    z, r1 = G.moe_pre_norm(x.cuda(), w1.cuda(), save=True)
    rows = G.moe_grouped_gemm(sh, z, W.cuda(), od, perm=pd, k=k)
    ref, mag = P.grouped(z, W, off, src)
    _close(rows, ref, P.product_bound(ref, mag, h, BF), "rows")
    inv = torch.empty(R, dtype=torch.int32)
    inv[perm] = torch.arange(R, dtype=torch.int32)
    y = (rows.float()[inv.long().cuda()].view(T, k, h).sum(1) * 0.5).to(BF)
    u, _, r2, _ = G.moe_post_norm(x.cuda(), y, w2.cuda(), save=True)
    gr = G.moe_post_norm_backward(du.cuda(), y, r2, w2.cuda())
    want = P.post_norm_grads(du, y, r2, w2, None, None, 1.0)
    for n in ("dres", "dy", "dw"):
        _close(gr[n], want[n][0], _grad_bound(want[n][0], want[n][1], T + 2 * h, gr[n].dtype), n)
    drows = (0.5 * gr["dy"].float())[src.cuda()].to(BF).contiguous()
    dW = G.moe_grouped_gemm_wgrad(sh, z, drows, od, perm=pd, k=k)
    ref, mag = P.wgrad(z, P.f8(drows), off, src)
    _close(dW, ref, P.product_bound(ref, mag, R, F32), "dW")
    dzr = G.moe_grouped_gemm_dgrad(sh, drows, W.cuda(), od)
    ref, mag = P.grouped(drows, W, off, trans=True)
    _close(dzr, ref, P.product_bound(ref, mag, h, BF), "dz rows")
    dz = dzr.float()[inv.long().cuda()].view(T, k, h).sum(1).to(BF)
    dx, dw1 = G.moe_pre_norm_backward(dz, x.cuda(), r1, w1.cuda(), d_res=gr["dres"])
    ref, rw, mag, mw = P.norm_grads(P.f8(dz), P.f8(x), P.f8(r1), P.f8(w1))
    ref, mag = ref + P.f8(gr["dres"]), mag + P.f8(gr["dres"]).abs()
    _close(dx, ref, _grad_bound(ref, mag, h, BF), "dx")
    _close(dw1, rw, _grad_bound(rw, mw, T, F32), "dw1")
