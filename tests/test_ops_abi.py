"""Refusals of the ragged products, the int8 products and the block norms, on the host: every call
below fails its checks (or has nothing to do), so nothing is ever enqueued. And the binding's tensor
checks on stand-in tensors."""
import ctypes
import os

import pytest

FAKE = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from routing_expert_grouped_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from routing_expert_grouped_amd import build
        build.build(verbose=False)
    return _lib


def _s(lib, R=64, K=100, N=60, E=4):
    return ctypes.byref(lib.MoeGemmShape(R, K, N, E))


BF, HF, F32 = 0, 1, 2
BIG = [dict(R=(1 << 30) + 1), dict(K=(1 << 20) + 1), dict(N=(1 << 20) + 1), dict(E=1025),
       dict(R=1 << 30, N=1 << 20)]
BAD = [dict(R=-1), dict(K=0), dict(N=0), dict(E=0), dict(K=-5)]


def _fwd(lib, L, fn="moe_grouped_gemm", shape=None, dt=BF, rows=FAKE, ld=200, src=None, div=1,
         nsrc=64, w=FAKE, off=FAKE, out=FAKE, ldo=200, odt=BF):
    return getattr(L, fn)(shape or _s(lib), dt, rows, ld, src, div, nsrc, w, off, out, ldo, odt,
                          None)


@pytest.mark.parametrize("fn", ["moe_grouped_gemm", "moe_grouped_gemm_dgrad"])
def test_grouped_product_refusals(lib, fn):
    L = lib.load()
    bad = [dict(rows=None), dict(w=None), dict(off=None), dict(out=None), dict(rows=FAKE + 2),
           dict(w=FAKE + 8), dict(out=FAKE + 4), dict(off=FAKE + 4), dict(dt=F32), dict(dt=7),
           dict(odt=HF), dict(odt=9), dict(nsrc=63), dict(src=FAKE, div=0),
           dict(src=FAKE, nsrc=0), dict(src=FAKE + 4)]
    bad += [dict(ld=99 if fn == "moe_grouped_gemm" else 59),
            dict(ldo=59 if fn == "moe_grouped_gemm" else 99)]
    for kw in bad:
        assert _fwd(lib, L, fn, **kw) == lib.MOE_EINVAL, kw
    for kw in BAD:
        assert _fwd(lib, L, fn, shape=_s(lib, **kw)) == lib.MOE_EINVAL, kw
    for kw in BIG:
        assert _fwd(lib, L, fn, shape=_s(lib, **kw), nsrc=1 << 30, ld=1 << 21, ldo=1 << 21) == \
            lib.MOE_EUNSUPPORTED, kw
    assert getattr(L, fn)(None, BF, FAKE, 200, None, 1, 64, FAKE, FAKE, FAKE, 200, BF, None) == \
        lib.MOE_EINVAL
    # no rows: nothing to do, and buffers without elements may be null
    assert _fwd(lib, L, fn, shape=_s(lib, R=0), rows=None, out=None, nsrc=0) == lib.MOE_OK


def test_wgrad_refusals(lib):
    L = lib.load()

    def call(shape=None, dt=BF, rows=FAKE, ld=100, src=None, div=1, nsrc=64, dy=FAKE, ldy=60,
             off=FAKE, dw=FAKE, wdt=F32, ws=FAKE):
        return L.moe_grouped_gemm_wgrad(shape or _s(lib), dt, rows, ld, src, div, nsrc, dy, ldy,
                                        off, dw, wdt, ws, None)

    # many rows into a small gradient: room for the parts; else next to none
    assert L.moe_grouped_gemm_wgrad_workspace_bytes(_s(lib, R=8192, K=64, N=64, E=1)) >= \
        2 * 64 * 64 * 4
    assert 0 < L.moe_grouped_gemm_wgrad_workspace_bytes(_s(lib, R=100, K=64, N=64)) <= 256
    assert L.moe_grouped_gemm_wgrad_workspace_bytes(_s(lib, R=-1)) == 0
    for kw in [dict(ws=None), dict(ws=FAKE + 8), dict(rows=None), dict(dy=None), dict(dw=None), dict(off=None), dict(dw=FAKE + 4),
               dict(ld=99), dict(ldy=59), dict(wdt=HF), dict(dt=F32), dict(nsrc=10),
               dict(src=FAKE, div=-1)]:
        assert call(**kw) == lib.MOE_EINVAL, kw
    for kw in BAD:
        assert call(shape=_s(lib, **kw)) == lib.MOE_EINVAL, kw
    for kw in BIG:
        assert call(shape=_s(lib, **kw), nsrc=1 << 30, ld=1 << 21, ldy=1 << 21) == \
            lib.MOE_EUNSUPPORTED, kw


def test_int8_refusals(lib):
    L = lib.load()
    assert [L.moe_int8_pitch(k) for k in (-1, 0, 1, 128, 129)] == [0, 0, 128, 128, 256]
    assert L.moe_int8_weight_bytes(_s(lib, K=100, N=60, E=4)) == 4 * 64 * 128
    assert L.moe_int8_weight_bytes(_s(lib, K=131072)) == 0
    assert L.moe_int8_weight_bytes(_s(lib, E=0)) == 0

    def q(R=4, K=100, dt=BF, x=FAKE, ld=200, sw=0, c=FAKE, s=FAKE):
        return L.moe_quantize_int8(R, K, dt, x, ld, sw, c, s, None)

    for kw in [dict(x=None), dict(c=None), dict(s=None), dict(x=FAKE + 2), dict(ld=99),
               dict(sw=1, ld=199), dict(sw=2), dict(dt=F32), dict(R=-1), dict(K=0)]:
        assert q(**kw) == lib.MOE_EINVAL, kw
    assert q(K=16385, ld=1 << 20) == lib.MOE_EUNSUPPORTED
    assert q(R=0, x=None, c=None, s=None) == lib.MOE_OK
    assert L.moe_int8_pack_weights(_s(lib), None, FAKE, None) == lib.MOE_EINVAL
    assert L.moe_int8_pack_weights(_s(lib, K=131072), FAKE, FAKE, None) == lib.MOE_EUNSUPPORTED
    assert L.moe_int8_prepare_weights(_s(lib), FAKE, FAKE, None, None) == lib.MOE_EINVAL

    def dense(shape=None, c=FAKE, s=FAKE, p=FAKE, ws=FAKE, b=None, o=FAKE, ldo=60, odt=BF):
        return L.moe_gemm_int8(shape or _s(lib, E=1), c, s, p, ws, b, o, ldo, odt, None)

    for kw in [dict(c=None), dict(s=None), dict(p=None), dict(ws=None), dict(b=FAKE + 4),
               dict(o=None), dict(ldo=59), dict(odt=5), dict(shape=_s(lib, E=2))]:
        assert dense(**kw) == lib.MOE_EINVAL, kw
    assert dense(shape=_s(lib, E=1, K=131072)) == lib.MOE_EUNSUPPORTED
    assert dense(shape=_s(lib, E=1, R=0), c=None, s=None, o=None) == lib.MOE_OK

    def grp(src=None, div=1, nsrc=64, off=FAKE, shape=None):
        return L.moe_grouped_gemm_int8(shape or _s(lib), FAKE, FAKE, src, div, nsrc, off, FAKE,
                                       FAKE, None, FAKE, 60, BF, None)

    for kw in [dict(off=None), dict(nsrc=63), dict(src=FAKE, div=0), dict(src=FAKE, nsrc=0)]:
        assert grp(**kw) == lib.MOE_EINVAL, kw
    for kw in BAD:
        assert grp(shape=_s(lib, **kw)) == lib.MOE_EINVAL, kw


def test_norm_refusals(lib):
    L = lib.load()
    nan = float("nan")

    def pre(T=4, h=100, dt=BF, x=FAKE, w=None, eps=1e-6, z=FAKE, c=None, s=None, r=None):
        return L.moe_pre_norm(T, h, dt, x, w, eps, z, c, s, r, None)

    for kw in [dict(x=None), dict(z=None), dict(c=FAKE), dict(s=FAKE), dict(eps=0.0),
               dict(eps=nan), dict(eps=-1.0), dict(eps=1.0), dict(dt=F32), dict(T=-1), dict(h=0),
               dict(x=FAKE + 2), dict(w=FAKE + 2), dict(r=FAKE + 4)]:
        assert pre(**kw) == lib.MOE_EINVAL, kw
    assert pre(h=16385) == lib.MOE_EUNSUPPORTED
    assert pre(T=0, x=None, z=None) == lib.MOE_OK

    def post(T=4, h=100, dt=HF, res=FAKE, y=FAKE, w=None, g=None, t=None, a=1.0, eps=1e-6, u=FAKE,
             r=None, wn=None, z=None, c=None, s=None, rn=None):
        return L.moe_post_norm(T, h, dt, res, y, w, g, t, a, eps, u, r, wn, z, c, s, rn, None)

    for kw in [dict(res=None), dict(y=None), dict(u=None), dict(g=FAKE + 2), dict(t=FAKE + 4),
               dict(wn=FAKE), dict(rn=FAKE), dict(c=FAKE), dict(z=FAKE, s=FAKE), dict(eps=nan)]:
        assert post(**kw) == lib.MOE_EINVAL, kw
    assert post(h=20000) == lib.MOE_EUNSUPPORTED

    assert L.moe_norm_backward_workspace_bytes(4, 100) >= 2 * 4 * 100 * 4
    assert L.moe_norm_backward_workspace_bytes(4, 16385) == 0
    assert L.moe_norm_backward_workspace_bytes(-1, 16) == 0
    assert L.moe_norm_backward_workspace_bytes(0, 16) > 0

    def preb(T=4, h=100, dt=BF, dz=FAKE, x=FAKE, r=FAKE, w=None, d=None, dx=FAKE, dw=None,
             ws=FAKE):
        return L.moe_pre_norm_backward(T, h, dt, dz, x, r, w, d, dx, dw, ws, None)

    for kw in [dict(dz=None), dict(x=None), dict(r=None), dict(dx=None), dict(ws=None),
               dict(d=FAKE + 2), dict(dt=F32), dict(h=0)]:
        assert preb(**kw) == lib.MOE_EINVAL, kw

    def postb(T=4, h=100, dt=BF, du=FAKE, y=FAKE, r=FAKE, dz=None, u=None, rn=None, wn=None,
              dres=FAKE, dy=FAKE, dwn=None, ws=FAKE):
        return L.moe_post_norm_backward(T, h, dt, du, y, r, None, None, None, 1.0, dz, u, rn, wn,
                                        dres, dy, None, None, None, dwn, ws, None)

    for kw in [dict(y=None), dict(r=None), dict(dres=None), dict(dy=None), dict(ws=None),
               dict(du=None), dict(dz=FAKE), dict(dz=FAKE, u=FAKE), dict(dz=FAKE, rn=FAKE),
               dict(u=FAKE), dict(wn=FAKE), dict(dwn=FAKE), dict(rn=FAKE)]:
        assert postb(**kw) == lib.MOE_EINVAL, kw
    assert postb(h=16400) == lib.MOE_EUNSUPPORTED


def test_product_kernels_keep_their_registers():
    """The direct-load tiles hold up to 256 sums per lane and their fragments in registers: a spill
    inside their loop would wait for every load in flight."""
    import json
    from routing_expert_grouped_amd import build
    with open(os.path.join(build.BUILD, build.RESOURCES)) as f:
        usage = json.load(f)
    big = {k: v for k, v in usage.items() if "product_big_kernel" in k}
    assert len(big) == 5 * 4 + 2 * 2
    for name, v in big.items():
        assert v["VGPRs Spill"] == 0 and v["ScratchSize [bytes/lane]"] == 0, name


def test_binding_checks_without_gpu():
    torch = pytest.importorskip("torch")
    import routing_expert_grouped_amd as G
    from routing_expert_grouped_amd._launch import Launch, elt16

    sh = G.make_gemm_shape(4, 8, 8, 1)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        G.moe_grouped_gemm(sh, x, x, x)
    with pytest.raises(ValueError, match="dtype"):
        G.moe_quantize_int8(x.float())
    with pytest.raises(ValueError, match="shape"):
        G.moe_quantize_int8(torch.zeros(4, 7, dtype=torch.float16), swiglu=True)
    with pytest.raises(ValueError, match="shape"):
        G.moe_pre_norm(torch.zeros(4, dtype=torch.float16))
    with pytest.raises(ValueError, match="offsets"):
        G.moe_grouped_gemm_int8(sh, x, x, x, x, None)
    assert elt16(x, "x") == 0

    cpu = torch.device("cpu")
    L = Launch.__new__(Launch)
    L.device, L.index, L.handle, L._guards = cpu, -1, 0, ()
    wide = torch.zeros(6, 20, dtype=torch.float16)
    assert L.rows(wide[:, 4:12], "x", torch.float16, 8)[1:] == (20, 6)
    assert L.rows(wide[:1, 4:12], "x", torch.float16, 8)[1:] == (20, 1)
    with pytest.raises(ValueError, match="strides"):
        L.rows(wide.t(), "x", torch.float16, 6)
    with pytest.raises(ValueError, match="strides"):
        L.rows(wide[:1].expand(6, 20), "x", torch.float16, 20)
    with pytest.raises(ValueError, match="shape"):
        L.rows(wide, "x", torch.float16, 19)
    with pytest.raises(ValueError, match="shape"):
        L.rows(wide, "x", torch.float16, 20, 5)
    with pytest.raises(ValueError, match="contiguous"):
        L.dense(wide[:, :4], "x", torch.float16, 6, 4)
    with pytest.raises(ValueError, match="dtype"):
        L.dense(wide, "x", torch.float32, 6, 20)
    with pytest.raises(ValueError, match="bytes"):
        L.buffer(torch.zeros(7), "ws", 29)
    assert L.dense(None, "x", torch.float16, 3) is None
