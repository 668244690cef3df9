"""GPU parity of the ragged grouped products and the int8 products against their plain 64-bit forms,
within the bounds of tests/_plain_ops.py; int8 codes, scales and sums exactly."""
import pytest

from tests import _plain_ops as P
from tests._gpu_helpers import note, poisoned, require_gpu, torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _offsets(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return o


def _dev_i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _close(got, ref, bound, what):
    got = P.f8(got)
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, bad.nonzero()[0].tolist(),
                           got[bad][0].item(), ref[bad][0].item(), bound[bad][0].item())


# rows per expert: none, one, tile edges, and sizes that select each row tile
RAGGED = [
    [1], [0, 5, 0], [33, 0, 1, 31, 32], [64, 65, 63, 0, 2], [129, 128, 127], [0, 300, 3, 257],
    [1] * 70, [520, 9],
]
SIZES = [(64, 128), (1, 1), (8, 8), (200, 130), (63, 7), (65, 257), (136, 96), (40, 129)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("i", range(len(RAGGED)))
def test_grouped_products_ragged(i, dtype):
    G = require_gpu()
    counts = RAGGED[i]
    E, R = len(counts), sum(counts)
    off = _offsets(counts)
    for j, (K, N) in enumerate(SIZES):
        g = torch.Generator().manual_seed(100 * i + j)
        note(f"grouped {counts} K={K} N={N} {dtype}")
        x, dy = _rand(g, R, K, dtype=dtype), _rand(g, R, N, dtype=dtype)
        w = _rand(g, E, K, N, dtype=dtype, scale=K ** -0.5)
        sh = G.make_gemm_shape(R, K, N, E)
        xd, dyd, wd, od = x.cuda(), dy.cuda(), w.cuda(), _dev_i32(off)
        for odt in (dtype, F32):
            out = G.moe_grouped_gemm(sh, xd, wd, od, out=poisoned((R, N), odt))
            ref, mag = P.grouped(x, w, off)
            _close(out, ref, P.product_bound(ref, mag, K, odt), ("fwd", counts, K, N, odt))
            dx = G.moe_grouped_gemm_dgrad(sh, dyd, wd, od, out=poisoned((R, K), odt))
            ref, mag = P.grouped(dy, w, off, trans=True)
            _close(dx, ref, P.product_bound(ref, mag, N, odt), ("dgrad", counts, K, N, odt))
            dw = G.moe_grouped_gemm_wgrad(sh, xd, dyd, od, dw=poisoned((E, K, N), odt))
            ref, mag = P.wgrad(x, P.f8(dy), off)
            _close(dw, ref, P.product_bound(ref, mag, max(counts), odt), ("wgrad", counts, K, N))


@pytest.mark.parametrize("shape", [(700, 512, 768, 5, BF), (2100, 320, 512, 3, HF),
                                   (1500, 1024, 264, 2, BF), (96, 2048, 640, 40, BF)],
                         ids=lambda s: "x".join(map(str, s[:4])))
def test_grouped_products_larger(shape):
    """Sizes that take the larger tiles, with a skewed schedule."""
    G = require_gpu()
    R, K, N, E, dtype = shape
    g = torch.Generator().manual_seed(R)
    e = torch.multinomial(torch.arange(1, E + 1).double() ** -1.2, R, replacement=True,
                          generator=g)
    off = _offsets(torch.bincount(e, minlength=E).tolist())
    x, dy = _rand(g, R, K, dtype=dtype), _rand(g, R, N, dtype=dtype)
    w = _rand(g, E, K, N, dtype=dtype, scale=K ** -0.5)
    sh, od = G.make_gemm_shape(R, K, N, E), _dev_i32(off)
    note(f"grouped larger {shape}")
    out = G.moe_grouped_gemm(sh, x.cuda(), w.cuda(), od, out=poisoned((R, N), dtype))
    ref, mag = P.grouped(x, w, off)
    _close(out, ref, P.product_bound(ref, mag, K, dtype), "fwd")
    dx = G.moe_grouped_gemm_dgrad(sh, dy.cuda(), w.cuda(), od, out=poisoned((R, K), dtype))
    ref, mag = P.grouped(dy, w, off, trans=True)
    _close(dx, ref, P.product_bound(ref, mag, N, dtype), "dgrad")
    dw = G.moe_grouped_gemm_wgrad(sh, x.cuda(), dy.cuda(), od, dw=poisoned((E, K, N), F32))
    ref, mag = P.wgrad(x, P.f8(dy), off)
    _close(dw, ref, P.product_bound(ref, mag, R, F32), "wgrad")


@pytest.mark.parametrize("case", [([5000], 64, 64), ([3000, 0, 2100], 72, 40), ([9000], 65, 33),
                                  ([1100, 1500], 1, 3), ([4000, 70], 200, 128)], ids=str)
def test_weight_gradient_in_parts(case):
    """Small gradients over many rows are summed in parts, added in a fixed order: within the bound,
    the same twice, and with a caller's workspace."""
    G = require_gpu()
    counts, K, N = case
    E, R = len(counts), sum(counts)
    g = torch.Generator().manual_seed(K)
    x, dy, off = _rand(g, R, K), _rand(g, R, N), _offsets(counts)
    sh = G.make_gemm_shape(R, K, N, E)
    nws = G.moe_grouped_gemm_wgrad_workspace_bytes(sh)
    assert nws > 2 * E * K * N * 4
    for odt in (F32, BF):
        dw = G.moe_grouped_gemm_wgrad(sh, x.cuda(), dy.cuda(), _dev_i32(off),
                                      dw=poisoned((E, K, N), odt))
        ref, mag = P.wgrad(x, P.f8(dy), off)
        _close(dw, ref, P.product_bound(ref, mag, max(counts), odt), case)
        again = G.moe_grouped_gemm_wgrad(sh, x.cuda(), dy.cuda(), _dev_i32(off),
                                         dw=poisoned((E, K, N), odt),
                                         ws=poisoned((nws,), torch.uint8))
        assert torch.equal(dw, again)
    with pytest.raises(ValueError, match="ws"):
        G.moe_grouped_gemm_wgrad(sh, x.cuda(), dy.cuda(), _dev_i32(off),
                                 ws=torch.empty(nws - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("case", [(1000, 4, 8, 256, 512), (40, 2, 2, 136, 264), (2000, 2, 3, 512, 72)],
                         ids=str)
def test_gather_through_perm(case):
    """Tokens gathered through perm by the direct-load tiles, every row tile height."""
    G = require_gpu()
    T, k, E, K, N = case
    R = T * k
    g = torch.Generator().manual_seed(T)
    assign = torch.randint(0, E, (R,), generator=g)
    perm = torch.argsort(assign, stable=True).to(torch.int32)
    off = _offsets(torch.bincount(assign, minlength=E).tolist())
    x, w = _rand(g, T, K), _rand(g, E, K, N, scale=K ** -0.5)
    sh = G.make_gemm_shape(R, K, N, E)
    out = G.moe_grouped_gemm(sh, x.cuda(), w.cuda(), _dev_i32(off), perm=perm.cuda(), k=k,
                             out=poisoned((R, N), BF))
    ref, mag = P.grouped(x, w, off, (perm // k).long())
    _close(out, ref, P.product_bound(ref, mag, K, BF), case)


@pytest.mark.parametrize("dims", [(72, 136), (71, 33), (512, 256)], ids=str)
def test_gather_strides_and_foreign_rows(dims):
    """Rows gathered through perm, rows and outputs that are column slices of wider tensors, and
    infinities and NaN everywhere a product must not read or write: rows of no expert, columns
    beside the slices, weights of experts without rows."""
    G = require_gpu()
    K, N = dims
    T, k, E = 40, 3, 6
    g = torch.Generator().manual_seed(K)
    counts, first = [30, 0, 17, 1, 0, 60], 5
    off = _offsets(counts, first)
    R = T * k  # 5 rows before and 7 behind the experts' rows
    perm = torch.randperm(R, generator=g).to(torch.int32)
    used = perm[first:off[-1]]
    src = (perm // k).long()
    lead, pad = 8, 24
    wide = torch.full((T, K + pad), float("inf"), dtype=BF)
    x = _rand(g, T, K)
    unused = torch.ones(T, dtype=torch.bool)
    unused[(used // k).long()] = False
    x[unused] = float("nan")
    wide[:, lead:lead + K] = x
    w = _rand(g, E, K, N, scale=K ** -0.5)
    w[1], w[4] = float("nan"), float("inf")
    dy = _rand(g, R, N)
    dy[:first], dy[off[-1]:] = float("nan"), float("inf")
    sh, od, pd = G.make_gemm_shape(R, K, N, E), _dev_i32(off), perm.cuda()
    wided = wide.cuda()
    xv = wided[:, lead:lead + K]
    if xv.data_ptr() % 16:
        xv = wided[:, 8:8 + K]
    big = torch.full((R, N + 16), 7.0, dtype=BF, device="cuda")
    out = G.moe_grouped_gemm(sh, xv, w.cuda(), od, perm=pd, k=k, out=big[:, 8:8 + N])
    ref, mag = P.grouped(x, w, off, src)
    s = slice(first, off[-1])
    _close(out[s], ref[s], P.product_bound(ref[s], mag[s], K, BF), "gathered forward")
    keep = big.clone()
    keep[s, 8:8 + N] = 7.0
    assert (keep == 7.0).all(), "wrote outside the experts' rows or the slice"
    dx = torch.full((R, K), 7.0, dtype=BF, device="cuda")
    G.moe_grouped_gemm_dgrad(sh, dy.cuda(), w.cuda(), od, out=dx)
    ref, mag = P.grouped(dy, w, off, trans=True)
    _close(dx[s], ref[s], P.product_bound(ref[s], mag[s], N, BF), "dgrad")
    assert (dx[:first] == 7.0).all() and (dx[off[-1]:] == 7.0).all()
    dw = G.moe_grouped_gemm_wgrad(sh, xv, dy.cuda(), od, perm=pd, k=k,
                                  dw=poisoned((E, K, N), F32))
    ref, mag = P.wgrad(x, P.f8(dy), off, src)
    _close(dw, ref, P.product_bound(ref, mag, 64, F32), "gathered wgrad")
    assert (dw[1] == 0).all() and (dw[4] == 0).all()


def test_far_rows():
    """Rows more than 4 MB apart: beyond the direct loads' 32-bit offsets within a tile."""
    G = require_gpu()
    g = torch.Generator().manual_seed(3)
    R, K, N = 40, 64, 136
    x, dy, w = _rand(g, R, K), _rand(g, R, N), _rand(g, 1, K, N, scale=0.1)
    far = torch.empty(R, (1 << 21) + 8, dtype=BF, device="cuda")
    xv, dv = far[:, :K], far[:, 512:512 + N]
    xv.copy_(x)
    dv.copy_(dy)
    sh, off = G.make_gemm_shape(R, K, N, 1), _dev_i32([0, R])
    out = G.moe_grouped_gemm(sh, xv, w.cuda(), off)
    ref, mag = P.grouped(x, w, [0, R])
    _close(out, ref, P.product_bound(ref, mag, K, BF), "far rows")
    dw = G.moe_grouped_gemm_wgrad(sh, xv, dv, off)
    ref, mag = P.wgrad(x, P.f8(dy), [0, R])
    _close(dw, ref, P.product_bound(ref, mag, R, F32), "far rows' gradient")


@pytest.mark.parametrize("odt", [BF, HF, F32], ids=["bf16", "fp16", "f32"])
@pytest.mark.parametrize("case", [(700, 517, [300, 0, 400]), (8192, 1003, [8192]),
                                  (8200, 1799, [8, 8192]), (60, 131, [20, 0, 40])], ids=str)
def test_odd_output_widths(case, odt):
    """Outputs whose rows start at any element, and whose width is no whole run of four, at every tile
    of the direct loads, into a slice of a wider tensor whose other columns keep their values."""
    G = require_gpu()
    R, cols, counts = case
    sums, E, off = 72, len(counts), _offsets(counts)
    dt = BF if odt == F32 else odt
    g = torch.Generator().manual_seed(cols)
    dy, w = _rand(g, R, sums, dtype=dt), _rand(g, E, cols, sums, dtype=dt, scale=0.1)
    wide = torch.full((R, cols + 10), 7.0, dtype=odt, device="cuda")
    out = wide[:, :cols]
    note(f"odd widths {case} {odt}")
    G.moe_grouped_gemm_dgrad(G.make_gemm_shape(R, cols, sums, E), dy.cuda(), w.cuda(),
                             _dev_i32(off), out=out)
    ref, mag = P.grouped(dy, w, off, trans=True)
    _close(out, ref, P.product_bound(ref, mag, sums, odt), "input gradient")
    assert (wide[:, cols:] == 7).all()

    q = torch.randint(-127, 128, (E, cols, sums), generator=g, dtype=torch.int8)
    ws, bias = torch.rand(E, cols, generator=g) / sums, torch.randn(E, cols, generator=g)
    sh = G.make_gemm_shape(R, sums, cols, E)
    packed = G.moe_int8_pack_weights(sh, q.cuda())
    codes, scales = G.moe_quantize_int8(dy.cuda())
    wide.fill_(7.0)
    G.moe_grouped_gemm_int8(sh, codes, scales, packed, ws.cuda(), _dev_i32(off), bias=bias.cuda(),
                            out=out)
    ref, mag = _int8_ref(codes, scales, q, ws, bias, off, torch.arange(R))
    _close(out, ref, P.half_step(odt, ref) * (1 + 2.0 ** -8) + 4 * P.EPS24 * mag, "int8")
    assert (wide[:, cols:] == 7).all()


def test_dgrad_is_the_product_of_transposed_weights():
    """Weights stored [E][out][in] ("y = x W^T"), with tokens gathered through perm."""
    G = require_gpu()
    T, k, E, n_in, n_out = 50, 2, 3, 96, 72
    R = T * k
    g = torch.Generator().manual_seed(6)
    assign = torch.randint(0, E, (R,), generator=g)
    perm = torch.argsort(assign, stable=True).to(torch.int32)
    off = _offsets(torch.bincount(assign, minlength=E).tolist())
    x, w = _rand(g, T, n_in), _rand(g, E, n_out, n_in, scale=0.1)
    out = G.moe_grouped_gemm_dgrad(G.make_gemm_shape(R, n_out, n_in, E), x.cuda(), w.cuda(),
                                   _dev_i32(off), perm=perm.cuda(), k=k)
    ref, mag = P.grouped(x, w, off, (perm // k).long(), trans=True)
    _close(out, ref, P.product_bound(ref, mag, n_in, BF), "x W^T")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts", [[20], [700]], ids=["few", "many"])
def test_smallest_and_largest_values(counts, dtype):
    """Subnormal rows against large weights, and products near the end of the type's range."""
    G = require_gpu()
    R, K, N = counts[0], 128, 256
    g = torch.Generator().manual_seed(R)
    tiny = torch.finfo(dtype).tiny
    x = (torch.randn(R, K, generator=g).double() * tiny / 16).to(dtype)
    w = _rand(g, 1, K, N, dtype=dtype, scale=float(torch.finfo(dtype).max) ** 0.5 / 8)
    sh, off = G.make_gemm_shape(R, K, N, 1), _dev_i32([0, R])
    out = G.moe_grouped_gemm(sh, x.cuda(), w.cuda(), off, out_dtype=F32)
    ref, mag = P.grouped(x, w, [0, R])
    _close(out, ref, P.product_bound(ref, mag, K, F32), "subnormal rows")
    x = _rand(g, R, K, dtype=dtype, scale=float(torch.finfo(dtype).max) ** 0.5 / 64)
    out = G.moe_grouped_gemm(sh, x.cuda(), w.cuda(), off)
    ref, mag = P.grouped(x, w, [0, R])
    assert torch.isfinite(out).all()
    _close(out, ref, P.product_bound(ref, mag, K, dtype), "large values")


def test_infinities_stay_in_their_rows():
    G = require_gpu()
    g = torch.Generator().manual_seed(9)
    counts, K, N = [40, 40], 96, 160
    off, R = _offsets(counts), 80
    x, w = _rand(g, R, K), _rand(g, 2, K, N)
    x[3, 5], x[50, 7] = float("nan"), float("inf")
    out = G.moe_grouped_gemm(G.make_gemm_shape(R, K, N, 2), x.cuda(), w.cuda(), _dev_i32(off))
    ok = torch.isfinite(out).all(dim=1).cpu()
    assert not ok[3] and not ok[50] and ok.sum() == R - 2
    assert torch.isnan(out[3]).all()


def test_no_rows_and_clamped_offsets():
    """R = 0: nothing is launched but the zero weight gradient; offsets beyond R or descending are
    taken as clamped and ascending."""
    G = require_gpu()
    K, N, E = 24, 40, 3
    w = torch.randn(E, K, N).to(BF).cuda()
    sh = G.make_gemm_shape(0, K, N, E)
    e0 = torch.empty(0, K, dtype=BF, device="cuda")
    off = _dev_i32([0, 0, 0, 0])
    assert G.moe_grouped_gemm(sh, e0, w, off).shape == (0, N)
    dw = G.moe_grouped_gemm_wgrad(sh, e0, torch.empty(0, N, dtype=BF, device="cuda"), off,
                                  dw=poisoned((E, K, N), F32))
    assert (dw == 0).all()
    R = 20
    g = torch.Generator().manual_seed(1)
    x = _rand(g, R, K)
    out = torch.full((R, N), 7.0, dtype=BF, device="cuda")
    G.moe_grouped_gemm(G.make_gemm_shape(R, K, N, E), x.cuda(), w, _dev_i32([-4, 6, 2, 900]),
                       out=out)
    # expert 0: rows 0..5, expert 1: none (2 < 6), expert 2: rows 2..19, where 2..5 are also 0's
    ref, mag = P.grouped(x, w, [0, 2, 2, 20])
    _close(out[6:], ref[6:], P.product_bound(ref, mag, K, BF)[6:], "clamped")


def test_many_experts_few_rows():
    G = require_gpu()
    E, K, N, R = 1024, 96, 80, 50
    g = torch.Generator().manual_seed(2)
    e = torch.randint(0, E, (R,), generator=g)
    off = _offsets(torch.bincount(e, minlength=E).tolist())
    x, w = _rand(g, R, K), _rand(g, E, K, N, scale=0.1)
    out = G.moe_grouped_gemm(G.make_gemm_shape(R, K, N, E), x.cuda(), w.cuda(), _dev_i32(off),
                             out=poisoned((R, N), BF))
    ref, mag = P.grouped(x, w, off)
    _close(out, ref, P.product_bound(ref, mag, K, BF), "1024 experts")


# ---------------------------------------------------------------------------------------------------
# int8
# ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("K", [1, 7, 8, 127, 128, 511, 513, 1000, 2048, 4100, 6144, 8192, 9000,
                               16384])
def test_quantise_exact(K, dtype):
    G = require_gpu()
    R = 9
    g = torch.Generator().manual_seed(K)
    x = _rand(g, R, K, dtype=dtype, scale=3.0)
    x[1] = 0
    x[2] = x[2].sign() * x[2].abs().amax()          # every code at the end of the range
    x[3, 0], x[3, 1:] = 2.0, 1.0                     # exact ties: 63.5 goes to 64
    x[4] = torch.finfo(dtype).tiny * torch.randint(0, 9, (K,), generator=g).to(dtype) / 8
    x[5] = x[5] * (torch.finfo(dtype).max / 64 if dtype == BF else 64)
    x[6, K // 2] = 1000.0
    note(f"quantise K={K} {dtype}")
    codes, scales = G.moe_quantize_int8(x.cuda(), codes=poisoned((R, (K + 127) // 128 * 128),
                                                                 torch.int8),
                                        scales=poisoned((R,), F32))
    ref, amax = P.quantise(P.f8(x))
    got = codes.cpu()
    assert (got[:, K:] == 0).all()
    assert torch.equal(got[:, :K].to(P.F8), ref)
    assert torch.equal(scales.cpu(), P.scale32(amax))


def test_quantise_strided_and_not_finite():
    G = require_gpu()
    g = torch.Generator().manual_seed(5)
    wide = _rand(g, 70, 400)
    x = wide[:, 16:316]
    codes, scales = G.moe_quantize_int8(wide.cuda()[:, 16:316])
    ref, amax = P.quantise(P.f8(x))
    assert torch.equal(codes.cpu()[:, :300].to(P.F8), ref)
    assert torch.equal(scales.cpu(), P.scale32(amax))
    x = _rand(g, 4, 64)
    x[1, 3], x[2, 4] = float("nan"), float("-inf")
    _, scales = G.moe_quantize_int8(x.cuda())
    fin = torch.isfinite(scales).cpu().tolist()
    assert fin == [True, False, False, True] and torch.isnan(scales[1])
    empty, s0 = G.moe_quantize_int8(torch.empty(0, 64, dtype=BF, device="cuda"))
    assert empty.shape == (0, 128) and s0.shape == (0,)


@pytest.mark.parametrize("m", [5, 128, 1000, 2048])
def test_quantise_swiglu(m):
    """silu(G) U is formed in float32: with a relative error of at most 2^-20 (the hardware
    exponential and reciprocal, three products), a code differs only where the 64-bit quotient is
    within 127 2^-19 of a rounding border, and then by one."""
    G = require_gpu()
    g = torch.Generator().manual_seed(m)
    x = _rand(g, 33, 2 * m, scale=2.0)
    codes, scales = G.moe_quantize_int8(x.cuda(), swiglu=True)
    a, b = P.f8(x[:, :m]), P.f8(x[:, m:])
    h = a / (1 + torch.exp(-a)) * b
    ref, amax = P.quantise(h)
    q = 127.0 * h / amax[:, None]
    got = codes.cpu()[:, :m].to(P.F8)
    near = ((q - torch.floor(q)) - 0.5).abs() <= 127 * 2.0 ** -19
    assert ((got - ref).abs() <= near.to(P.F8)).all()
    assert ((P.f8(scales) * 127 - amax).abs() <= amax * 2.0 ** -19).all()


def _int8_ref(codes, scales, q, ws, bias, off, src):
    c, s = P.f8(codes)[:, :q.shape[2]], P.f8(scales)
    R = len(src)
    out = torch.full((R, q.shape[1]), float("nan"), dtype=P.F8)
    mag = torch.zeros_like(out)
    for e, a, b in P.segments(off):
        if a < b:
            y = c[src[a:b]] @ P.f8(q[e]).t() * s[src[a:b]][:, None] * P.f8(ws[e])[None]
            bb = P.f8(bias[e])[None] if bias is not None else 0.0
            out[a:b] = y + bb
            mag[a:b] = 2 * y.abs() + out[a:b].abs()
    return out, mag


@pytest.mark.parametrize("case", [
    (1, 64, 16), (3, 100, 60), (17, 513, 33), (33, 128, 129), (70, 1000, 200), (130, 2048, 256),
    (300, 384, 520), (16, 7168, 96), (600, 256, 1024)], ids=str)
def test_gemm_int8(case):
    """The integer sum is exact; the two scale products, the bias and a sum beyond 2^24 each round
    once in float32, the output once more."""
    G = require_gpu()
    R, K, N = case
    g = torch.Generator().manual_seed(K + N)
    x = _rand(g, R, K)
    q = torch.randint(-128, 128, (1, N, K), generator=g, dtype=torch.int8)
    ws = torch.rand(1, N, generator=g) + 0.5
    bias = torch.randn(1, N, generator=g) * 100
    sh = G.make_gemm_shape(R, K, N)
    note(f"int8 {case}")
    packed = G.moe_int8_pack_weights(sh, q.cuda())
    codes, scales = G.moe_quantize_int8(x.cuda())
    for b in (None, bias):
        for odt in (BF, HF, F32):
            s = ws * (1e-4 if odt == HF else 1.0)
            out = G.moe_gemm_int8(sh, codes, scales, packed, s.cuda(), out=poisoned((R, N), odt),
                                  bias=b.cuda() if b is not None else None)
            ref, mag = _int8_ref(codes, scales, q, s, b, [0, R], torch.arange(R))
            _close(out, ref, P.half_step(odt, ref) * (1 + 2.0 ** -8) + 4 * P.EPS24 * mag,
                   (case, odt))


def test_gemm_int8_widest_sums():
    """Sums at the ends of the 32-bit range stay exact (K = 131071, the widest covered)."""
    G = require_gpu()
    K, N, R = 131071, 2, 2
    pitch = G.moe_int8_pitch(K)
    codes = torch.zeros(R, pitch, dtype=torch.int8)
    codes[0, :K], codes[1, :K] = -128, 127
    q = torch.full((1, N, K), -128, dtype=torch.int8)
    q[0, 1] = 127
    sh = G.make_gemm_shape(R, K, N)
    one = torch.ones(2, device="cuda")
    out = G.moe_gemm_int8(sh, codes.cuda(), one, G.moe_int8_pack_weights(sh, q.cuda()),
                          one.view(1, 2), out_dtype=F32)
    want = torch.tensor([[128. * 128 * K, -128. * 127 * K], [-127. * 128 * K, 127. * 127 * K]],
                        dtype=P.F8)
    assert torch.equal(out.cpu(), want.to(F32))


@pytest.mark.parametrize("case", [(16, 2, 8, 96, 64), (40, 3, 5, 200, 130), (300, 4, 6, 512, 256),
                                  (9, 8, 64, 1024, 80), (500, 2, 3, 128, 300)], ids=str)
def test_grouped_gemm_int8(case):
    G = require_gpu()
    T, k, E, K, N = case
    R = T * k
    g = torch.Generator().manual_seed(R + K)
    assign = torch.randint(0, E, (R,), generator=g)
    assign[assign == E // 2] = 0  # one expert without rows
    perm = torch.argsort(assign, stable=True).to(torch.int32)
    off = _offsets(torch.bincount(assign, minlength=E).tolist())
    x = _rand(g, T, K)
    q = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8)
    ws = torch.rand(E, N, generator=g) / K
    bias = torch.randn(E, N, generator=g)
    sh = G.make_gemm_shape(R, K, N, E)
    packed = G.moe_int8_pack_weights(sh, q.cuda())
    codes, scales = G.moe_quantize_int8(x.cuda())
    od = _dev_i32(off)
    out = G.moe_grouped_gemm_int8(sh, codes, scales, packed, ws.cuda(), od, perm=perm.cuda(), k=k,
                                  bias=bias.cuda(), out=poisoned((R, N), BF))
    src = (perm // k).long()
    ref, mag = _int8_ref(codes, scales, q, ws, bias, off, src)
    _close(out, ref, P.half_step(BF, ref) * (1 + 2.0 ** -8) + 4 * P.EPS24 * mag, case)
    rc, rs = codes[src.cuda()].contiguous(), scales[src.cuda()].contiguous()
    again = G.moe_grouped_gemm_int8(sh, rc, rs, packed, ws.cuda(), od, bias=bias.cuda())
    assert torch.equal(out, again)


@pytest.mark.parametrize("dims", [(3, 100, 40), (2, 256, 128), (1, 130, 65)], ids=str)
def test_int8_prepare_weights(dims):
    """Quantised per column like the rows, and packed as the codes themselves pack."""
    G = require_gpu()
    E, K, N = dims
    g = torch.Generator().manual_seed(K)
    w = _rand(g, E, K, N)
    w[0, :, 1] = 0
    sh = G.make_gemm_shape(1, K, N, E)
    packed, ws = G.moe_int8_prepare_weights(sh, w.cuda())
    codes = torch.empty(E, N, K, dtype=torch.int8)
    for e in range(E):
        c, amax = P.quantise(P.f8(w[e]).t().contiguous())
        codes[e] = c.to(torch.int8)
        assert torch.equal(ws[e].cpu(), P.scale32(amax))
    assert torch.equal(packed, G.moe_int8_pack_weights(sh, codes.cuda()))


# ---------------------------------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------------------------------
def test_other_stream_and_graph_replays():
    """A call on another stream, and a captured chain replayed with new inputs and eager work
    between the replays, give the eager results bit for bit."""
    G = require_gpu()
    T, k, E, K, N = 64, 2, 4, 160, 136
    R = T * k
    g = torch.Generator().manual_seed(11)
    assign = torch.randint(0, E, (R,), generator=g)
    perm = torch.argsort(assign, stable=True).to(torch.int32).cuda()
    od = _dev_i32(_offsets(torch.bincount(assign, minlength=E).tolist()))
    xs = [_rand(g, T, K).cuda() for _ in range(3)]
    w = _rand(g, E, K, N).cuda()
    q = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8).cuda()
    ws = (torch.rand(E, N, generator=g) / K).cuda()
    sh = G.make_gemm_shape(R, K, N, E)
    packed = G.moe_int8_pack_weights(sh, q)

    def chain(x):
        a = G.moe_grouped_gemm(sh, x, w, od, perm=perm, k=k)
        dw = G.moe_grouped_gemm_wgrad(sh, x, a, od, perm=perm, k=k)
        dx = G.moe_grouped_gemm_dgrad(sh, a, w, od)
        c, s = G.moe_quantize_int8(x)
        return a, dw, dx, G.moe_grouped_gemm_int8(sh, c, s, packed, ws, od, perm=perm, k=k)

    want = [[t.clone() for t in chain(x)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = G.moe_grouped_gemm(sh, xs[1], w, od, perm=perm, k=k, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want[1][0])
    x = xs[0].clone()
    with torch.cuda.stream(side):
        chain(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(x)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
        chain(xs[2 - i])  # eager work between the replays
