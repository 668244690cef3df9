"""The plain 64-bit forms that the GPU tests compare with: their gradients against central
differences of their forward passes, and the rounding rules on hand cases (CPU)."""
import torch

from tests import _plain_ops as P

F8 = P.F8


def _diff(f, x, step=1e-6):
    """Central differences of a scalar function of x."""
    g = torch.zeros_like(x)
    flat, gf = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + step
        hi = f()
        flat[i] = keep - step
        lo = f()
        flat[i] = keep
        gf[i] = (hi - lo) / (2 * step)
    return g


def test_post_norm_gradients_are_differences():
    g = torch.Generator().manual_seed(3)
    T, h, eps, a = 3, 5, 2.0 ** -10, 0.75
    res, y, ca, cz = (torch.randn(T, h, generator=g, dtype=F8) for _ in range(4))
    w, gate, wn = (1 + 0.3 * torch.randn(h, generator=g, dtype=F8) for _ in range(3))
    tau = torch.rand(T, generator=g, dtype=F8)

    def loss():
        u, _, _ = P.post_norm(res, y, w, gate, tau, a, eps)
        z = u * P.rstd(u, eps)[:, None] * wn
        return ((u * ca).sum() + (z * cz).sum()).item()

    u, r, _ = P.post_norm(res, y, w, gate, tau, a, eps)
    got = P.post_norm_grads(ca, y, r, w, gate, tau, a, cz, u, P.rstd(u, eps), wn)
    for name, x in (("dres", res), ("dy", y), ("dw", w), ("dgate", gate), ("dtoken_gate", tau),
                    ("dw_next", wn)):
        assert torch.allclose(got[name][0], _diff(loss, x), rtol=1e-7, atol=1e-8), name


def test_grouped_gradients_are_differences():
    g = torch.Generator().manual_seed(4)
    off, src = [0, 2, 2, 5], [1, 0, 2, 2, 1]
    x = torch.randn(3, 4, generator=g, dtype=F8)
    w = torch.randn(3, 4, 3, generator=g, dtype=F8)
    c = torch.randn(5, 3, generator=g, dtype=F8)

    def loss():
        return (P.grouped(x, w, off, src)[0] * c).sum().item()

    dw, _ = P.wgrad(x, c, off, src)
    assert torch.allclose(dw, _diff(loss, w), rtol=1e-8, atol=1e-8)
    drow, _ = P.grouped(c, w, off, trans=True)  # per routed row; a token's gradient is their sum
    dx = torch.zeros_like(x).index_add_(0, torch.tensor(src), drow)
    assert torch.allclose(dx, _diff(loss, x), rtol=1e-8, atol=1e-8)


def test_quantise_ties_and_zero_rows():
    p = torch.tensor([[2.0, 1.0, -1.0, 0.0], [0.0, 0.0, 0.0, 0.0]], dtype=F8)
    codes, amax = P.quantise(p)
    assert codes.tolist() == [[127, 64, -64, 0], [0, 0, 0, 0]]  # 63.5 goes to even
    assert amax.tolist() == [2.0, 0.0]
