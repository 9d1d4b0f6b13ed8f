"""The gated feed-forward block against its formulas in 64 bits.

Bounds.  g and u are fp32 sums (D 2^-24 of their terms' magnitudes); act and
its derivative are Lipschitz with constants below 1.13 and 1 (silu, gelu), and
the hardware's exponential and reciprocal add 2^-20 relatively.  h, dg and du
are rounded to bf16 once, and the products of dg and du once more."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
from train_reference import HALF_BF16, HALF_F32, act, act8_bytes, inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FAST = 2.0 ** -19


def inputs(t, d, f, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return ((r(t, d)).to(torch.bfloat16), (r(f, d) / d ** 0.5).to(torch.bfloat16),
            (r(f, d) / d ** 0.5).to(torch.bfloat16), r(t, f).to(torch.bfloat16))


def products(x, wg, wu):
    X, G, U = x.double(), wg.double(), wu.double()
    e = 1.01 * X.shape[1] * HALF_F32
    return X @ G.t(), X @ U.t(), e * (X.abs() @ G.abs().t()), e * (X.abs() @ U.abs().t())


def check_h(h, g, u, ge, ue, kind, what):
    a, _ = act(g, kind)
    ref = a * u
    b = 1.13 * ge * (u.abs() + ue) + a.abs() * ue + FAST * (a.abs() + g.abs() * 2.0 ** -4) * u.abs()
    inside(h.to(ref.device), ref, HALF_BF16 * ref.abs() + 1.01 * b + 1e-38, what)


def check_back(got, dh, X, g, u, ge, ue, wg, wu, kind, what):
    """X, g, u: float64 values the gradients are those of; ge, ue: how far the
    operator's own g and u may be from them."""
    dx, dwg, dwu = got
    D, G, U = dh.double(), wg.double(), wu.double()
    a, da = act(g, kind)
    dg, du = D * u * da, D * a
    # |act''| < 1.2 for both
    dge = HALF_BF16 * dg.abs() + D.abs() * (ue * da.abs() + (u.abs() + ue) * 1.2 * ge + FAST * u.abs() * (da.abs() + 1))
    due = HALF_BF16 * du.abs() + D.abs() * (1.13 * ge + FAST * (a.abs() + g.abs() * 2.0 ** -4))
    t, f = D.shape
    ref = dg @ G + du @ U
    terms = dg.abs() @ G.abs() + du.abs() @ U.abs()
    inside(dx.to(ref.device), ref, HALF_BF16 * ref.abs() + 1.02 * (dge @ G.abs() + due @ U.abs() + 2 * f * HALF_F32 * terms)
           + 1e-38, f"{what} dx")
    for name, got_w, v, ve in (("dw_gate", dwg, dg, dge), ("dw_up", dwu, du, due)):
        ref = v.t() @ X
        b = ve.t() @ X.abs() + t * HALF_F32 * (v.abs().t() @ X.abs())
        inside(got_w.to(ref.device), ref, HALF_BF16 * ref.abs() + 1.02 * b + 1e-38, f"{what} {name}")


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 5, 3), (16, 64, 32), (33, 40, 31), (65, 64, 65), (64, 96, 96), (128, 128, 128),
          (130, 200, 129), (300, 72, 257), (257, 256, 520), (40, 1000, 100), (600, 33, 64)]


@pytest.mark.parametrize("t,d,f", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward_and_backward(t, d, f, kind):
    x, wg, wu, dh = inputs(t, d, f, t + d + f)
    xd, gd, ud, dhd = (a.to(DEV) for a in (x, wg, wu, dh))
    g, u, ge, ue = products(x, wg, wu)
    h = z.glu_forward(xd, gd, ud, act=kind)
    check_h(h, g, u, ge, ue, kind, f"{kind} {t}x{d}x{f} h")
    h2 = torch.empty_like(h)
    got = z.glu_backward(dhd, xd, gd, ud, act=kind, h=h2)
    assert torch.equal(h, h2)
    check_back(got, dh, x.double(), g, u, ge, ue, wg, wu, kind, f"{kind} {t}x{d}x{f}")


@pytest.mark.parametrize("t,d,f", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_checkpoint_and_backward_from_it(t, d, f, kind):
    x, wg, wu, dh = inputs(t, d, f, 2 * t + d + f)
    xd, gd, ud, dhd = (a.to(DEV) for a in (x, wg, wu, dh))
    h, (cg, cu) = z.glu_forward(xd, gd, ud, act=kind, checkpoint=True)
    assert torch.equal(h, z.glu_forward(xd, gd, ud, act=kind))
    g, u, ge, ue = products(x, wg, wu)
    for name, c, v, e in (("g", cg, g, ge), ("u", cu, u, ue)):
        # each value is the nearest e4m3 of a product within its error
        want, byte = act8_bytes(v)
        got = z.act8_unpack(c).cpu().double()
        step = (2.0 ** (byte.double() - 127 - 10)).repeat_interleave(32, 1)[:, :f]
        # (a block's scale may be a power of two larger where its largest value lies at the border)
        inside(got, v, torch.maximum(2.0 ** -4 * v.abs(), 2 * step) + 1.07 * e, f"{name} checkpoint")
    xc = z.act8_pack(xd)
    X = z.act8_unpack(xc).cpu().double()
    kg, ku = z.act8_unpack(cg).cpu().double(), z.act8_unpack(cu).cpu().double()
    zero = torch.zeros_like(kg)
    hb = torch.empty_like(h)
    got = z.glu_backward(dhd, xc, gd, ud, act=kind, checkpoint=(cg, cu), h=hb)
    check_back(got, dh, X, kg, ku, zero, zero, wg, wu, kind, f"{kind} {t}x{d}x{f} act8")
    check_h(hb, kg, ku, zero, zero, kind, "h from the checkpoint")
    # x itself beside the checkpoint, and x's checkpoint alone
    got = z.glu_backward(dhd, xd, gd, ud, act=kind, checkpoint=(cg, cu))
    check_back(got, dh, x.double(), kg, ku, zero, zero, wg, wu, kind, "x in bf16")
    got = z.glu_backward(dhd, xc, gd, ud, act=kind)
    g, u, ge, ue = products(X, wg, wu)
    check_back(got, dh, X, g, u, ge, ue, wg, wu, kind, "x8 alone")


def test_no_rows():
    w = torch.ones((40, 24), dtype=torch.bfloat16, device=DEV)
    x = torch.empty((0, 24), dtype=torch.bfloat16, device=DEV)
    h, kept = z.glu_forward(x, w, w, checkpoint=True)
    assert tuple(h.shape) == (0, 40)
    dx, dg, du = z.glu_backward(h, x, w, w, checkpoint=kept)
    assert tuple(dx.shape) == (0, 24) and not bool(dg.any()) and not bool(du.any())


def test_fused_weight_views_and_flat_gradients():
    """gate and up as halves of one weight, x, dh and h as column slices, the
    gradients in a flat vector at an odd offset."""
    t, d, f = 77, 60, 90
    g = torch.Generator().manual_seed(3)
    W = (torch.randn((2 * f, d + 5), generator=g) / 8).to(torch.bfloat16)
    X = torch.randn((2 * t, d + 9), generator=g).to(torch.bfloat16)
    H = torch.randn((t, f + 3), generator=g).to(torch.bfloat16)
    w, x, dh = W.to(DEV)[:, 2:2 + d], X.to(DEV)[::2, 5:5 + d], H.to(DEV)[:, 1:1 + f]
    out = torch.full((t, f + 4), 5.0, dtype=torch.bfloat16, device=DEV)
    h = z.glu_forward(x, w[:f], w[f:], out=out[:, 3:3 + f])
    assert h.data_ptr() == out[:, 3:].data_ptr()
    assert bool((out[:, :3] == 5).all() and (out[:, 3 + f:] == 5).all())
    xc, wc, dc = x.cpu(), w.cpu(), dh.cpu()
    pg, pu, ge, ue = products(xc, wc[:f], wc[f:])
    check_h(h, pg, pu, ge, ue, "silu", "h")
    flat = torch.full((2 * f * d + 3,), 5.0, dtype=torch.bfloat16, device=DEV)
    dw = flat[1:1 + 2 * f * d].view(2 * f, d)
    got = z.glu_backward(dh, x, w[:f], w[f:], dw_gate=dw[:f], dw_up=dw[f:])
    check_back(got, dc, xc.double(), pg, pu, ge, ue, wc[:f], wc[f:], "silu", "views")
    assert float(flat[0]) == 5 and bool((flat[1 + 2 * f * d:] == 5).all())


def test_not_finite_inputs_stay_in_their_rows():
    x, wg, wu, dh = inputs(70, 48, 100, 5)
    x[3, 7] = float("nan")
    x[9, 0] = float("inf")
    h, (cg, cu) = z.glu_forward(x.to(DEV), wg.to(DEV), wu.to(DEV), checkpoint=True)
    bad = torch.zeros(70, dtype=torch.bool)
    bad[[3, 9]] = True
    assert bool(torch.isfinite(h.float().cpu()[~bad]).all()) and bool(torch.isnan(h[3]).all())
    back = z.act8_unpack(cg).cpu().float()
    assert bool(torch.isfinite(back[~bad]).all()) and bool(torch.isnan(back[bad]).all())


def test_gradient_against_differences():
    x, wg, wu, dh = inputs(10, 16, 24, 6)
    for kind in ("silu", "gelu"):
        got = z.glu_backward(dh.to(DEV), x.to(DEV), wg.to(DEV), wu.to(DEV), act=kind)
        f = lambda a, b, c: (act(a @ b.t(), kind)[0] * (a @ c.t()) * dh.double()).sum()  # noqa: E731
        at = [a.double() for a in (x, wg, wu)]
        g = torch.Generator().manual_seed(7)
        for _ in range(8):
            u = [torch.randn(a.shape, generator=g).double() for a in at]
            e = 1e-5
            num = (f(*(a + e * b for a, b in zip(at, u))) - f(*(a - e * b for a, b in zip(at, u)))) / (2 * e)
            ana = sum((a.cpu().double() * b).sum() for a, b in zip(got, u))
            size = sum((a.cpu().double() * b).abs().sum() for a, b in zip(got, u))
            assert abs(float(num - ana)) <= 4 * HALF_BF16 * float(size)


def test_another_stream_and_graph():
    x, wg, wu, dh = (a.to(DEV) for a in inputs(300, 96, 200, 8))

    def step(**kw):
        h, kept = z.glu_forward(x, wg, wu, checkpoint=True, **kw)
        return (h, *z.glu_backward(dh, z.act8_pack(x, **kw), wg, wu, checkpoint=kept, **kw))

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(stream=s)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        for a, b in zip((x, wg, wu, dh), inputs(300, 96, 200, 30 + k)):
            a.copy_(b.to(DEV))
        want = [a.clone() for a in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
