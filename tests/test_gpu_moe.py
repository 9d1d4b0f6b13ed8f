"""The experts' gated feed-forward against its formulas in 64 bits, within
bounds that count the roundings (layer_reference)."""
import math

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z
from train_reference import inside

DEV = torch.device("cuda:0")
NAMES = ("dx", "dw_gate", "dw_up", "dw_down", "dweights")


def inputs(t, d, f, e, top, seed, skew=0.5, none=0.1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, dy = r(t, d).to(torch.bfloat16), r(t, d).to(torch.bfloat16)
    wg, wu, wd = ((r(e, a, b) / b ** 0.5).to(torch.bfloat16) for a, b in ((f, d), (f, d), (d, f)))
    score = r(t, e) + skew * r(1, e)
    chosen = score.topk(min(top, e), 1).indices.to(torch.int32)
    if top > e:
        chosen = torch.cat([chosen, chosen[:, :1].expand(t, top - e)], 1)  # the same one again
    chosen = chosen.masked_fill(torch.rand(chosen.shape, generator=g) < none, -1)
    return x, dy, wg, wu, wd, chosen, torch.rand((t, top), generator=g) * (chosen >= 0)


def check(x, dy, wg, wu, wd, chosen, share, kind, what, y=None, grads=None):
    """The operator's results (its own calls if not given) against the formulas."""
    D = [v.to(DEV) for v in (x, dy, wg, wu, wd, chosen, share)]
    r = z.moe_plan(D[5], D[6], wg.shape[0])
    y = z.moe_forward(D[0], *D[2:5], r, act=kind) if y is None else y
    grads = z.moe_backward(D[1], D[0], *D[2:5], r, act=kind) if grads is None else grads
    dev = lambda v: v.double().to(DEV)  # noqa: E731 (products of 64 bits, on the GPU for speed)
    live = (chosen >= 0).any(1).unsqueeze(1)
    (ry, ey), back = ref.moe(dev(torch.where(live, x, 0)), dev(wg), dev(wu), dev(wd), D[5], dev(share), kind,
                             dev(torch.where(live, dy, 0)))
    inside(y, ry, ey, f"{what} y")
    for name, got, (want, bound) in zip(NAMES, grads, back):
        inside(got, want, bound, f"{what} {name}")
    return y, grads


SHAPES = [  # tokens, width, an expert's, experts, experts of a token
    (1, 1, 1, 1, 1), (1, 8, 8, 2, 2), (2, 5, 3, 3, 2), (5, 16, 24, 4, 6), (16, 64, 32, 4, 2), (33, 40, 31, 5, 3),
    (65, 64, 65, 7, 2), (64, 96, 96, 64, 8), (130, 200, 129, 3, 1), (257, 72, 257, 9, 4), (300, 256, 520, 4, 2),
    (40, 1000, 100, 16, 2), (900, 33, 64, 2, 1), (700, 264, 136, 1, 1), (12, 512, 256, 1000, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f,e,top", SHAPES)
def test_forward_and_backward(t, d, f, e, top, kind):
    check(*inputs(t, d, f, e, top, t + d + f), kind, f"{kind} {t}x{d}x{f} e{e} k{top}")


@pytest.mark.gpu
@pytest.mark.parametrize("t,d,f,e,top", [(1500, 512, 384, 6, 2), (2100, 776, 1032, 3, 2), (4000, 128, 1000, 40, 4)])
def test_more_rows_than_a_tile(t, d, f, e, top):
    check(*inputs(t, d, f, e, top, t, skew=1.5), "silu", f"{t}x{d}x{f} e{e} k{top}")


@pytest.mark.gpu
def test_one_expert_has_all_and_experts_without_tokens():
    x, dy, wg, wu, wd, chosen, share = inputs(300, 64, 72, 6, 2, 3)
    chosen[:] = 4
    chosen[:, 1] = -1
    y, grads = check(x, dy, wg, wu, wd, chosen, share, "silu", "one")
    for k in range(1, 4):
        assert not grads[k][:4].any() and not grads[k][5].any()
    chosen[:] = -1
    D = [v.to(DEV) for v in (x, dy, wg, wu, wd, chosen, share)]
    r = z.moe_plan(D[5], D[6], 6)
    assert not z.moe_forward(D[0], *D[2:5], r).any()
    out = [torch.full_like(v, math.nan) for v in grads]
    z.moe_backward(D[1], D[0], *D[2:5], r, dx=out[0], dw_gate=out[1], dw_up=out[2], dw_down=out[3], dweights=out[4])
    assert not any(v.any() for v in out)
    # ... and no tokens at all
    r = z.moe_plan(D[5][:0], D[6][:0], 6)
    assert z.moe_forward(D[0][:0], *D[2:5], r).shape == (0, 64)
    got = z.moe_backward(D[1][:0], D[0][:0], *D[2:5], r)
    assert got[0].shape == (0, 64) and not any(v.any() for v in got)


@pytest.mark.gpu
def test_rows_without_an_expert_reach_nothing():
    x, dy, wg, wu, wd, chosen, share = inputs(200, 48, 40, 5, 2, 4)
    gone = torch.arange(200) % 3 == 0
    chosen[gone] = -1
    want = [v.clone() for v in (x, dy)]
    x[gone], dy[gone], share[gone] = math.nan, math.inf, math.nan
    y, grads = check(x, dy, wg, wu, wd, chosen, torch.where(gone.unsqueeze(1), 0, share), "gelu", "padded")
    D = [v.to(DEV) for v in (x, dy, wg, wu, wd, chosen, share)]
    r = z.moe_plan(D[5], D[6], 5)
    assert torch.equal(z.moe_forward(D[0], *D[2:5], r, act="gelu"), y)
    assert all(torch.equal(a, b) for a, b in zip(z.moe_backward(D[1], D[0], *D[2:5], r, act="gelu"), grads))
    assert not y[gone].any() and not grads[0][gone].any() and not grads[4][gone].any()
    D[0].copy_(want[0])
    D[1].copy_(want[1])
    assert torch.equal(z.moe_forward(D[0], *D[2:5], r, act="gelu"), y)


@pytest.mark.gpu
@pytest.mark.parametrize("d,f", [(64, 72), (37, 51)])
def test_strided_operands_and_outputs(d, f):
    t, e, top = 150, 4, 2
    data = inputs(t, d, f, e, top, 5)
    D = [v.to(DEV) for v in data]
    r = z.moe_plan(D[5], D[6], e)
    y = z.moe_forward(D[0], *D[2:5], r)
    grads = z.moe_backward(D[1], D[0], *D[2:5], r)

    def spread(v, pad, value=7.0):
        """v's values in a larger tensor of `value`, rows and matrices apart, at an odd element."""
        shape = [s + p for s, p in zip(v.shape, pad)]
        big = torch.full((math.prod(shape) + 1,), value, dtype=v.dtype, device=DEV)
        view = big[1:].view(shape)[tuple(slice(0, s) for s in v.shape)]
        view.copy_(v)
        return big, view

    for pad in (1, 8):
        x, dy = spread(D[0], (0, pad))[1], spread(D[1], (0, pad))[1]
        w = [spread(v, (2, 1, pad))[1] for v in D[2:5]]
        outs = [spread(torch.full_like(v, math.nan), (0,) * (v.dim() - 2) + (1, pad)) for v in (y, *grads[:4])]
        before = [b.clone() for b, _ in outs]
        assert torch.equal(z.moe_forward(x, *w, r, out=outs[0][1]), y)
        got = z.moe_backward(dy, x, *w, r, dx=outs[1][1], dw_gate=outs[2][1], dw_up=outs[3][1], dw_down=outs[4][1])
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
        for (big, view), was in zip(outs, before):
            view.fill_(math.nan)
            assert torch.equal(big.view(torch.int16), was.view(torch.int16))  # nothing between the rows
    # one of the gate's and up's gradients given: the other takes its layout
    _, dg = spread(torch.zeros_like(grads[1]), (0, 3, 5))
    got = z.moe_backward(D[1], D[0], *D[2:5], r, dw_gate=dg)
    assert got[1] is dg and all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.gpu
def test_gradients_into_a_flat_vector():
    t, d, f, e, top = 90, 56, 40, 3, 2
    D = [v.to(DEV) for v in inputs(t, d, f, e, top, 6)]
    r = z.moe_plan(D[5], D[6], e)
    want = z.moe_backward(D[1], D[0], *D[2:5], r)
    flat = torch.full((3 * e * f * d + 11,), 3.0, dtype=torch.bfloat16, device=DEV)
    parts = [flat[5 + k * e * f * d:5 + (k + 1) * e * f * d] for k in range(3)]
    got = z.moe_backward(D[1], D[0], *D[2:5], r, dw_gate=parts[0].view(e, f, d), dw_up=parts[1].view(e, f, d),
                         dw_down=parts[2].view(e, d, f))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (flat[:5] == 3).all() and (flat[-6:] == 3).all()


@pytest.mark.gpu
def test_a_route_that_is_none_stays_in_bounds():
    """Arrays of any content: wrong sums, but no access outside the buffers."""
    t, d, f, e, top = 64, 32, 24, 4, 2
    D = [v.to(DEV) for v in inputs(t, d, f, e, top, 7)]
    g = torch.Generator().manual_seed(8)
    wild = lambda *s: torch.randint(-(1 << 31), 1 << 31, s, generator=g).to(torch.int32).to(DEV)  # noqa: E731
    good = z.moe_plan(D[5], D[6], e)
    for r in (z.Route(wild(t, top), D[6], wild(e + 1), wild(t * top), wild(t, top)),
              good._replace(order=wild(t * top)), good._replace(place=wild(t, top)), good._replace(offsets=wild(e + 1)),
              good._replace(offsets=torch.tensor([0, t * top, 0, t * top, 5], dtype=torch.int32, device=DEV))):
        y = z.moe_forward(D[0], *D[2:5], r)
        z.moe_backward(D[1], D[0], *D[2:5], r)
        z.moe_route_backward(D[6], torch.zeros((t, e), device=DEV), r)
        torch.cuda.synchronize()
        assert y.shape == (t, d)
    check(*inputs(t, d, f, e, top, 7), "silu", "after")


@pytest.mark.gpu
def test_two_streams_and_captured():
    shapes = [(300, 128, 96, 8, 2), (520, 64, 72, 5, 3)]
    sets = [[v.to(DEV) for v in inputs(*s, 9 + k)] for k, s in enumerate(shapes)]

    def step(D):
        r = z.moe_plan(D[5], D[6], D[2].shape[0])
        return (z.moe_forward(D[0], *D[2:5], r), *z.moe_backward(D[1], D[0], *D[2:5], r))

    want = [step(D) for D in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        for s, D in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(step(D))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    graph = torch.cuda.CUDAGraph()
    D = sets[0]
    with torch.cuda.graph(graph):
        kept = step(D)
    for k in range(3):
        fresh = inputs(*shapes[0], 20 + k, skew=2.0 * k)
        for a, b in zip(D, fresh):
            a.copy_(b.to(DEV))
        graph.replay()
        now = step(D)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, now))


@pytest.mark.gpu
def test_x_past_the_products_offsets():
    """x and dy of more than 4 GiB: copied by expert instead of gathered."""
    t, d, f, e = 1 << 18, 8200, 8, 2
    x = torch.empty((t, d), dtype=torch.bfloat16, device=DEV)
    dy = torch.empty_like(x)
    live = torch.cat([torch.arange(0, 40), torch.arange(t - 40, t)]).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(10)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    x[live], dy[live] = r(80, d), r(80, d)
    w = [r(e, f, d), r(e, f, d), r(e, d, f)]
    chosen = torch.full((t, 1), -1, dtype=torch.int32, device=DEV)
    chosen[live] = torch.arange(80, device=DEV, dtype=torch.int32).unsqueeze(1) % 2
    share = torch.rand((t, 1), generator=g, device=DEV)
    route = z.moe_plan(chosen, share, e)
    y, grads = z.moe_forward(x, *w, route), z.moe_backward(dy, x, *w, route)
    assert not y[100].any() and not grads[0][100].any() and not grads[4][100].any()
    c = lambda v: v.cpu()  # noqa: E731
    check(c(x[live]), c(dy[live]), *map(c, w), c(chosen[live]), c(share[live]), "silu", "far rows", y=y[live],
          grads=(grads[0][live], *grads[1:4], grads[4][live]))


def test_reference_gradients_are_differences():
    t, d, f, e, top = 6, 5, 4, 3, 2
    x, dy, wg, wu, wd, chosen, share = inputs(t, d, f, e, top, 11)
    v = [a.double() for a in (x, wg, wu, wd, share)]
    go = lambda a: ref.moe(*a[:4], chosen, a[4], kind)[0]  # noqa: E731
    g = torch.Generator().manual_seed(12)
    for kind in ("silu", "gelu"):
        _, back = ref.moe(*v[:4], chosen, v[4], kind, dy.double())
        grads = [b[0] for b in back]
        for i, name in enumerate(NAMES):
            step = torch.randn(v[i].shape, generator=g, dtype=torch.float64)
            s = 1e-5
            up, down = ([a + (s * sign * step if k == i else 0) for k, a in enumerate(v)] for sign in (1, -1))
            diff = float(((go(up) - go(down)) * dy.double()).sum()) / (2 * s)
            want = float((grads[i] * step).sum()) if name != "dweights" else float((grads[4] * step * (chosen >= 0)).sum())
            assert abs(diff - want) < 1e-7 * max(1.0, abs(want)), name
