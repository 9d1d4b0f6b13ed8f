"""Norms and rotation of queries and keys against their formulas in 64 bits,
within bounds that count the roundings (layer_reference)."""
import math

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z
from train_reference import inside

DEV = torch.device("cuda:0")
EPS = 1e-6


def inputs(t, hq, hk, width, seed, weights=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    mixed = r(t, hq + 2 * hk, width).to(torch.bfloat16)
    w = [(1 + 0.3 * r(width)).to(torch.bfloat16) if weights else None for _ in range(2)]
    return mixed, r(t, hq, width).to(torch.bfloat16), r(t, hk, width).to(torch.bfloat16), w


def dev(v):
    return None if v is None else v.to(DEV)


def wide(v):
    return None if v is None else v.double()


def check(got, x, dy, w, cs, style, what, eps=EPS, live=None):
    """got: (y, dx, dw) of one side; rows that are not live are zero."""
    y, dx, dw = got
    live = torch.ones(x.shape[0], dtype=torch.bool) if live is None else live
    ry, rdx, rdw, ey, edx, edw = ref.rope(x[live].double(), dy[live].double(), wide(w), cs[live].double(), eps, style)
    for name, v, r, e in (("y", y, ry, ey), ("dx", dx, rdx, edx)):
        inside(v.cpu()[live], r, e + 1e-38, f"{what} {name}")
        assert not v.cpu()[~live].any()
    if w is not None:
        inside(dw.cpu(), rdw, edw + 1e-38, f"{what} dw")


SIZES = [  # tokens, heads, key heads, width, turned
    (1, 1, 1, 2, 2), (1, 1, 1, 1, 0), (3, 2, 1, 7, 4), (5, 12, 12, 64, 64), (17, 7, 1, 80, 48), (33, 4, 2, 128, 128),
    (2, 3, 3, 100, 100), (9, 5, 2, 96, 32), (40, 32, 8, 128, 64), (11, 2, 2, 256, 256), (6, 1, 1, 512, 512),
    (7, 3, 1, 511, 510), (4, 2, 2, 36, 20), (8, 1, 5, 24, 22), (300, 3, 2, 48, 48), (2050, 2, 1, 64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("t,hq,hk,width,rot", SIZES)
def test_forward_and_backward(t, hq, hk, width, rot, style):
    mixed, dyq, dyk, (wq, wk) = inputs(t, hq, hk, width, t + width)
    q, k = mixed[:, :hq], mixed[:, hq:hq + hk]
    cs = ref.table(t + 3, rot, 10000.0).float() if rot else None
    position = torch.randint(0, t + 3, (t,), generator=torch.Generator().manual_seed(t))
    m = mixed.to(DEV)
    args = (m[:, :hq], m[:, hq:hq + hk], dev(cs), dev(position), dev(wq), dev(wk), EPS, style)
    yq, yk = z.qk_norm_rope(*args)
    dq, dk, dwq, dwk = z.qk_norm_rope_backward(dev(dyq), dev(dyk), *args)
    at = cs[position] if rot else torch.zeros(t, 0, 2)
    what = f"{t}x({hq}+{hk})x{width}/{rot} {style}"
    check((yq, dq, dwq), q, dyq, wq, at, style, what + " q")
    check((yk, dk, dwk), k, dyk, wk, at, style, what + " k")


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("style", ["half", "pairs"])
def test_rows_without_a_position_take_no_part(style, weights):
    t, hq, hk, width, rot = 37, 3, 2, 64, 48
    mixed, dyq, dyk, (wq, wk) = inputs(t, hq, hk, width, 5, weights)
    position = torch.arange(t)
    gone = torch.arange(t) % 5 == 2
    position[gone] = -1
    mixed[gone], dyq[gone], dyk[gone] = math.nan, math.inf, math.nan
    cs = ref.table(t, rot, 500.0).float()
    m = mixed.to(DEV)
    args = (m[:, :hq], m[:, hq:hq + hk], dev(cs), dev(position), dev(wq), dev(wk), EPS, style)
    yq, yk = z.qk_norm_rope(*args)
    dq, dk, dwq, dwk = z.qk_norm_rope_backward(dev(dyq), dev(dyk), *args)
    at = cs[position.clamp(min=0)]
    check((yq, dq, dwq), mixed[:, :hq], dyq, wq, at, style, "q", live=~gone)
    check((yk, dk, dwk), mixed[:, hq:hq + hk], dyk, wk, at, style, "k", live=~gone)
    assert weights or (dwq is None and dwk is None)


@pytest.mark.gpu
def test_positions_past_the_table_are_nan_alone():
    t, width = 9, 32
    mixed, dyq, dyk, (wq, wk) = inputs(t, 2, 1, width, 6)
    cs = ref.table(t, width, 100.0).float()
    position = torch.arange(t)
    args = lambda p: (dev(mixed[:, :2]), dev(mixed[:, 2:3]), dev(cs), dev(p), None, None)  # noqa: E731
    want, _ = z.qk_norm_rope(*args(position))
    wrong = position.clone()
    wrong[4], wrong[7] = t, 1 << 40
    got, _ = z.qk_norm_rope(*args(wrong))
    bad = torch.tensor([i in (4, 7) for i in range(t)], device=DEV)
    assert got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])
    dq, _, _, _ = z.qk_norm_rope_backward(dev(dyq), dev(dyk), *args(wrong))
    full, _, _, _ = z.qk_norm_rope_backward(dev(dyq), dev(dyk), *args(position))
    assert dq[bad].isnan().all() and torch.equal(dq[~bad], full[~bad])


@pytest.mark.gpu
def test_layouts_outputs_and_queries_alone():
    """Heads of tokens, tokens of heads, unaligned views and outputs in place of
    the inputs all give the same."""
    t, hq, hk, width = 50, 4, 2, 64
    mixed, dyq, dyk, (wq, wk) = inputs(t, hq, hk, width, 7)
    cs = dev(ref.table(t, width, 10000.0).float())
    q, k = dev(mixed[:, :hq].contiguous()), dev(mixed[:, hq:hq + hk].contiguous())
    rest = (cs, None, dev(wq), dev(wk))
    want = z.qk_norm_rope(q, k, *rest)
    grads = z.qk_norm_rope_backward(dev(dyq), dev(dyk), q, k, *rest)
    # head by head
    hm = lambda v: v.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    out = hm(torch.empty_like(q))
    yq, yk = z.qk_norm_rope(hm(q), hm(k), *rest, out_q=out)
    assert yq is out and torch.equal(yq, want[0]) and torch.equal(yk, want[1])
    got = z.qk_norm_rope_backward(hm(dev(dyq)), hm(dev(dyk)), hm(q), hm(k), *rest, dq=hm(torch.empty_like(q)))
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    # views at any element
    flat = torch.zeros(t * (hq * width + 3) + 1, dtype=torch.bfloat16, device=DEV)
    odd = flat[1:].as_strided((t, hq, width), (hq * width + 3, width, 1))
    odd.copy_(q)
    to = torch.full_like(flat, 7.0)
    yo, none = z.qk_norm_rope(odd, None, cs, None, dev(wq), out_q=to[1:].as_strided(odd.shape, odd.stride()))
    assert none is None and torch.equal(yo, want[0])
    left = to[1:][:t * (hq * width + 3)].view(t, -1)[:, hq * width:]
    assert (left == 7.0).all() and to[0] == 7.0  # what lies between the rows
    dq, dk, dwq, dwk = z.qk_norm_rope_backward(dev(dyq), None, odd, None, cs, None, dev(wq))
    assert dk is None and dwk is None and torch.equal(dq, grads[0]) and torch.equal(dwq, grads[2])
    # in place, of the inputs and of the gradients
    q2, k2 = q.clone(), k.clone()
    z.qk_norm_rope(q2, k2, *rest, out_q=q2, out_k=k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    g2, h2 = dev(dyq), dev(dyk)
    z.qk_norm_rope_backward(g2, h2, q, k, *rest, dq=g2, dk=h2)
    assert torch.equal(g2, grads[0]) and torch.equal(h2, grads[1])
    # a broadcast input is read as it lies
    one = q[:1].expand(t, hq, width)
    yb, _ = z.qk_norm_rope(one, None, cs, torch.zeros(t, dtype=torch.int64, device=DEV), dev(wq))
    assert torch.equal(yb, want[0][:1].expand_as(yb))


@pytest.mark.gpu
def test_odd_values():
    """Zero rows, the smallest and largest values, infinities."""
    width = 64
    x = torch.zeros(6, 1, width, dtype=torch.bfloat16)
    x[1, 0, 3] = 1.0
    x[2] = 1e-20
    x[3] = 1e18
    x[4, 0, 0] = math.inf
    x[5] = -2.0 ** -126
    cs = ref.table(6, width, 10.0).float()
    y, _ = z.qk_norm_rope(dev(x), None, dev(cs))
    want, *_, e = ref.rope(x.double(), None, None, cs.double(), EPS, "half")[:4]
    live = torch.tensor([0, 1, 2, 3, 5])
    inside(y.cpu()[live], want[live], e[live] + 1e-38, "y")
    assert y[4].isnan().any() and not y[0].any()
    # no eps: a zero row is 0 / 0
    y0, _ = z.qk_norm_rope(dev(x[:1]), None, None, eps=0.0)
    assert y0.isnan().all()


@pytest.mark.gpu
def test_many_rows_sums_of_dw():
    """dw over far more rows than blocks, and the same on every run."""
    t, hq, hk, width = 20000, 5, 1, 128
    g = torch.Generator(device=DEV).manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, k, dyq, dyk, w = r(t, hq, width), r(t, hk, width), r(t, hq, width), r(t, hk, width), r(width)
    cs = z.rope_table(t, width)
    got = z.qk_norm_rope_backward(dyq, dyk, q, k, cs, None, w, w)
    again = z.qk_norm_rope_backward(dyq, dyk, q, k, cs, None, w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for x, dy, dw in ((q, dyq, got[2]), (k, dyk, got[3])):
        *_, want, _, _, e = ref.rope(x.double().cpu(), dy.double().cpu(), w.double().cpu(), cs.double().cpu(), EPS, "half")
        inside(dw.cpu(), want, e, "dw")


@pytest.mark.gpu
def test_rows_past_32_bits():
    """Elements that lie more than 2^32 bytes apart."""
    t, width, gap = 5, 64, 1 << 30
    flat = torch.zeros(4 * gap + width * 2, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((t, 2, width), (gap, width, 1))
    src = torch.randn((t, 2, width), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    x.copy_(src)
    cs = z.rope_table(t, width)
    want, _ = z.qk_norm_rope(dev(src), None, cs)
    got, _ = z.qk_norm_rope(x, None, cs, out_q=x)
    assert torch.equal(got, want)
    del flat, x, got


@pytest.mark.gpu
@pytest.mark.parametrize("positions,rot,base", [(1, 2, 10000.0), (70000, 128, 10000.0), (33, 30, 5e5), (1 << 20, 4, 1.5)])
def test_table(positions, rot, base):
    got = z.rope_table(positions, rot, base)
    want = ref.table(positions, rot, base)
    # the angle in 64 bits: at 2^20 still good to 2^-32; then one rounding to fp32
    assert float((got.cpu().double() - want).abs().max()) <= 2.0 ** -25 + 2.0 ** -30


def test_gradients_are_the_formulas_differences():
    """The 64-bit reference's gradients against central differences."""
    g = torch.Generator().manual_seed(10)
    t, h, width, rot = 3, 2, 10, 6
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, dy, w, cs = r(t, h, width), r(t, h, width), r(width), ref.table(t, rot, 7.0)
    for style in ("half", "pairs"):
        f = lambda a, b: float((ref.rope(a, None, b, cs, 0.1, style)[0] * dy).sum())  # noqa: E731
        _, dx, dw, *_ = ref.rope(x, dy, w, cs, 0.1, style)
        for _ in range(5):
            vx, vw, s = r(t, h, width), r(width), 1e-5
            diff = (f(x + s * vx, w + s * vw) - f(x - s * vx, w - s * vw)) / (2 * s)
            # the third derivative's share, some s^2 times the values' size
            assert abs(diff - float((dx * vx).sum() + (dw * vw).sum())) < 1e-7


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    t, hq, hk, width = 64, 4, 2, 128
    mixed, dyq, dyk, (wq, wk) = inputs(t, hq, hk, width, 11)
    m, cs = mixed.to(DEV), z.rope_table(t, width)
    gq, gk, w1, w2 = dev(dyq), dev(dyk), dev(wq), dev(wk)
    args = (m[:, :hq], m[:, hq:hq + hk], cs, None, w1, w2)

    def step():
        return (*z.qk_norm_rope(*args), *z.qk_norm_rope_backward(gq, gk, *args))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for k in range(3):
        fresh = torch.randn((t, hq + 2 * hk, width), generator=torch.Generator().manual_seed(k)).to(torch.bfloat16)
        m.copy_(fresh.to(DEV))
        graph.replay()
        now = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, now))
