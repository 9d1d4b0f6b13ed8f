"""Linear cross entropy against the formulas in 64 bits.

Bounds.  A logit is off by at most D 2^-24 sum |x||w| (fp32 sums); so a row's
loss is off by twice the largest such error of the row, plus a few fp32
roundings of values of the size of the logits.  P is bf16 (2^-8 of itself),
formed from fp16 exponentials (2^-11, and 2^-25 absolutely below fp16's normal
range) whose logits carry the error above; dx and dw sum those errors times
the other factor's magnitude and round once more."""
import math

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
from train_reference import HALF_BF16, HALF_F16, HALF_F32, inside, xent

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
IGN = -100


def inputs(t, d, v, seed, ignored=0.0, std=None, lean=0.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((v, d), generator=g) * (std or 1.0 / math.sqrt(d))).to(torch.bfloat16)
    x = torch.randn((t, d), generator=g)
    y = torch.randint(0, v, (t,), generator=g)
    if lean:
        r = w[y].float()
        x = x + r * (lean * torch.rand((t, 1), generator=g) / r.square().sum(1, keepdim=True))
    if ignored:
        y = torch.where(torch.rand((t,), generator=g) < ignored, torch.full_like(y, IGN), y)
    return x.to(torch.bfloat16), w, y


def check(x, w, y, mean, scale, got, what):
    loss, row, dx, dw = got
    X, W = x.double(), w.double()
    t, d = X.shape
    v = W.shape[0]
    rl, rr, rdx, rdw, p, c = xent(X, W, y, IGN, mean, scale)
    zerr = (1.01 * d * HALF_F32 * (X.abs() @ W.abs().t())).amax(1, keepdim=True)  # of a row's logits
    big = (X @ W.t()).abs().amax(1)
    # exponentials and logarithms of the hardware: 2^-21 of values of the logits' size, and of log v
    rbound = 2 * zerr[:, 0] + 2.0 ** -21 * (big + math.log(v) + 1)
    inside(row.to(X.device), rr, rbound, f"{what} row_loss")
    keep = (y != IGN).double()
    share = c / scale
    inside(loss.to(X.device)[0], rl, (rbound * keep).sum() * share + HALF_F32 * rl.abs() * 4, f"{what} loss")
    q = torch.exp(X @ W.t() - torch.logsumexp(X @ W.t(), 1, keepdim=True)) * keep.unsqueeze(1)
    perr = HALF_BF16 * 1.01 * p.abs() + (HALF_F16 * 1.01 + 2 * rbound.unsqueeze(1)) * q + 2.0 ** -25 * keep.unsqueeze(1)
    if dx is not None:
        b = c * (perr @ W.abs() + 1.01 * v * HALF_F32 * (p.abs() @ W.abs()))
        inside(dx.to(X.device), rdx, HALF_BF16 * rdx.abs() + 1.01 * b + 1e-38, f"{what} dx")
    if dw is not None:
        b = c * (perr.t() @ X.abs() + 1.01 * t * HALF_F32 * (p.abs().t() @ X.abs()))
        inside(dw.to(X.device), rdw, HALF_BF16 * rdw.abs() + 1.01 * b + 1e-38, f"{what} dw")


SHAPES = [(1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 1000), (17, 33, 63), (64, 64, 64), (65, 40, 65), (127, 96, 129),
          (128, 128, 512), (130, 72, 777), (300, 200, 1001), (257, 256, 2048), (600, 130, 300), (33, 1000, 4099)]


@pytest.mark.parametrize("t,d,v", SHAPES)
@pytest.mark.parametrize("mean", [False, True])
def test_loss_and_gradients(t, d, v, mean):
    x, w, y = inputs(t, d, v, t * 7 + d * 3 + v, ignored=0.25 if t > 2 else 0.0)
    got = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV), mean=mean, grad_scale=3.0)
    check(x, w, y, mean, 3.0, got, f"{t}x{d}x{v}")
    loss, row = z.linear_xent_loss(x.to(DEV), w.to(DEV), y.to(DEV), mean=mean)
    assert torch.equal(loss, got[0]) and torch.equal(row, got[1])


@pytest.mark.parametrize("want_dx,want_dw", [(True, False), (False, True)])
def test_one_gradient_alone_is_the_same(want_dx, want_dw):
    x, w, y = (a.to(DEV) for a in inputs(100, 80, 300, 1, ignored=0.2))
    both = z.linear_xent_grad(x, w, y)
    one = z.linear_xent_grad(x, w, y, want_dx=want_dx, want_dw=want_dw)
    assert torch.equal(both[0], one[0]) and torch.equal(both[1], one[1])
    assert (one[2] is None) == (not want_dx) and (one[3] is None) == (not want_dw)
    assert torch.equal(both[2] if want_dx else both[3], one[2] if want_dx else one[3])


def test_sure_and_unsure_rows():
    """Rows whose target has nearly all of the probability, rows with large
    logits, rows of equal logits."""
    x, w, y = inputs(200, 64, 500, 3, lean=30.0)
    x[:20] *= 20
    x[20:30] = 0
    got = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV))
    check(x, w, y, True, 1.0, got, "sure")


def test_every_row_ignored():
    x, w, _ = inputs(70, 48, 130, 4)
    y = torch.full((70,), IGN)
    x[3] = float("nan")
    for mean in (True, False):
        loss, row, dx, dw = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV), mean=mean)
        assert float(loss) == 0 and not bool(row.any()) and not bool(dx.any()) and not bool(dw.any())


def test_what_ignored_rows_hold_does_not_matter():
    x, w, y = inputs(150, 64, 200, 5, ignored=0.3)
    rows = (y == IGN).nonzero()[:, 0]
    clean = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV))
    for k, v in enumerate((float("nan"), float("inf"), float("-inf"), 3e38)):
        x[rows[k::4]] = v
    got = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV))
    for a, b in zip(clean, got):
        assert torch.equal(a, b)
    loss, row = z.linear_xent_loss(x.to(DEV), w.to(DEV), y.to(DEV))
    assert torch.equal(loss, got[0]) and torch.equal(row, got[1])


def test_ignore_index_may_be_a_class():
    x, w, y = inputs(90, 32, 40, 6)
    got = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV), ignore_index=7)
    y2 = torch.where(y == 7, torch.full_like(y, IGN), y)
    check(x, w, y2, True, 1.0, got, "class 7 ignored")


@pytest.mark.parametrize("bad", [-1, 200, 1 << 40, -(1 << 62)])
def test_target_outside_the_vocabulary_is_nan(bad):
    x, w, y = inputs(70, 32, 200, 7)
    y[5] = bad
    loss, row, dx, dw = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV))
    assert bool(torch.isnan(loss).all()) and bool(torch.isnan(row[5])) and bool(torch.isnan(dx[5]).all())
    assert bool(torch.isnan(dw).all())
    others = [k for k in range(70) if k != 5]
    assert bool(torch.isfinite(row[others]).all()) and bool(torch.isfinite(dx[others].float()).all())


def test_infinite_logits():
    """A vocabulary row that makes some logits -inf has no probability there;
    one that makes them +inf makes its rows NaN, and no other."""
    x, w, y = inputs(66, 16, 90, 8)
    x[:, 0] = torch.where(torch.arange(66) % 2 == 0, 1.0, 2.0).to(torch.bfloat16)
    w[:, 0] = 0
    y[:] = 3
    w[70, 0] = float("-inf")
    loss, row, dx, _ = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV), want_dw=False, want_dx=False)
    X, W = x.double(), w.double()
    W[70, :] = 0
    zz = X @ W.t()
    zz[:, 70] = -math.inf
    want = torch.logsumexp(zz, 1) - zz[:, 3]
    inside(row.cpu(), want, torch.full_like(want, 1e-5), "row_loss with -inf")
    x[::2, 0] = 0
    w[70, 0] = float("inf")
    row = z.linear_xent_loss(x.to(DEV), w.to(DEV), y.to(DEV))[1].cpu()
    assert bool(torch.isnan(row).all())  # 0 * inf, and inf - inf


def test_strided_and_unaligned_operands_and_flat_gradient():
    X = torch.randn((120, 100), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    W = (torch.randn((260, 90), generator=torch.Generator().manual_seed(2)) / 8).to(torch.bfloat16)
    y = torch.randint(0, 250, (60,), generator=torch.Generator().manual_seed(3))
    x, w = X[::2, 3:67], W[5:255, 11:75]
    xd, wd = X.to(DEV)[::2, 3:67], W.to(DEV)[5:255, 11:75]
    flat = torch.full((250 * 64 + 9,), 5.0, dtype=torch.bfloat16, device=DEV)
    dw = flat[5:5 + 250 * 64].view(250, 64)
    dxb = torch.full((61, 70), 5.0, dtype=torch.bfloat16, device=DEV)
    got = z.linear_xent_grad(xd, wd, y.to(DEV), dw=dw, dx=dxb[:60, 1:65])
    check(x, w, y, True, 1.0, got, "views")
    assert bool((flat[:5] == 5).all() and (flat[5 + 250 * 64:] == 5).all())
    assert bool((dxb[60] == 5).all() and (dxb[:, 0] == 5).all() and (dxb[:, 65:] == 5).all())


def test_no_rows():
    w = torch.ones((50, 24), dtype=torch.bfloat16, device=DEV)
    x = torch.empty((0, 24), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((0,), dtype=torch.int64, device=DEV)
    loss, row, dx, dw = z.linear_xent_grad(x, w, y)
    assert float(loss) == 0 and row.numel() == 0 and tuple(dx.shape) == (0, 24) and not bool(dw.any())


def test_pieces_equal_one_piece():
    """More rows than one piece of exponentials holds: the pieces' own calls
    give the same within the roundings of another order of summation (how a
    product is divided depends on its sizes)."""
    t, d, v = 20_000, 64, 131_072
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn((t, d), generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn((v, d), generator=g, device=DEV) / 8).to(torch.bfloat16)
    y = torch.randint(0, v, (t,), generator=g, device=DEV)
    loss, row, dx, dw = z.linear_xent_grad(x, w, y, mean=False)
    parts = [z.linear_xent_grad(x[a:a + 5000], w, y[a:a + 5000], mean=False) for a in range(0, t, 5000)]
    for k, p in enumerate(parts):
        rows = slice(5000 * k, 5000 * (k + 1))
        size = (x[rows].float().abs() @ w.float().abs().t()).amax(1).double()  # of a row's logits
        order = 4 * 1.01 * d * HALF_F32 * size + 2.0 ** -20 * (size + math.log(v) + 1)
        inside(row[rows], p[1].double(), order, f"row_loss of piece {k}")
        terms = torch.softmax(x[rows].float() @ w.float().t(), 1) @ w.float().abs() + w[y[rows]].float().abs()
        order = 2 * 1.01 * v * HALF_F32 * terms.double()
        bound = HALF_BF16 * (dx[rows].double().abs() + p[2].double().abs()) + order
        inside(dx[rows], p[2].double(), bound, f"dx of piece {k}")
    total = sum(p[3].double() for p in parts)
    size = sum(p[3].double().abs() for p in parts)
    assert bool(((dw.double() - total).abs() <= HALF_BF16 * (total.abs() + 1.01 * size) + 1e-3 * size).all())


def test_gradient_against_differences():
    """dx and dw against central differences of the 64-bit loss."""
    x, w, y = inputs(12, 16, 30, 11, ignored=0.2)
    _, _, dx, dw = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV))
    X, W = x.double(), w.double()
    f = lambda a, b: xent(a, b, y, IGN, True, 1.0)[0]  # noqa: E731
    g = torch.Generator().manual_seed(12)
    for _ in range(10):
        u, v = torch.randn(X.shape, generator=g).double(), torch.randn(W.shape, generator=g).double()
        h = 1e-5
        num = (f(X + h * u, W + h * v) - f(X - h * u, W - h * v)) / (2 * h)
        ana = (dx.cpu().double() * u).sum() + (dw.cpu().double() * v).sum()
        size = (dx.cpu().double() * u).abs().sum() + (dw.cpu().double() * v).abs().sum()
        # two bf16 roundings of every term (P, and the gradient), and the fp16 one
        assert abs(float(num - ana)) <= 4 * HALF_BF16 * float(size) + 1e-8


def test_another_stream_and_repeats_are_equal():
    x, w, y = (a.to(DEV) for a in inputs(700, 128, 3000, 13, ignored=0.1))
    want = z.linear_xent_grad(x, w, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = z.linear_xent_grad(x, w, y, stream=s)
        s.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_captured_in_a_graph():
    x, w, y = (a.to(DEV) for a in inputs(200, 64, 900, 14, ignored=0.1))
    outs = [torch.empty(1, device=DEV), torch.empty(200, device=DEV), torch.empty_like(x), torch.empty_like(w)]
    call = lambda: z.linear_xent_grad(x, w, y, loss=outs[0], row_loss=outs[1], dx=outs[2], dw=outs[3])  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        x2, w2, y2 = inputs(200, 64, 900, 20 + k, ignored=0.1 * k)
        x.copy_(x2.to(DEV))
        w.copy_(w2.to(DEV))
        y.copy_(y2.to(DEV))
        want = [a.clone() for a in z.linear_xent_grad(x, w, y)]
        for o in outs:
            o.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
