"""Routing of tokens to experts: choice, order and places against a plain
walk in 64 bits, weights and the logits' gradient against their formulas.

Bounds.  A weight is a quotient of exponentials: the exponent is a difference of
logits, each off by 2^-23 of its size (of log logistic's values too), the
exponential by 2 steps, the sum by its terms; so (8 + 4 range + terms) steps
relatively, the range of the logits that take part being below 60 here."""
import math

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z
from train_reference import HALF_BF16, HALF_F32, inside

DEV = torch.device("cuda:0")


def logits(t, experts, seed, dtype=torch.float32, masked=0.0, empty=0.0):
    g = torch.Generator().manual_seed(seed)
    x = 1.5 * torch.randn((t, experts), generator=g)
    x = x.masked_fill(torch.rand((t, experts), generator=g) < masked, -math.inf)
    x = x.masked_fill(torch.rand((t, 1), generator=g) < empty, -math.inf)
    return x.to(dtype)


def close(v, experts):
    return (8 + 4 * 60 + experts) * HALF_F32 * v.abs() + 1e-38


def check(x, top, r, score, bias, groups, top_groups, renormalise, scale, what):
    experts = x.shape[1]
    wide = x.double().cpu()
    chosen = ref.choose(wide, top, score, None if bias is None else bias.double().cpu(), groups, top_groups)
    assert torch.equal(r.experts.cpu(), chosen), what
    want = ref.weights(wide, chosen, score, renormalise, scale)
    inside(r.weights.cpu(), want, close(want, experts), f"{what} weights")
    for got, exact in zip((r.offsets, r.order, r.place), ref.plan(chosen, experts)):
        assert torch.equal(got.cpu(), exact), what
    return chosen


def check_back(x, r, chosen, score, renormalise, scale, seed, what):
    t, experts = x.shape
    top = chosen.shape[1]
    dw = torch.randn((t, top), generator=torch.Generator().manual_seed(seed))
    dw = torch.where(chosen >= 0, dw, math.nan)  # (not looked at)
    got = z.moe_route_backward(dw.to(DEV), x, r, score=score, renormalise=renormalise, scale=scale)
    assert got.dtype == x.dtype
    leaf = x.double().cpu().requires_grad_(True)
    w = ref.weights(leaf, chosen, score, renormalise, scale)
    g = torch.where(chosen >= 0, dw.double(), 0.0)
    want, = torch.autograd.grad(w, leaf, g)
    # terms of a gradient: w g, w sum(w g), and for softmax p times either
    size = (w.detach() * g).abs().sum(1, keepdim=True) + scale * g.abs().sum(1, keepdim=True) * w.detach().amax(1, keepdim=True)
    bound = close(want, experts) + close(size, experts).expand_as(want) * (1.0 if score == "sigmoid" or renormalise else 4.0)
    if x.dtype == torch.bfloat16:
        bound = bound + HALF_BF16 * want.abs()
    inside(got.cpu(), want, bound, f"{what} dlogits")
    assert not got.cpu()[x.cpu() == -math.inf].any()


CASES = [  # tokens, experts, top, groups, top groups
    (1, 1, 1, 1, 1), (1, 2, 2, 1, 1), (3, 5, 3, 1, 1), (64, 8, 2, 1, 1), (65, 8, 8, 1, 1), (7, 64, 6, 8, 3),
    (33, 60, 6, 1, 1), (40, 60, 4, 4, 2), (20, 160, 6, 8, 3), (90, 256, 8, 8, 4), (17, 1024, 32, 64, 8), (5, 1000, 7, 8, 2),
    (300, 128, 8, 1, 1), (1200, 16, 4, 1, 1), (9, 33, 32, 1, 1), (700, 64, 8, 64, 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,experts,top,groups,top_groups", CASES)
def test_choice_weights_order_and_gradient(t, experts, top, groups, top_groups, score, dtype):
    for seed, (biased, renormalise, scale) in enumerate([(False, True, 1.0), (True, False, 2.5), (True, True, 1.0)]):
        x = logits(t, experts, t + seed, dtype, masked=0.2 * seed, empty=0.1 * seed).to(DEV)
        bias = (0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(seed))).to(DEV) if biased else None
        r = z.moe_route(x, top, score=score, bias=bias, groups=groups, top_groups=top_groups, renormalise=renormalise,
                        scale=scale)
        what = f"{t}x{experts} top {top} {score} {seed}"
        chosen = check(x, top, r, score, bias, groups, top_groups, renormalise, scale, what)
        check_back(x, r, chosen, score, renormalise, scale, seed, what)


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ranks_closer_than_fp32_are_settled_in_64_bits(score, groups):
    """Biases that put neighbours within some 2^-26 of each other, either way."""
    t, experts, top = 256, 32, 4
    x = logits(t, experts, 3)
    x[:, 1::2] = x[:, 0::2] + 2.0 ** -20 * torch.randn((t, experts // 2), generator=torch.Generator().manual_seed(4))
    bias = 0.01 * torch.randn(experts, generator=torch.Generator().manual_seed(5))
    bias[1::2] = bias[0::2] + 2.0 ** -28
    x, bias = x.to(DEV), bias.to(DEV)
    r = z.moe_route(x, top, score=score, bias=bias, groups=groups, top_groups=min(2, groups))
    check(x, top, r, score, bias, groups, min(2, groups), True, 1.0, score)


@pytest.mark.gpu
@pytest.mark.parametrize("biased", [False, True])
def test_equal_ranks_go_to_the_lower_expert(biased):
    x = torch.zeros((5, 16), device=DEV)
    x[1, 7] = 1.0
    x[2, 3] = x[2, 12] = 0.5
    x[3] = -0.0
    x[4, 8:] = -math.inf
    bias = torch.zeros(16, device=DEV) if biased else None
    for score in ("softmax", "sigmoid"):
        r = z.moe_route(x, 3, score=score, bias=bias)
        assert r.experts.tolist() == [[0, 1, 2], [7, 0, 1], [3, 12, 0], [0, 1, 2], [0, 1, 2]]


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_infinities_and_nan(score, groups):
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[1.0, -math.inf, 2.0, -math.inf], [-math.inf] * 4, [low, low, low, low], [low, 1.0, -math.inf, low],
                      [-90.0, -100.0, -110.0, -math.inf], [math.nan, 1.0, 0.0, -1.0], [200.0, 0.0, 190.0, -200.0]])
    x = x.to(DEV)
    r = z.moe_route(x, 3, score=score, groups=groups, top_groups=groups)
    e, w = r.experts.cpu(), r.weights.cpu()
    assert e[0].tolist() == [2, 0, -1] and w[0, 2] == 0 and abs(float(w[0].sum()) - 1) < 1e-6
    assert e[1].tolist() == [-1, -1, -1] and not w[1].any()
    assert e[2].tolist() == [0, 1, 2]
    assert e[3, 0] == 1 and e[4].tolist() == [0, 1, 2] and e[6].tolist() == [0, 2, 1]
    if score == "softmax" or groups == 1:
        assert w[4, 0] > 0.9 and w[4, 1] > 1e-5  # far below every exponential's range, still in proportion
    assert 0 not in e[5].tolist() or groups > 1  # a NaN ranks last
    assert bool(((e >= -1) & (e < 4)).all())
    for i in (0, 1, 3, 4, 6):
        assert torch.isfinite(w[i]).all()
    # an expert with a bias of -inf is not there
    bias = torch.tensor([0.0, 0.0, -math.inf, 0.0], device=DEV)
    r = z.moe_route(torch.ones((3, 4), device=DEV), 4, score=score, bias=bias)
    assert r.experts.tolist() == [[0, 1, 3, -1]] * 3 and r.offsets.tolist() == [0, 3, 6, 6, 9]
    back = z.moe_route_backward(torch.ones((7, 3), device=DEV), x, z.moe_route(x, 3, score=score), score=score)
    assert not back[1].any() and back[0, 1] == 0 and back[0, 3] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t,experts,top", [(1, 1, 1), (3, 4, 5), (700, 3, 2), (257, 1024, 8), (5000, 60, 6), (100000, 7, 1),
                                           (40000, 256, 8)])
def test_plan_of_experts_given(t, experts, top):
    g = torch.Generator().manual_seed(t)
    chosen = torch.randint(-1, experts, (t, top), generator=g).to(torch.int32)
    chosen[t // 2:] = chosen[t // 2:].clamp(max=max(0, experts // 3))  # uneven
    chosen[::7, 0] = experts  # out of range: none
    w = torch.rand((t, top), generator=g)
    r = z.moe_plan(chosen.to(DEV), w.to(DEV), experts)
    for got, want in zip((r.offsets, r.order, r.place), ref.plan(chosen, experts)):
        assert torch.equal(got.cpu(), want)
    again = z.moe_plan(chosen.to(DEV), w.to(DEV), experts)
    assert all(torch.equal(a, b) for a, b in zip(r, again))


@pytest.mark.gpu
def test_nothing_and_outputs_given():
    x = torch.randn((40, 8), generator=torch.Generator().manual_seed(1)).to(DEV)
    want = z.moe_route(x, 2)
    out = z.Route(*(torch.full_like(v, 77) for v in want))
    assert z.moe_route(x, 2, out=out) is out and all(torch.equal(a, b) for a, b in zip(out, want))
    odd = torch.zeros((40, 11), device=DEV)[:, 2:10]
    odd.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(z.moe_route(odd, 2), want))
    dw = torch.randn((40, 2), generator=torch.Generator().manual_seed(2)).to(DEV)
    grad = z.moe_route_backward(dw, x, want)
    to = torch.full((40, 13), 5.0, device=DEV)
    assert torch.equal(z.moe_route_backward(dw, odd, want, out=to[:, 3:11]), grad)
    assert (to[:, :3] == 5).all() and (to[:, 11:] == 5).all()
    r = z.moe_route(x[:0], 2)
    assert r.offsets.tolist() == [0] * 9 and r.order.numel() == 0
    assert z.moe_route_backward(dw[:0], x[:0], r).shape == (0, 8)
    p = z.moe_plan(torch.empty((0, 3), dtype=torch.int32, device=DEV), torch.empty((0, 3), device=DEV), 4)
    assert p.offsets.tolist() == [0] * 5


@pytest.mark.gpu
def test_captured():
    t, experts, top = 600, 64, 6
    x = logits(t, experts, 1).to(DEV)
    bias = (0.05 * torch.randn(experts, generator=torch.Generator().manual_seed(2))).to(DEV)
    dw = torch.randn((t, top), generator=torch.Generator().manual_seed(3)).to(DEV)

    def step():
        r = z.moe_route(x, top, score="sigmoid", bias=bias, groups=8, top_groups=4)
        return (*r, z.moe_route_backward(dw, x, r, score="sigmoid"))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for k in range(4):
        x.copy_(logits(t, experts, 10 + k, masked=0.3 * (k % 2)))
        graph.replay()
        now = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, now))


def test_reference_gradients_are_differences():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((4, 9), generator=g, dtype=torch.float64)
    x[1, 3:] = -math.inf
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            chosen = ref.choose(x, 3, score, None, 1, 1)
            f = lambda v: ref.weights(v, chosen, score, renormalise, 1.5)  # noqa: E731
            dw = torch.randn((4, 3), generator=g, dtype=torch.float64)
            leaf = x.clone().requires_grad_(True)
            grad, = torch.autograd.grad(f(leaf), leaf, dw)
            v, s = torch.randn(x.shape, generator=g, dtype=torch.float64), 1e-5
            diff = float(((f(x + s * v) - f(x - s * v)) * dw).sum()) / (2 * s)
            assert abs(diff - float((grad * v).sum())) < 1e-8
