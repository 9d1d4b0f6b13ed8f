"""Ranks of experts that lie within fp32's error of each other although made of
unequal parts, against a 64-bit sort.  Inputs come from a seed; each test first
shows that 64 bits settle them: no two ranks that matter are within 2^-48 of the
larger."""
import math

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

DEV = torch.device("cuda:0")
T = 4096


def keys(x, bias, score):
    wide = x.double()
    p = torch.sigmoid(wide) if score == "sigmoid" else torch.softmax(wide, 1)
    return p + bias.double()


def sort_exactly(x, bias, score, top):
    """The `top` best experts, and whether 64 bits settle them."""
    key = keys(x, bias, score)
    value, order = torch.sort(key, dim=1, descending=True, stable=True)
    gap = value[:, :top] - value[:, 1:top + 1]
    return order[:, :top].int(), bool((gap > 2.0 ** -48 * value[:, :top].abs()).all())


def check(x, bias, score, top, groups=1, top_groups=1):
    want, settled = sort_exactly(x, bias, score, top)
    assert settled
    r = z.moe_route(x.to(DEV), top, score=score, bias=bias.to(DEV), groups=groups, top_groups=top_groups)
    wrong = (r.experts.cpu() != want).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {len(x)} tokens, first {int(wrong.nonzero()[0])}"


def unequal_parts(score, experts, seed):
    """Experts 0 .. 5 of a score of some 6e-6 and a bias of some 0.01, 1.5e-8 apart, and the
    last but one of a score near 0.75 whose bias takes most of it away: its fp32
    rank is off by some 2^-25, theirs by 1e-9."""
    g = torch.Generator().manual_seed(seed)
    x = torch.full((T, experts), -40.0)
    x[:, :6] = -12.0
    bias = torch.full((experts,), -3.0)
    bias[:6] = 0.01 - 1.5e-8 * torch.arange(6, dtype=torch.float64)
    bias[-2] = -0.7445300221443176
    # (their own ranks vary by 2^-24 from token to token, the other's lies 3e-8 above at most)
    x[:, :6] += (0.02 * torch.rand((T, 1), generator=g) - 0.01)
    if score == "softmax":
        x[:, :6] += 0.3
    small = x[:, 0].double()
    own = torch.sigmoid(small) if score == "sigmoid" else 0.75 * small.exp()
    p = bias[0].double() + own + 3e-8 * torch.rand(T, generator=g, dtype=torch.float64) - bias[-2].double()
    if score == "sigmoid":
        x[:, -2] = torch.log(p / (1 - p)).float()
    else:
        x[:, -2] = 0.0
        x[:, -1] = torch.log(1 / p - 1 - 6 * small.exp()).float()
    return x, bias


@pytest.mark.gpu
@pytest.mark.parametrize("top", [1, 3])
@pytest.mark.parametrize("experts", [8, 33, 128, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_left_out_may_be_further_off_than_the_first_left_out(score, experts, top):
    x, bias = unequal_parts(score, experts, experts + top)
    check(x, bias, score, top)


def far_below(experts, distance, seed):
    """Two experts whose logits lie `distance` and some 3 more below the largest, with biases
    of their scores' size: of the first, 0.1 is left, to which the second's 0.05 and its bias
    add up within 2e-6 of the first's score.  Of the others none comes near."""
    g = torch.Generator().manual_seed(seed)
    uniform = lambda lo, hi: lo + (hi - lo) * torch.rand(T, generator=g, dtype=torch.float64)  # noqa: E731
    x = torch.full((T, experts), -200.0)
    x[:, 0] = uniform(6.0, 8.0).float()
    top = x[:, 0].double()
    at = math.exp(-distance)  # (the largest has all of the sum but some 1e-3 at most)
    bias = torch.full((experts,), -1.0)
    bias[0], bias[1], bias[2] = -1.5, -0.9 * at, 0.05 * at
    x[:, 1] = (top - distance + uniform(-2e-3, 2e-3)).float()
    first = (x[:, 1].double() - top).exp()
    for _ in range(3):  # (the second's score is a part of the sum)
        total = 1 + first + torch.where(x[:, 2] > -200.0, (x[:, 2].double() - top).exp(), 0.0)
        second = first / total + bias[1].double() - bias[2].double() + 2e-6 * at * uniform(-1, 1)
        x[:, 2] = (top + (second * total).log()).float()
    return x, bias


@pytest.mark.gpu
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("distance", [7, 20, 40, 60])
@pytest.mark.parametrize("experts", [8, 60, 256])
def test_softmax_scores_far_below_the_largest_are_off_by_more(experts, distance, top):
    check(*far_below(experts, distance, distance + experts), "softmax", top)


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("experts", [8, 200])
def test_scores_below_fp32_keep_their_order(experts, groups):
    """Logistic scores that fp32 does not hold, down to e^-700."""
    g = torch.Generator().manual_seed(experts)
    x = -90.0 - 20.0 * torch.rand((T, experts), generator=g)
    x[:, ::3] *= 5.0
    for top in (1, 4):
        check(x, torch.zeros(experts), "sigmoid", top, groups, groups)
