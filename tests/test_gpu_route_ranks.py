"""Ranks of experts that lie within fp32's error of each other although made of
unequal parts, against a 64-bit sort.  Inputs come from a seed; each test first
shows that 64 bits settle them: no two ranks that matter are within 2^-48 of the
larger."""
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
