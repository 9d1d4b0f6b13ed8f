"""Ranges of experts with NaN logits: behind every number, before experts that are
not there."""
import math

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
NAN, NONE = math.nan, -math.inf


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2, 4, 5, 16])
def test_a_range_of_nan_is_there(score, size):
    """... and comes before one with no expert, wherever either lies."""
    for front in (0, 1, 2):
        x = torch.full((3, 3 * size), NONE)
        x[:, front * size:(front + 1) * size] = NAN
        r = z.moe_route(x.to(DEV), 2, score=score, groups=3, top_groups=1)
        assert r.experts.tolist() == [[front * size, front * size + 1]] * 3
        assert r.offsets.tolist()[-1] == 6


@pytest.mark.parametrize("experts,groups,top_groups,top", [(8, 4, 1, 2), (8, 4, 3, 6), (15, 5, 2, 4), (60, 4, 2, 8),
                                                           (256, 8, 3, 8), (64, 32, 5, 8)])
def test_nan_and_experts_that_are_not_there(experts, groups, top_groups, top):
    g = torch.Generator().manual_seed(experts)
    t = 200
    x = 1.5 * torch.randn((t, experts), generator=g)
    # whole ranges of either, and single experts
    kind = torch.rand((t, groups, 1), generator=g).expand(t, groups, experts // groups).reshape(t, experts)
    one = torch.rand((t, experts), generator=g)
    x = x.masked_fill((kind < 0.4) | (one < 0.1), NAN).masked_fill(((kind >= 0.4) & (kind < 0.8)) | (one > 0.9), NONE)
    bias = (0.1 * torch.randn(experts, generator=g)).to(DEV)
    for b in (None, bias):
        r = z.moe_route(x.to(DEV), top, score="sigmoid", bias=b, groups=groups, top_groups=top_groups)
        want = ref.choose(x.double(), top, "sigmoid", None if b is None else b.double().cpu(), groups, top_groups)
        assert torch.equal(r.experts.cpu(), want)
        for got, exact in zip((r.offsets, r.order, r.place), ref.plan(want, experts)):
            assert torch.equal(got.cpu(), exact)
