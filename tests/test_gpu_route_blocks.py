"""Routing and sorting at the sizes around which one block or several do it."""
import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def same(route, chosen, experts):
    for got, want in zip((route.offsets, route.order, route.place), ref.plan(chosen, experts)):
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("experts", [3, 512, 513, 1024])
@pytest.mark.parametrize("slots", [256, 257, 2048, 2049, 4096, 4097, 8192, 8193])
def test_the_sort_alone(slots, experts):
    g = torch.Generator().manual_seed(slots)
    chosen = torch.randint(-1, experts, (slots, 1), generator=g).to(torch.int32)
    same(z.moe_plan(chosen.to(DEV), torch.zeros(slots, 1, device=DEV), experts), chosen, experts)


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("experts,top", [(8, 2), (16, 16), (40, 7), (200, 8)])
def test_the_choice_and_the_sort(experts, top, scored):
    g = torch.Generator().manual_seed(experts)
    bias = (0.1 * torch.randn(experts, generator=g)).to(DEV) if scored else None
    for t in (1, 31, 32, 33, 63, 64, 65, 128, 129, 255, 256, 257, 511, 512, 513):
        x = torch.randn((t, experts), generator=g).to(DEV)
        r = z.moe_route(x, top, score="sigmoid", bias=bias)
        p = torch.sigmoid(x.double()) + bias.double() if scored else x
        assert torch.equal(r.experts, torch.sort(p, dim=1, descending=True, stable=True).indices[:, :top].int())
        same(r, r.experts.cpu(), experts)
