"""Norms with rotation of rows without a position beside weights that are no numbers."""
import math

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("width,rot", [(64, 48), (40, 8), (36, 20), (14, 2)])
def test_rows_without_a_position_are_zero_whatever_the_weights(width, rot):
    t, heads = 23, 3
    g = torch.Generator().manual_seed(width)
    q, dy = (torch.randn((t, heads, width), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    w = torch.ones(width, dtype=torch.bfloat16)
    w[0], w[width // 2], w[-1] = math.nan, math.inf, -math.inf
    position = torch.arange(t)
    gone = torch.arange(t) % 4 == 1
    position[gone] = -1
    cs = z.rope_table(t, rot)
    args = (q, None, cs, position.to(DEV), w.to(DEV))
    y, _ = z.qk_norm_rope(*args)
    dq, _, dw, _ = z.qk_norm_rope_backward(dy, None, *args)
    assert not y.cpu()[gone].any() and not dq.cpu()[gone].any()
    assert y.cpu()[~gone].isnan().any(2).all() and dq.cpu()[~gone].isnan().any(2).all()
    assert torch.isfinite(dw).all()  # (they have no part in it)
