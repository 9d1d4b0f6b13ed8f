"""Norms with rotation of rows without a position beside weights that are no numbers, and of
rows whose squares leave fp32, against the formulas in 64 bits with the bounds of the
other tests."""
import math

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z
from train_reference import inside

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


SCALES = [1e-39, 3e-37, 1e-30, 1e-23, 1e-19, 1e-12, 1e-11, 1.0, 1e17, 2e19, 1e20, 1e25, 4e37]


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-34, 1e-24, 1e-6])
@pytest.mark.parametrize("width,rot", [(64, 48), (512, 512), (128, 0), (40, 8), (36, 20), (14, 2), (1, 0)])
def test_rows_whose_squares_leave_fp32(width, rot, eps, style):
    """Rows of every size beside each other, one with a single large element, from 2^-130 to 2^127."""
    g = torch.Generator().manual_seed(width)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    size = torch.tensor(SCALES + SCALES[::-1], dtype=torch.float64).view(-1, 1, 1)
    t = size.shape[0]
    x = (size * r(t, 3, width).clamp(-4, 4)).to(torch.bfloat16)
    x[::5, 1, 1:] *= 1e-12
    # (gradients that neither overflow nor vanish beside their row)
    dy = (size.clamp(1e-30, 1e30) ** 0.5 * r(t, 3, width)).to(torch.bfloat16)
    w = (1 + 0.3 * r(width)).to(torch.bfloat16)
    cs = ref.table(t, rot, 100.0).float() if rot else torch.zeros(t, 0, 2)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    args = (x.to(DEV), None, cs.to(DEV) if rot else None, None, w.to(DEV), None, eps, style)
    y, _ = z.qk_norm_rope(*args)
    dq, _, _, _ = z.qk_norm_rope_backward(dy.to(DEV), None, *args)
    want, dx, _, y_e, dx_e, _ = ref.rope(x.double(), dy.double(), w.double(), cs.double(), eps, style)
    # (one dimension of one element of 0, say: 0 / 0)
    live = ~want.isnan().any(2)
    big = 3.3e38  # (bf16 holds up to 3.39e38)
    held = live.unsqueeze(2) & (dx.abs() < big)
    inside(y.cpu()[live], want[live], y_e[live] + 1e-38, "y")
    inside(dq.cpu()[held], dx[held], dx_e[held] + 1e-38, "dx")
    assert y.cpu()[~live].isnan().any() or live.all()
