"""The gated block far from zero: at g = +-2^64 and beyond the activation is g
or 0 and its derivative 1 or 0, in the forward and in the backward, with g
computed again and from its checkpoint.

x is (+-4 or +-3, 1/2), w_gate (+-2^k, 0), w_up (0, 1), dh 1: every product of
g, u, h and dh is exact, and a gradient sums at most four of them and is
rounded twice, to bf16."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
from train_reference import HALF_BF16, act, inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("k", [2, 20, 40, 62, 64, 100, 120])
@pytest.mark.parametrize("kept", [False, True])
def test_backward_of_large_finite_values(kind, k, kept):
    x = torch.tensor([[4.0, 0.5], [-4.0, 0.5], [3.0, 0.5], [-3.0, 0.5]])
    wg = torch.tensor([[2.0 ** k, 0.0], [-(2.0 ** k), 0.0]])
    wu = torch.tensor([[0.0, 1.0], [0.0, 1.0]])
    dh = torch.ones((4, 2))
    xd, gd, ud, dhd = (a.to(torch.bfloat16).to(DEV) for a in (x, wg, wu, dh))
    h, c = z.glu_forward(xd, gd, ud, act=kind, checkpoint=True)
    X, G, U = x.double(), wg.double(), wu.double()
    g, u = X @ G.t(), X @ U.t()
    got = z.glu_backward(dhd, xd, gd, ud, act=kind, checkpoint=c if kept else None)
    a, da = act(g, kind)
    # (at 8 2^k and more both activations are g or 0 to every bit of bf16 but at k = 2, where silu(-12)
    # and gelu's tail are small beside the sums' largest terms)
    small = 2.0 ** -13
    inside(h.cpu(), a * u, HALF_BF16 * (a * u).abs() + small, "h")
    dg, du = u * da, a
    for what, t, ref, terms in (("dx", got[0], dg @ G + du @ U, dg.abs() @ G.abs() + du.abs() @ U.abs()),
                                ("dw_gate", got[1], dg.t() @ X, dg.abs().t() @ X.abs()),
                                ("dw_up", got[2], du.t() @ X, du.abs().t() @ X.abs())):
        inside(t.cpu(), ref, 2.02 * HALF_BF16 * terms + small * 2.0 ** (k if what == "dx" else 2), what)
