"""The example runs the gradient operators and the optimizers together: its
gradients agree with torch's through the same model in float32, and it learns."""
import os
import sys

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z  # noqa: F401
from train_reference import act

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_gated_lm as ex  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_gradients_agree_with_float32_torch():
    m = ex.Model(300, 64, 96, 2, DEV, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    tokens = torch.randint(0, 300, (512,), generator=g, device=DEV)
    targets = torch.randint(0, 300, (512,), generator=g, device=DEV)
    targets[::5] = -100
    loss = ex.forward_backward(m, tokens, targets)
    w = {n: v.float().requires_grad_() for n, v in m.weight.items()}
    rms = lambda x: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    x = w["embed"][tokens]
    for k in range(2):
        n = rms(x)
        x = x + (act(n @ w[f"gate{k}"].t(), "silu")[0] * (n @ w[f"up{k}"].t())) @ w[f"down{k}"].t()
    want = torch.nn.functional.cross_entropy(rms(x) @ w["embed"].t(), targets, ignore_index=-100)
    want.backward()
    # bf16 activations: 2^-8 each, a dozen in a row
    assert abs(float(loss) - float(want.detach())) <= 12 * 2.0 ** -8 * float(want.detach())
    for n, v in w.items():
        off = float((m.grad[n].float() - v.grad).norm() / v.grad.norm())
        print(f"{n}: gradient off by {off:.4f}", flush=True)
        # a block's values pass three 8-bit checkpoints (2^-4 at most each, half of that in the mean square
        # at most) and the roundings above
        assert off <= 3 * 2.0 ** -5 + 12 * 2.0 ** -8


def test_the_example_learns():
    losses = ex.train(steps=40, tokens=2048, vocab=1009, width=128, ffn=352)
    print(losses[0], losses[-1], flush=True)
    assert losses[-1] < 0.25 * losses[0]
