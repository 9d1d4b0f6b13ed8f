"""Linear cross entropy where logits are large and the model is sure.

Every logit here is a multiple of 1/4 below 2^12, so fp32 holds it and every
difference of two exactly, and what is left of the loss is

  log s, s = the sum of exp(z - m) over the row, m its largest logit

with an error that does not grow with |z|: an exponential is off by 2^-22 of
itself and by the two roundings of its argument, 2 * 2^-24 (m - z), whose mean
under the row's own probabilities is at most log V + 1; about 32 additions and
10 rescalings (2^-22 each) join them.  With V = 1003 that is below 2^-17 of s,
to which come the logarithm's and the last sum's roundings of the loss
(2^-21 of it).  m's own term is exactly 1, so no loss is negative."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
from train_reference import HALF_BF16, inside, xent

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
WORDS = 40  # the words that are targets: each has a column of x of its own


def inputs(t, v, d, top, seed):
    """Logits 8 base + gap [own word] + a sum of quarters, base up to `top`."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-4, 5, (v, d), generator=g) / 4.0
    w[:, 0] = 8.0
    w[:, 8:8 + WORDS] = 0
    y = torch.randint(0, WORDS, (t,), generator=g)
    w[torch.arange(WORDS), 8 + torch.arange(WORDS)] = 1.0
    x = torch.zeros((t, d))
    x[:, 0] = torch.randint(0, top + 1, (t,), generator=g).float()
    x[:, 1:8] = torch.randint(-1, 2, (t, 7), generator=g).float()
    gap = torch.tensor([0.0, 2.0, 6.0, 12.0, 40.0])[torch.arange(t) % 5]
    x[torch.arange(t), 8 + y] = gap
    return x.to(torch.bfloat16), w.to(torch.bfloat16), y


@pytest.mark.parametrize("top", [0, 2, 10, 255])
@pytest.mark.parametrize("t", [5, 320])
def test_loss_is_as_exact_with_large_logits(t, top):
    x, w, y = inputs(t, 1003, 64, top, t + top)
    loss, row, dx, _ = z.linear_xent_grad(x.to(DEV), w.to(DEV), y.to(DEV), mean=False)
    _, want, _, _, p, _ = xent(x.double(), w.double(), y, -100, False, 1.0)
    row = row.cpu()
    assert bool((row >= 0).all()), float(row.min())
    bound = 2.0 ** -17 + 2.0 ** -21 * want
    inside(row, want, bound, "row_loss")
    inside(loss.cpu()[0], want.sum(), bound.sum() + 2.0 ** -24 * want.sum(), "loss")
    # a target's own column of dx is its entry of softmax - onehot, rounded to bf16 twice: never positive
    at = torch.arange(t)
    own = dx.cpu()[at, 8 + y]
    assert bool((own <= 0).all()), float(own.max())
    ref = p[at, y]
    inside(own, ref, 2.02 * HALF_BF16 * ref.abs() + 2.0 ** -17, "target's own entry")
