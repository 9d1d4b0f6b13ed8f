"""A small language model trained with every part of the library on one GPU.

    python examples/train_gated_lm.py [--steps 60] [--tokens 4096]

The model is a tied embedding [V, D] and gated feed-forward blocks with a
pre-norm each; it learns which token follows which.  One step:

  forward   z.glu_forward keeps g and u of each block as 8-bit checkpoints, and
            z.act8_pack its input: nothing else of a block is kept
  loss      z.linear_xent_grad: the loss and both gradients of the head, the
            embedding's written straight into the flat gradient vector; no
            [tokens, V] logits are left behind
  backward  z.glu_backward from the checkpoints, which also forms h again for
            the down projection's weight gradient
  step      z.grad_sq_norm, z.grad_clip_stats and z.adamw_shard_step_clipped
            on the embedding, z.muon_step_groups on the blocks' matrices

The norms, the residual and the down projection are plain torch operations.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sharded_optimizer_step_adamw_amd as z  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """Weights (bf16), their gradients as views of one flat bf16 vector, and
    the fp32 state of the optimizers."""

    def __init__(self, vocab, width, ffn, blocks, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        shapes = [("embed", vocab, width)]
        for k in range(blocks):
            shapes += [(f"gate{k}", ffn, width), (f"up{k}", ffn, width), (f"down{k}", width, ffn)]
        total = sum(r * c for _, r, c in shapes)
        self.blocks, self.shapes = blocks, {n: (r, c) for n, r, c in shapes}
        self.flat_grad = torch.zeros(total, dtype=BF16, device=device)
        self.master, self.weight, self.grad = {}, {}, {}
        at = 0
        for name, r, c in shapes:
            self.master[name] = torch.randn((r, c), generator=g, device=device) * (0.02 if name == "embed" else c ** -0.5)
            self.weight[name] = self.master[name].to(BF16)
            self.grad[name] = self.flat_grad[at:at + r * c].view(r, c)
            at += r * c
        self.avg = [torch.zeros(vocab * width, device=device) for _ in range(2)]
        self.momentum = {n: torch.zeros_like(m) for n, m in self.master.items() if n != "embed"}


def norm(x):
    """x / rms(x) in bf16, and the fp32 1 / rms."""
    r = torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)
    return (x.float() * r).to(BF16), r


def norm_backward(dn, x, r):
    n = x.float() * r
    d = dn.float()
    return r * (d - n * (d * n).mean(1, keepdim=True))


def forward_backward(m, tokens, targets):
    """The loss (device scalar); every gradient is left in m.flat_grad."""
    w = m.weight
    x = w["embed"][tokens].float()
    kept = []
    for k in range(m.blocks):
        n, r = norm(x)
        h, gu = z.glu_forward(n, w[f"gate{k}"], w[f"up{k}"], checkpoint=True)
        kept.append((x, r, z.act8_pack(n), gu))
        x = x + (h @ w[f"down{k}"].t()).float()
    n, r = norm(x)
    loss, _, dn, _ = z.linear_xent_grad(n, w["embed"], targets, dw=m.grad["embed"])
    dx = norm_backward(dn, x, r)
    for k in reversed(range(m.blocks)):
        x, r, n8, gu = kept[k]
        dy = dx.to(BF16)
        h = torch.empty((len(tokens), m.shapes[f"gate{k}"][0]), dtype=BF16, device=dy.device)
        dn, _, _ = z.glu_backward(dy @ w[f"down{k}"], n8, w[f"gate{k}"], w[f"up{k}"], checkpoint=gu, h=h,
                                  dw_gate=m.grad[f"gate{k}"], dw_up=m.grad[f"up{k}"])
        m.grad[f"down{k}"].copy_(dy.t() @ h)
        dx = dx + norm_backward(dn, x, r)
    # the embedding is also the input
    rows = torch.zeros(m.shapes["embed"], device=dx.device).index_add_(0, tokens, dx)
    m.grad["embed"].copy_((m.grad["embed"].float() + rows).to(BF16))
    return loss


def optimizer_step(m, step, lr=3e-3, max_norm=1.0):
    rows, cols = m.shapes["embed"]
    n = rows * cols
    sq = z.grad_sq_norm(m.grad["embed"].view(-1), n, n, 1, 0)
    stats = z.grad_clip_stats(sq, max_norm)
    z.adamw_shard_step_clipped(m.master["embed"].view(-1), *m.avg, m.grad["embed"].view(-1),
                               m.weight["embed"].view(-1), n, n, 1, 0, lr, 0.9, 0.95, 1e-8, 0.01, step, stats)
    groups = []
    for kind in ("gate", "up", "down"):
        names = [f"{kind}{k}" for k in range(m.blocks)]
        groups.append(([m.master[i] for i in names], [m.momentum[i] for i in names], [m.grad[i] for i in names],
                       [m.weight[i] for i in names]))
    z.muon_step_groups(groups, lr=lr, weight_decay=0.01)


def train(steps=60, tokens=4096, vocab=5003, width=256, ffn=704, blocks=2, seed=0, device="cuda"):
    """The losses of `steps` steps on tokens that follow a fixed random rule."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    after = torch.randperm(vocab, generator=g, device=device)
    m = Model(vocab, width, ffn, blocks, device, seed)
    losses = []
    for step in range(1, steps + 1):
        batch = torch.randint(0, vocab, (tokens,), generator=g, device=device)
        target = after[batch]
        target[::8] = -100  # as padding: not learned from
        losses.append(forward_backward(m, batch, target))
        optimizer_step(m, step)
    return [float(v) for v in torch.cat(losses)]


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--tokens", type=int, default=4096)
    a = p.parse_args()
    for i, v in enumerate(train(a.steps, a.tokens), 1):
        if i == 1 or i % 10 == 0:
            print(f"step {i:4d}  loss {v:.4f}", flush=True)
