"""The example runs norms, rotation, routing, experts, the head's loss and the
optimizers together: its gradients agree with torch's through the same model in
float32, and it runs."""
import math
import os
import sys

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z  # noqa: F401
from train_reference import act

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_moe_lm as ex  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_gradients_agree_with_float32_torch():
    vocab, heads, kv, head, experts, top, n, length = 200, 4, 2, 16, 6, 2, 5, 24
    m = ex.Model(vocab, 48, heads, kv, head, 40, experts, top, 2, DEV, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    for name in m.adam:  # norms' weights other than 1
        if name[:2] in ("wq", "wk"):
            m.weight[name].copy_(1 + 0.3 * torch.randn(head, generator=g, device=DEV))
    tokens = torch.randint(0, vocab, (n, length), generator=g, device=DEV)
    targets = torch.randint(0, vocab, (n, length), generator=g, device=DEV)
    loss = ex.forward_backward(m, tokens, targets)
    w = {k: v.float().requires_grad_() for k, v in m.weight.items()}
    rms = lambda v: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    cs = ref.table(length, head, 10000.0).float().to(DEV).repeat(n, 1, 1)
    x = w["embed"][tokens.view(-1)]
    for k in range(2):
        mixed = (rms(x) @ w[f"qkv{k}"].t()).view(-1, heads + 2 * kv, head)
        q, ke, v = mixed.split([heads, kv, kv], 1)
        q = ref.turn(rms(q) * w[f"wq{k}"], cs, "half")
        ke = ref.turn(rms(ke) * w[f"wk{k}"], cs, "half")
        q, ke, v = (t.view(n, length, -1, head).transpose(1, 2) for t in (q, ke, v))
        ke, v = (t.repeat_interleave(heads // kv, 1) for t in (ke, v))
        s = (q @ ke.transpose(2, 3)) * head ** -0.5
        s = s.masked_fill(torch.ones(length, length, dtype=torch.bool, device=DEV).triu(1), -math.inf)
        o = (torch.softmax(s, 3) @ v).transpose(1, 2).reshape(n * length, -1)
        x = x + o @ w[f"out{k}"].t()
        b = rms(x)
        # (the same choice: it has no gradient)
        share = ref.weights(b @ w[f"router{k}"].t(), m.routes[k].experts, "sigmoid", True, 1.0)
        for e in range(experts):
            p = (share * (m.routes[k].experts == e)).sum(1, keepdim=True)
            h = act(b @ w[f"gate{k}"][e].t(), "silu")[0] * (b @ w[f"up{k}"][e].t())
            x = x + p * (h @ w[f"down{k}"][e].t())
    want = torch.nn.functional.cross_entropy(rms(x) @ w["embed"].t(), targets.view(-1))
    want.backward()
    # bf16 activations, some thirty roundings of 2^-8 in a row
    assert abs(float(loss) - float(want.detach())) <= 30 * 2.0 ** -8 * float(want.detach())
    for name, v in w.items():
        off = float((m.grad[name].float() - v.grad).norm() / v.grad.norm())
        print(f"{name}: gradient off by {off:.4f}", flush=True)
        assert off <= 30 * 2.0 ** -8, name


def test_the_example_runs():
    losses = ex.train(steps=3, sequences=4, length=40, vocab=307, width=64, head=16, ffn=48, experts=5, top=3)
    print(losses, flush=True)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
