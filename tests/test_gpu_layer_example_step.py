"""The example's step: every parameter of AdamW's and of Muon's moves, each expert's
matrices as they do alone, and the bias moves against how often experts were chosen."""
import os
import sys

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_moe_lm as ex  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_every_parameter_and_the_bias_move():
    vocab, heads, kv, head, experts, top, n, length, blocks = 150, 4, 2, 16, 6, 2, 6, 30, 2
    m = ex.Model(vocab, 48, heads, kv, head, 40, experts, top, blocks, DEV, seed=5)
    g = torch.Generator(device=DEV).manual_seed(6)
    batch = lambda: torch.randint(0, vocab, (n, length), generator=g, device=DEV)  # noqa: E731
    for step in (1, 2):
        ex.forward_backward(m, batch(), batch())
        before = {k: v.clone() for k, v in m.of_master.items()}
        momentum = {k: v.clone() for k, v in m.momentum.items()}
        bias = [b.clone() for b in m.bias]
        ex.optimizer_step(m, step)
        for name, v in m.of_master.items():
            assert torch.isfinite(v).all() and torch.equal(v.to(torch.bfloat16), m.weight[name]), name
            # (a row of the embedding that no token has moves by the head's gradient)
            moved = (v != before[name]).flatten(1) if v.dim() > 1 else (v != before[name]).view(1, -1)
            assert moved.any(1).all(), name
        for name in (k for k in m.momentum if k[:2] in ("ga", "up", "do")):
            for e in range(experts):
                p, mo = before[name][e].clone(), momentum[name][e].clone()
                w = torch.empty_like(m.weight[name][e])
                z.muon_step([p], [mo], [m.grad[name][e]], [w], lr=2e-3, weight_decay=0.01)
                assert torch.equal(mo, m.momentum[name][e]), (name, e)
                # (its own Newton-Schulz, in bf16: within 2e-2 of the step)
                step_of = m.of_master[name][e] - before[name][e]
                assert float((p - m.of_master[name][e]).norm()) <= 2e-2 * float(step_of.norm()) + 1e-12, (name, e)
        for b, old, route in zip(m.bias, bias, m.routes):
            counts = torch.bincount(route.experts.flatten().long(), minlength=experts).double()
            want = torch.sign(counts.mean() - counts)
            assert torch.equal(torch.sign((b - old).double()), want)
            assert float(((b - old).double() - 1e-3 * want).abs().max()) <= 2.0 ** -24 * (1e-3 + float(b.abs().max()))
