"""A small decoder with experts trained with the library's operators on one GPU.

    python examples/train_moe_lm.py [--steps 40] [--sequences 16] [--length 128]

A tied embedding [V, D] and blocks of causal attention and a feed-forward of
experts, with a pre-norm each; it learns which token follows which.  One step:

  attention   z.qk_norm_rope normalises and turns queries and keys, read as views
              of one projection; z.qk_norm_rope_backward gives their gradients
              and those of the norms' weights
  experts     z.moe_route chooses (logistic scores, a bias that only the choice
              sees), z.moe_forward and z.moe_backward run the experts, whose
              weights' gradients go straight into the flat gradient vector, and
              z.moe_route_backward takes the weights' gradient back to the router
  loss        z.linear_xent_grad
  step        z.adamw_shard_step_clipped on embedding, routers and norms,
              z.muon_step_groups on all other matrices, each expert's its own

The bias moves against how often an expert was chosen (the route's offsets), so
that all stay in use.  Scores, products and norms of the attention are plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sharded_optimizer_step_adamw_amd as z  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """Weights (bf16), their gradients as views of one flat bf16 vector, and the
    fp32 state of the optimizers: [embedding, routers, norms] in one AdamW
    vector, every other matrix for Muon."""

    def __init__(self, vocab, width, heads, kv_heads, head, ffn, experts, top, blocks, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv, self.head, self.top, self.blocks = heads, kv_heads, head, top, blocks
        shapes = [("embed", (vocab, width))]
        for k in range(blocks):
            shapes += [(f"router{k}", (experts, width)), (f"wq{k}", (head,)), (f"wk{k}", (head,))]
        self.adam = [n for n, _ in shapes]
        for k in range(blocks):
            shapes += [(f"qkv{k}", ((heads + 2 * kv_heads) * head, width)), (f"out{k}", (width, heads * head)),
                       (f"gate{k}", (experts, ffn, width)), (f"up{k}", (experts, ffn, width)),
                       (f"down{k}", (experts, width, ffn))]
        size = lambda s: torch.Size(s).numel()  # noqa: E731
        total = sum(size(s) for _, s in shapes)
        self.shapes = dict(shapes)
        self.master = torch.empty(total, device=device)
        self.flat_weight = torch.empty(total, dtype=BF16, device=device)
        self.flat_grad = torch.zeros(total, dtype=BF16, device=device)
        self.weight, self.grad, self.of_master = {}, {}, {}
        at = 0
        for name, s in shapes:
            cut = slice(at, at + size(s))
            for flat, views in ((self.master, self.of_master), (self.flat_weight, self.weight), (self.flat_grad, self.grad)):
                views[name] = flat[cut].view(s)
            std = 0.02 if name == "embed" else s[-1] ** -0.5
            self.of_master[name].copy_(torch.ones(s, device=device) if name[:2] in ("wq", "wk") else
                                       torch.randn(s, generator=g, device=device) * std)
            at += size(s)
            if name == self.adam[-1]:
                self.adam_size = at
        self.flat_weight.copy_(self.master)
        self.avg = [torch.zeros(self.adam_size, device=device) for _ in range(2)]
        self.momentum = {n: torch.zeros_like(v) for n, v in self.of_master.items() if n not in self.adam}
        self.bias = [torch.zeros(experts, device=device) for _ in range(blocks)]
        self.routes = [None] * blocks


def norm(x):
    """x / rms(x) in bf16, and the fp32 1 / rms."""
    r = torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)
    return (x.float() * r).to(BF16), r


def norm_backward(dn, x, r):
    n, d = x.float() * r, dn.float()
    return r * (d - n * (d * n).mean(1, keepdim=True))


def by_head(v, n, repeat=1):
    """[tokens, heads, head] to fp32 [n, heads, length, head], heads shared by `repeat` queries repeated."""
    v = v.view(n, -1, *v.shape[1:]).transpose(1, 2).float()
    return v.repeat_interleave(repeat, 1) if repeat > 1 else v


def attend(q, k, v):
    """Causal attention of [n, heads, length, head]: the result and the probabilities."""
    s = q @ k.transpose(2, 3).contiguous() * q.shape[3] ** -0.5
    s.masked_fill_(torch.ones(s.shape[2:], dtype=torch.bool, device=s.device).triu(1), -torch.inf)
    p = torch.softmax(s, 3)
    return p @ v, p


def attend_backward(do, q, k, v, p):
    dp = do @ v.transpose(2, 3).contiguous()
    ds = p * (dp - (dp * p).sum(3, keepdim=True)) * q.shape[3] ** -0.5
    return ds @ k, ds.transpose(2, 3).contiguous() @ q, p.transpose(2, 3).contiguous() @ do


def forward_backward(m, tokens, targets):
    """The loss (device scalar) of tokens and targets [n, length]; every gradient
    is left in m.flat_grad."""
    n, length = tokens.shape
    w, heads, kv, head = m.weight, m.heads, m.kv, m.head
    share = heads // kv
    table = z.rope_table(length, head)
    position = torch.arange(length, device=tokens.device).repeat(n)
    flat = lambda v: v.transpose(1, 2).reshape(n * length, -1)  # noqa: E731
    x = w["embed"][tokens.view(-1)].float()
    kept = []
    for k in range(m.blocks):
        a, ra = norm(x)
        mixed = (a @ w[f"qkv{k}"].t()).view(-1, heads + 2 * kv, head)
        rope = (mixed[:, :heads], mixed[:, heads:heads + kv], table, position, w[f"wq{k}"], w[f"wk{k}"])
        yq, yk = z.qk_norm_rope(*rope)
        parts = by_head(yq, n), by_head(yk, n, share), by_head(mixed[:, heads + kv:], n, share)
        o, p = attend(*parts)
        o = flat(o).to(BF16)
        x1 = x + (o @ w[f"out{k}"].t()).float()
        b, rb = norm(x1)
        logits = b.float() @ w[f"router{k}"].float().t()
        route = z.moe_route(logits, m.top, score="sigmoid", bias=m.bias[k])
        y = z.moe_forward(b, w[f"gate{k}"], w[f"up{k}"], w[f"down{k}"], route)
        kept.append((x, a, ra, rope, parts, p, o, x1, b, rb, logits))
        m.routes[k] = route
        x = x1 + y.float()
    h, r = norm(x)
    loss, _, dh, _ = z.linear_xent_grad(h, w["embed"], targets.view(-1), dw=m.grad["embed"])
    dx = norm_backward(dh, x, r)
    for k in reversed(range(m.blocks)):
        x, a, ra, rope, parts, p, o, x1, b, rb, logits = kept[k]
        dy = dx.to(BF16)
        db, _, _, _, dweights = z.moe_backward(dy, b, w[f"gate{k}"], w[f"up{k}"], w[f"down{k}"], m.routes[k],
                                               dw_gate=m.grad[f"gate{k}"], dw_up=m.grad[f"up{k}"],
                                               dw_down=m.grad[f"down{k}"])
        dlogits = z.moe_route_backward(dweights, logits, m.routes[k], score="sigmoid")
        m.grad[f"router{k}"].copy_(dlogits.t() @ b.float())
        dx = dx + norm_backward(db.float() + dlogits @ w[f"router{k}"].float(), x1, rb)
        dy = dx.to(BF16)
        m.grad[f"out{k}"].copy_(dy.t() @ o)
        dq, dk, dv = attend_backward(by_head((dy @ w[f"out{k}"]).view(-1, heads, head), n), *parts, p)
        dk, dv = (v.view(n, kv, share, length, head).sum(2) for v in (dk, dv))
        dmixed = torch.empty_like(rope[0].as_strided((n * length, heads + 2 * kv, head), rope[0].stride()))
        dmixed[:, heads + kv:] = flat(dv).view(-1, kv, head).to(BF16)
        z.qk_norm_rope_backward(flat(dq).view(-1, heads, head).to(BF16), flat(dk).view(-1, kv, head).to(BF16), *rope,
                                dq=dmixed[:, :heads], dk=dmixed[:, heads:heads + kv], dw_q=m.grad[f"wq{k}"],
                                dw_k=m.grad[f"wk{k}"])
        dmixed = dmixed.view(n * length, -1)
        m.grad[f"qkv{k}"].copy_(dmixed.t() @ a)
        dx = dx + norm_backward(dmixed @ w[f"qkv{k}"], x, ra)
    # the embedding is also the input
    rows = torch.zeros(m.shapes["embed"], device=dx.device).index_add_(0, tokens.view(-1), dx)
    m.grad["embed"].copy_((m.grad["embed"].float() + rows).to(BF16))
    return loss


def optimizer_step(m, step, lr=2e-3, max_norm=1.0):
    n = m.adam_size
    sq = z.grad_sq_norm(m.flat_grad[:n], n, n, 1, 0)
    stats = z.grad_clip_stats(sq, max_norm)
    z.adamw_shard_step_clipped(m.master[:n], *m.avg, m.flat_grad[:n], m.flat_weight[:n], n, n, 1, 0, lr, 0.9, 0.95, 1e-8,
                               0.01, step, stats)
    groups = {}
    for name, momentum in m.momentum.items():
        # an expert's matrices step as matrices of their own
        for part in zip(*(v.view(-1, *v.shape[-2:]) for v in (m.of_master[name], momentum, m.grad[name], m.weight[name]))):
            groups.setdefault(tuple(part[0].shape), []).append(part)
    for parts in groups.values():
        for at in range(0, len(parts), z.MAX_BATCH):
            z.muon_step_groups([tuple(map(list, zip(*parts[at:at + z.MAX_BATCH])))], lr=lr, weight_decay=0.01)
    for bias, route in zip(m.bias, m.routes):
        chosen = (route.offsets[1:] - route.offsets[:-1]).float()
        bias += 1e-3 * torch.sign(chosen.mean() - chosen)


def train(steps=40, sequences=16, length=128, vocab=1009, width=128, heads=4, kv_heads=2, head=32, ffn=96, experts=8,
          top=2, blocks=2, seed=0, device="cuda"):
    """The losses of `steps` steps on tokens that follow a fixed random rule."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    after = torch.randperm(vocab, generator=g, device=device)
    m = Model(vocab, width, heads, kv_heads, head, ffn, experts, top, blocks, device, seed)
    losses = []
    for step in range(1, steps + 1):
        batch = torch.randint(0, vocab, (sequences, length), generator=g, device=device)
        losses.append(forward_backward(m, batch, after[batch]))
        optimizer_step(m, step)
    return [float(v) for v in torch.cat(losses)]


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--sequences", type=int, default=16)
    p.add_argument("--length", type=int, default=128)
    a = p.parse_args()
    for i, v in enumerate(train(a.steps, a.sequences, a.length), 1):
        if i == 1 or i % 10 == 0:
            print(f"step {i:4d}  loss {v:.4f}", flush=True)
