"""The measured cases of a decoder layer's operators: norms and rotation of
queries and keys, routing to experts, and the experts' gated feed-forward.

Three kinds of pass, as a training program makes them:

  rope   queries and keys normalised for each head and rotated to their
         positions, forward alone or with the gradients of both inputs and of
         the norms' weights
  route  a router's logits to each token's experts and weights and to the
         order in which the experts read the tokens, forward alone or with the
         gradient of the logits
  moe    the experts' gated feed-forward of tokens whose experts are chosen:
         y, or y and the gradients of x, of every expert's three weights and of
         the tokens' weights

Sizes: t tokens; hq, hk heads of queries and keys, hd their width, rot of it
rotated; e experts, k of them a token; d model width, f an expert's width.
"""
import math

import torch

own = False

EPS = 1e-6


def _rope(name, t, hq, hk, hd, rot, style, weights, back):
    return {"name": name, "op": "rope", "t": t, "hq": hq, "hk": hk, "hd": hd, "rot": rot, "style": style,
            "weights": weights, "back": back}


def _route(name, t, e, k, score, bias, groups, top, norm, scale, logits, padded, back):
    return {"name": name, "op": "route", "t": t, "e": e, "k": k, "score": score, "bias": bias, "groups": groups,
            "top": top, "norm": norm, "scale": scale, "logits": logits, "padded": padded, "back": back}


def _moe(name, t, d, f, e, k, act, skew, padded, back):
    return {"name": name, "op": "moe", "t": t, "d": d, "f": f, "e": e, "k": k, "act": act, "skew": skew,
            "padded": padded, "back": back}


def listed():
    return [
        # a short sequence through the small model's heads of 64, forward alone: latency
        _rope("rope_fwd_64x12+12x64", 64, 12, 12, 64, 64, "half", True, False),
        # one micro-batch of a decoder with 32 query and 8 key heads of 128, its training pass
        _rope("rope_step_8192x32+8x128", 8192, 32, 8, 128, 128, "half", True, True),
        # a long packed batch of the same heads: past the memory-side cache
        _rope("rope_step_65536x32+8x128", 65536, 32, 8, 128, 128, "half", True, True),
        # uneven sequences, heads of 80 of which 48 turn, neighbours in pairs, no weights: no power of two
        _rope("rope_step_1531x7+1x80", 1531, 7, 1, 80, 48, "pairs", False, True),
        # a short sequence over few experts, forward alone: latency
        _route("route_fwd_64x8k2", 64, 8, 2, "softmax", False, 1, 1, True, 1.0, "fp32", 0.0, False),
        # a long micro-batch over many experts in groups: sigmoid scores, a bias for balance, the training pass
        _route("route_step_16384x256k8", 16384, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "fp32", 0.0, True),
        # a padded batch, 60 experts, bf16 logits with their ties, weights not renormalised
        _route("route_step_4099x60k6", 4099, 60, 6, "softmax", True, 1, 1, False, 1.0, "bf16", 0.1, True),
        # scoring a short sequence: few tokens an expert, one read of every expert's weights
        _moe("moe_fwd_48x768x512e16k2", 48, 768, 512, 16, 2, "silu", 0.5, 0.0, False),
        # evaluation of a layer of few wide experts, forward alone
        _moe("moe_fwd_4096x2048x5632e8k2", 4096, 2048, 5632, 8, 2, "silu", 0.3, 0.0, False),
        # a training pass over many narrow experts: products of 512 tokens each
        _moe("moe_step_4096x2048x1024e64k8", 4096, 2048, 1024, 64, 8, "silu", 0.3, 0.0, True),
        # a training pass of a 4096-wide decoder's layer: the largest call
        _moe("moe_step_8192x4096x2048e16k4", 8192, 4096, 2048, 16, 4, "silu", 0.3, 0.0, True),
        # a padded batch on odd sizes, a few experts with most of the tokens
        _moe("moe_step_1777x1000x602e13k3", 1777, 1000, 602, 13, 3, "gelu", 1.5, 0.2, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["rope", "route", "moe", "moe"])
    if op == "rope":
        hd = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(16, 128)])
        hk = rng.randint(1, 8)
        return _rope("", _log(rng, 16, 32768), hk * rng.randint(1, 5), hk, hd,
                     hd if rng.random() < 0.6 else 2 * rng.randint(1, hd // 2), rng.choice(["half", "half", "pairs"]),
                     rng.random() < 0.7, rng.random() < 0.7)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        e = groups * _log(rng, 4, 512 // groups)
        top = rng.randint(1, groups)
        return _route("", _log(rng, 16, 16384), e, rng.randint(1, min(8, top * (e // groups))),
                      rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, top, rng.random() < 0.6,
                      rng.choice([1.0, 2.5]), rng.choice(["fp32", "fp32", "bf16"]), rng.choice([0.0, 0.1]),
                      rng.random() < 0.7)
    # (no more products than the largest listed case has)
    t, e = _log(rng, 16, 8192), _log(rng, 2, 64)
    k = rng.randint(1, min(8, e))
    most = 8192 * 4 * 4096 * 2048 // (t * k)
    d = _log(rng, 64, 4096)
    f = _log(rng, 64, max(65, min(5632, most // d, 4096 * 2048 * 16 // (d * e))))
    if rng.random() < 0.5:
        d, f = max(64, d // 64 * 64), max(64, f // 64 * 64)
    return _moe("", t, d, f, e, k, rng.choice(["silu", "gelu"]), rng.choice([0.0, 0.3, 1.0]),
                rng.choice([0.0, 0.2]), rng.random() < 0.6)


def _normal(shape, std, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = case["t"]
    s = dict(case)
    if case["op"] == "rope":
        hq, hk, hd, rot = case["hq"], case["hk"], case["hd"], case["rot"]
        # q and k are views of one projection, [t, (hq + 2 hk) hd], as a program has them
        mixed = _normal((t, hq + 2 * hk, hd), 1.0, gen)
        # uneven sequences, one behind the other
        starts = torch.rand((t,), generator=gen, device="cuda") < 4.0 / t
        starts[0] = True
        at = torch.arange(t, device="cuda")
        position = at - torch.cummax(torch.where(starts, at, 0), 0).values
        rate = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(t, device="cuda", dtype=torch.float64)[:, None] * rate
        s.update(q=mixed[:, :hq], k=mixed[:, hq:hq + hk], position=position,
                 table=torch.stack([angle.cos(), angle.sin()], 2).float(), wq=None, wk=None)
        if case["weights"]:
            s.update(wq=(1.0 + 0.2 * torch.randn((hd,), generator=gen, device="cuda")).to(torch.bfloat16),
                     wk=(1.0 + 0.2 * torch.randn((hd,), generator=gen, device="cuda")).to(torch.bfloat16))
        if case["back"]:
            s.update(dq=_normal((t, hq, hd), 1e-3, gen), dk=_normal((t, hk, hd), 1e-3, gen))
        return s
    e, k = case["e"], case["k"]
    pad = torch.rand((t, 1), generator=gen, device="cuda") < case["padded"]
    if case["op"] == "route":
        logits = torch.randn((t, e), generator=gen, device="cuda") * 1.5
        logits += 0.5 * torch.randn((1, e), generator=gen, device="cuda")  # experts of uneven popularity
        # the batch's padding: no expert is left
        logits = logits.masked_fill(pad, -math.inf).to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)
        s.update(x=logits, shift=None)
        if case["bias"]:
            s.update(shift=0.02 * torch.randn((e,), generator=gen, device="cuda"))
        if case["back"]:
            s.update(dw=1e-3 * torch.randn((t, k), generator=gen, device="cuda"))
        return s
    d, f = case["d"], case["f"]
    x = torch.randn((t, e), generator=gen, device="cuda")
    x += case["skew"] * torch.randn((1, e), generator=gen, device="cuda")
    x, experts = torch.topk(x, k, 1)
    s.update(x=_normal((t, d), 1.0, gen), wg=_normal((e, f, d), d ** -0.5, gen),
             wu=_normal((e, f, d), d ** -0.5, gen), wd=_normal((e, d, f), f ** -0.5, gen),
             experts=torch.where(pad, -1, experts).to(torch.int32),
             share=torch.where(pad, 0.0, torch.softmax(x, 1)))
    if case["back"]:
        s.update(dy=_normal((t, d), 1e-3, gen))
    return s


# ------------------------------------------------------------- plain forms

def _turn(v, c, s, style):
    """v [t, h, rot] turned by the angles of cosine c and sine s [t, 1, rot / 2]."""
    half = v.shape[2] // 2
    a, b = (v[..., :half], v[..., half:]) if style == "half" else (v[..., 0::2], v[..., 1::2])
    a, b = a * c - b * s, b * c + a * s
    return torch.cat([a, b], 2) if style == "half" else torch.stack([a, b], 3).flatten(2)


def _plain_rope(s):
    out = {}
    at = s["table"][s["position"]].unsqueeze(1)
    c, sn, rot, style = at[..., 0], at[..., 1], s["rot"], s["style"]
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].float()
        r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
        n = x * r
        y = n if w is None else n * w.float()
        out[name] = torch.cat([_turn(y[..., :rot], c, sn, style), y[..., rot:]], 2).to(torch.bfloat16)
        if s["back"]:
            g = s["d" + name].float()
            g = torch.cat([_turn(g[..., :rot], c, -sn, style), g[..., rot:]], 2)
            if w is not None:
                out["dw" + name] = (g * n).sum((0, 1)).to(torch.bfloat16)
                g = g * w.float()
            out["d" + name] = (r * (g - n * (g * n).mean(2, keepdim=True))).to(torch.bfloat16)
    return out


def _order(experts, e):
    """The slots of [t, k] experts sorted by expert (-1: none), each expert's
    first place, and every slot's place: int32, -1 behind the last and for
    slots without an expert."""
    flat = experts.flatten().long()
    n = flat.numel()
    key, order = torch.sort(torch.where(flat < 0, e, flat), stable=True)
    first = torch.searchsorted(key, torch.arange(e + 1, device=key.device))
    at = torch.arange(n, device=key.device)
    place = torch.empty_like(at)
    place[order] = torch.where(key < e, at, -1)
    return first.int(), torch.where(key < e, order, -1).int(), place.view(experts.shape).int()


def _plain_route(s):
    x, k, e, groups = s["x"].float(), s["k"], s["e"], s["groups"]
    there = x > -math.inf
    # which experts are chosen goes by values that lie close together: in 64 bits
    wide = torch.where(there, x.double(), -1e300)
    if s["score"] == "softmax":
        p = torch.exp(wide - wide.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-wide))
    key = p if s["shift"] is None else p + s["shift"].double()
    key = torch.where(there, key, -math.inf)
    if groups > 1:
        part = key.view(len(x), groups, e // groups)
        best = torch.sort(part, dim=2, descending=True).values[..., :2]
        best = torch.where(best > -math.inf, best, 0.0).sum(2)
        best = torch.where(part.amax(2) > -math.inf, best, -math.inf)
        rank = torch.sort(torch.sort(best, dim=1, descending=True, stable=True).indices, 1).indices
        key = torch.where((rank < s["top"]).unsqueeze(2), part, -math.inf).view(len(x), e)
    key, chosen = torch.sort(key, dim=1, descending=True, stable=True)
    some = key[:, :k] > -math.inf
    chosen = chosen[:, :k]
    w = torch.where(some, p.float().gather(1, chosen), 0.0)
    total = w.sum(1, keepdim=True)
    if s["norm"]:
        w = w / torch.where(total > 0, total, 1.0)
    out = {"experts": torch.where(some, chosen, -1).int(), "weights": w * s["scale"]}
    out["offsets"], out["order"], out["place"] = _order(out["experts"], e)
    if s["back"]:
        g = torch.where(some, s["dw"] * s["scale"], 0.0)
        if s["norm"]:
            g = (g - (g * w).sum(1, keepdim=True)) / torch.where(total > 0, total, 1.0)
        dp = torch.zeros_like(x).scatter_add_(1, chosen, torch.where(some, g, 0.0))
        p = torch.where(there, p.float(), 0.0)
        if s["score"] == "softmax":
            dx = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            dx = dp * p * (1.0 - p)
        out["dlogits"] = dx.to(s["x"].dtype)
    return out


def _act(g, kind):
    """The activation of g and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    k = math.sqrt(2.0 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * g * g)


def _plain_moe(s):
    experts, share = s["experts"], s["share"].flatten()
    e, k = s["e"], s["k"]
    first, order, _ = _order(experts, e)
    # (products of uneven sizes: a program of elementary operations goes through the experts)
    first, order = first.tolist(), order.long()
    x = s["x"].float()
    y = torch.zeros_like(x)
    back = s["back"]
    if back:
        dy, dx, dshare = s["dy"].float(), torch.zeros_like(x), torch.zeros_like(share)
        dwg, dwu, dwd = (torch.empty_like(s[n]) for n in ("wg", "wu", "wd"))
    for i in range(e):
        slot = order[first[i]:first[i + 1]]
        row, p = slot // k, share[slot].unsqueeze(1)
        wg, wu, wd = s["wg"][i].float(), s["wu"][i].float(), s["wd"][i].float()
        xe = x[row]
        g, u = xe @ wg.t(), xe @ wu.t()
        a, da = _act(g, s["act"])
        h = a * u
        y.index_add_(0, row, (h @ wd.t()) * p)
        if back:
            de = dy[row]
            dh = de @ wd
            dshare[slot] = (dh * h).sum(1)
            dwd[i] = (de.t() @ (h * p)).to(torch.bfloat16)
            dh = dh * p
            du, dg = dh * a, dh * u * da
            dx.index_add_(0, row, dg @ wg + du @ wu)
            dwg[i], dwu[i] = (dg.t() @ xe).to(torch.bfloat16), (du.t() @ xe).to(torch.bfloat16)
    out = {"y": y.to(torch.bfloat16)}
    if back:
        out.update(dx=dx.to(torch.bfloat16), dwg=dwg, dwu=dwu, dwd=dwd, dshare=dshare.view(experts.shape))
    return out


# ------------------------------------------------------- the framework's calls

def _own_rope(s):
    import sharded_optimizer_step_adamw_amd as z
    rest = {"w_q": s["wq"], "w_k": s["wk"], "eps": EPS, "style": s["style"]}
    out = dict(zip("qk", z.qk_norm_rope(s["q"], s["k"], s["table"], s["position"], **rest)))
    if s["back"]:
        out["dq"], out["dk"], dwq, dwk = z.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["table"],
                                                                 s["position"], **rest)
        if s["weights"]:
            out.update(dwq=dwq, dwk=dwk)
    return out


def _own_route(s):
    import sharded_optimizer_step_adamw_amd as z
    rest = {"score": s["score"], "renormalise": s["norm"], "scale": s["scale"]}
    r = z.moe_route(s["x"], s["k"], bias=s["shift"], groups=s["groups"], top_groups=s["top"], **rest)
    out = r._asdict()
    if s["back"]:
        out["dlogits"] = z.moe_route_backward(s["dw"], s["x"], r, **rest)
    return out


def _own_moe(s):
    import sharded_optimizer_step_adamw_amd as z
    r = z.moe_plan(s["experts"], s["share"], s["e"])
    w = (s["wg"], s["wu"], s["wd"])
    out = {"y": z.moe_forward(s["x"], *w, r, act=s["act"])}
    if s["back"]:
        out["dx"], out["dwg"], out["dwu"], out["dwd"], out["dshare"] = z.moe_backward(s["dy"], s["x"], *w, r,
                                                                                     act=s["act"])
    return out


def run(state):
    if state["op"] == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    if state["op"] == "route":
        return _own_route(state) if own else _plain_route(state)
    return _own_moe(state) if own else _plain_moe(state)


# ---------------------------------------------------------------------- work

def work(case):
    t = case["t"]
    if case["op"] == "rope":
        rows, hd = t * (case["hq"] + case["hk"]), case["hd"]
        # x in, y out; the backward dy and x in, dx out (the table's angles are those of t positions at most)
        each = 2 * rows * hd
        io = 2 * each + 8 * t + 4 * t * case["rot"]
        return {"bytes": io + (3 * each + 8 * t + 4 * t * case["rot"] if case["back"] else 0),
                "flops": rows * hd * (20 if case["back"] else 7)}
    if case["op"] == "route":
        e, k = case["e"], case["k"]
        each = 2 if case["logits"] == "bf16" else 4
        io = t * e * each + 16 * t * k + 4 * e
        # the backward: logits, experts and weights' gradients in, the logits' gradient out
        return {"bytes": io + (2 * t * e * each + 8 * t * k if case["back"] else 0),
                "flops": t * e * (20 if case["back"] else 10)}
    d, f, e, k = case["d"], case["f"], case["e"], case["k"]
    slots = t * k * (1.0 - case["padded"])
    io = 4 * t * d + 8 * t * k + 6 * e * d * f
    if not case["back"]:
        return {"bytes": io, "flops": 6 * slots * d * f}
    # the backward reads dy, x and the weights and writes dx, the weights' gradients and those of the tokens' weights
    return {"bytes": io + 6 * t * d + 12 * t * k + 12 * e * d * f, "flops": 18 * slots * d * f}


# -------------------------------------------------------------------- exact

def _exact_rope(s):
    c = torch.view_as_complex(s["table"].double()[s["position"]])[:, None]
    rot, out = s["rot"], {}
    for name in "qk":
        x = s[name].double().requires_grad_(s["back"])
        w = None if s["w" + name] is None else s["w" + name].double().requires_grad_(s["back"])
        y = x / (torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 / s["hd"] + EPS) ** 0.5
        if w is not None:
            y = y * w
        part = y[..., :rot].unflatten(2, (2, rot // 2) if s["style"] == "half" else (rot // 2, 2))
        part = part if s["style"] == "pairs" else part.transpose(2, 3)
        part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * c)
        part = part if s["style"] == "pairs" else part.transpose(2, 3)
        y = torch.cat([part.flatten(2), y[..., rot:]], 2)
        out[name] = y.detach()
        if s["back"]:
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["d" + name].double())
            out["d" + name] = grads[0]
            if w is not None:
                out["dw" + name] = grads[1]
    return out


def _exact_order(experts, e):
    """By counting: how many slots of smaller experts, and of the same one before."""
    flat = experts.flatten().long()
    one = torch.nn.functional.one_hot(torch.where(flat < 0, e, flat), e + 1)[:, :e].int()
    count = one.sum(0)
    first = torch.cat([torch.zeros_like(count[:1]), torch.cumsum(count, 0)])
    before = (torch.cumsum(one, 0) * one).sum(1) - 1
    used = flat >= 0
    place = torch.where(used, first[flat.clamp(min=0)] + before, -1)
    order = torch.full_like(flat, -1)
    order[place[used]] = torch.nonzero(used).squeeze(1)
    return first.int(), order.int(), place.view(experts.shape).int()


def _exact_route(s):
    x = s["x"].double().requires_grad_(s["back"])
    t, e, k = s["t"], s["e"], s["k"]
    gone = torch.isinf(x.detach())
    # (a row without any expert: any numbers, used by nobody)
    z = torch.where(gone & ~gone.all(1, keepdim=True), -math.inf, torch.where(gone, 0.0, x))
    p = torch.softmax(z, 1) if s["score"] == "softmax" else torch.sigmoid(z)
    key = p.detach().clone()
    if s["shift"] is not None:
        key += s["shift"].double()
    key[gone] = -math.inf
    if s["groups"] > 1:
        size = e // s["groups"]
        value = key.view(t, -1, size).topk(min(2, size), 2).values.clamp(min=-1e30)
        value = torch.where(value > -1e30, value, 0.0).sum(2)
        value[gone.view(t, -1, size).all(2)] = -math.inf
        for _ in range(s["groups"] - s["top"]):  # drop the worst, of equal ones the last
            worst = value.shape[1] - 1 - value.flip(1).argmin(1)
            key.view(t, -1, size)[torch.arange(t, device=key.device), worst] = -math.inf
            value[torch.arange(t, device=key.device), worst] = math.inf
    picked, rows = [], torch.arange(t, device=key.device)
    for _ in range(k):
        best = key.argmax(1)
        picked.append(torch.where(key[rows, best] > -math.inf, best, -1))
        key[rows, best] = -math.inf
    experts = torch.stack(picked, 1)
    some = experts >= 0
    w = torch.where(some, p.gather(1, experts.clamp(min=0)), 0.0)
    if s["norm"]:
        w = w / torch.where(some.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    w = w * s["scale"]
    out = {"experts": experts.int(), "weights": w.detach()}
    out["offsets"], out["order"], out["place"] = _exact_order(out["experts"], e)
    if s["back"]:
        out["dlogits"] = torch.autograd.grad(w, x, torch.where(some, s["dw"].double(), 0.0))[0]
    return out


def _exact_moe(s):
    """Expert by expert, the gradients by autograd of the definition."""
    back, y = s["back"], torch.zeros((s["t"], s["d"]), dtype=torch.float64, device="cuda")
    x = s["x"].double()
    share = s["share"].double()
    dx, dshare = torch.zeros_like(x), torch.zeros_like(share)
    dw = {n: torch.zeros(s[n].shape, dtype=torch.float32, device="cuda") for n in ("wg", "wu", "wd")} if back else {}
    for i in range(s["e"]):
        row, j = torch.nonzero(s["experts"] == i, as_tuple=True)
        with torch.enable_grad():
            leaf = [v.requires_grad_(back) for v in (x[row], share[row, j], *(s[n][i].double() for n in ("wg", "wu", "wd")))]
            g, u = torch.mm(leaf[0], leaf[2].T), torch.mm(leaf[0], leaf[3].T)
            kind = {"approximate": "tanh"} if s["act"] == "gelu" else {}
            a = getattr(torch.nn.functional, s["act"])(g, **kind)
            part = torch.mm(a * u, leaf[4].T) * leaf[1][:, None]
        y.index_add_(0, row, part.detach())
        if back:
            grads = torch.autograd.grad(part, leaf, s["dy"][row].double())
            dx.index_add_(0, row, grads[0])
            dshare[row, j] = grads[1]
            for n, v in zip(("wg", "wu", "wd"), grads[2:]):
                dw[n][i] = v
    out = {"y": y}
    if back:
        out.update(dx=dx, dwg=dw["wg"], dwu=dw["wu"], dwd=dw["wd"], dshare=dshare)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "route": _exact_route, "moe": _exact_moe}[case["op"]](s)
