"""Plain 64-bit references of a decoder layer's operators (norms and rotation
of queries and keys, routing, the experts' gated block) for the tests, and the
error bounds that follow from the roundings each operator makes.

HALF_F32 is half a step of fp32 relative to the value; a sum of n terms in any
order is off by at most n of those of its terms' magnitudes."""
import math

import torch

from train_reference import HALF_BF16, HALF_F16, HALF_F32, act

FAST = 2.0 ** -19  # the hardware's exponential and reciprocal in an activation, relatively


# ------------------------------------------------------------- norm, rotation

def turn(v, cs, style, back=False):
    """v [t, h, width], its first elements turned by cs [t, rot / 2, 2]."""
    half = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1 if back else 1)
    out = v.clone()
    a, b = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    out[..., a], out[..., b] = v[..., a] * c - v[..., b] * s, v[..., b] * c + v[..., a] * s
    return out


def rope(x, dy, w, cs, eps, style):
    """(y, dx, dw) and their bounds, of float64 x, dy [t, h, width] (dy or w may
    be None); cs [t, rot / 2, 2]."""
    width = x.shape[2]
    r = (x.square().mean(2, keepdim=True) + eps).rsqrt()
    n = x * r
    weight = torch.ones(width, dtype=torch.float64) if w is None else w
    y = turn(n * weight, cs, style)
    # n: the mean's width terms, halved by the root, and some 6 operations; the turn 3 more
    e = (width / 2 + 12) * HALF_F32
    y_e = HALF_BF16 * y.abs() + e * turn_terms((n * weight).abs(), cs, style)
    if dy is None:
        return y, None, None, y_e, None, None
    g, g_abs = turn(dy, cs, style, True), turn_terms(dy.abs(), cs, style)
    m = (g * weight * n).mean(2, keepdim=True)
    m_abs = (g_abs * weight.abs() * n.abs()).mean(2, keepdim=True)
    dx = r * (g * weight - n * m)
    dx_e = HALF_BF16 * dx.abs() + r * ((width / 2 + 20) * HALF_F32 * g_abs * weight.abs()
                                       + (2 * width + 40) * HALF_F32 * n.abs() * m_abs)
    dw = (g * n).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    dw_e = HALF_BF16 * dw.abs() + (terms + width / 2 + 20) * HALF_F32 * (g_abs * n.abs()).sum((0, 1))
    return y, dx, dw, y_e, dx_e, dw_e


def turn_terms(v, cs, style):
    """What the turn adds up, in magnitude: v >= 0."""
    half = cs.shape[1]
    c, s = cs[:, None, :, 0].abs(), cs[:, None, :, 1].abs()
    out = v.clone()
    a, b = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    out[..., a], out[..., b] = v[..., a] * c + v[..., b] * s, v[..., b] * c + v[..., a] * s
    return out


def table(positions, rot, base):
    i = torch.arange(rot // 2, dtype=torch.float64)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2 * i / rot)
    return torch.stack([angle.cos(), angle.sin()], 2)


# -------------------------------------------------------------------- routing

def choose(z, top, score, bias, groups, top_groups):
    """The chosen experts [t, top] of float64 logits, by going through them."""
    t, experts = z.shape
    out = torch.full((t, top), -1, dtype=torch.int32)
    for i in range(t):
        row = z[i]
        there = [e for e in range(experts) if row[e] != -math.inf and (bias is None or bias[e] != -math.inf)]
        finite = row[row > -math.inf]
        if score == "sigmoid":
            p = [float(torch.sigmoid(v)) for v in row]
        elif len(finite):
            lse = torch.logsumexp(finite, 0)
            p = [float(torch.exp(v - lse)) for v in row]
        else:
            p = [0.0] * experts
        plain = bias is None and groups == 1
        key = {e: float(row[e]) if plain else p[e] + (0.0 if bias is None else float(bias[e])) for e in there}
        key = {e: -1e308 if math.isnan(k) else k for e, k in key.items()}
        if groups > 1:
            size = experts // groups
            best = {}
            for g in range(groups):
                mine = sorted((key[e] for e in there if e // size == g), reverse=True)[:2]
                if mine:
                    best[g] = sum(mine)
            keep = sorted(best, key=lambda g: (-best[g], g))[:top_groups]
            key = {e: k for e, k in key.items() if e // size in keep}
        order = sorted(key, key=lambda e: (-key[e], e))[:top]
        out[i, :len(order)] = torch.tensor(order, dtype=torch.int32)
    return out


def weights(z, chosen, score, renormalise, scale):
    """Weights of float64 logits (differentiable), 0 where chosen is -1."""
    some = chosen >= 0
    at = chosen.clamp(min=0).long()
    safe = torch.where(z == -math.inf, torch.full_like(z, -1e30), z)
    if renormalise:
        l = (torch.nn.functional.logsigmoid(safe) if score == "sigmoid" else safe).gather(1, at)
        l = torch.where(some, l, torch.full_like(l, -1e30))
        w = torch.softmax(l, 1)
    elif score == "sigmoid":
        w = torch.sigmoid(safe).gather(1, at)
    else:
        w = torch.softmax(safe, 1).gather(1, at)
    return torch.where(some, w, torch.zeros_like(w)) * scale


def plan(chosen, experts):
    """(offsets, order, place) by going through the slots."""
    t, top = chosen.shape
    lists = [[] for _ in range(experts)]
    for s, e in enumerate(chosen.flatten().tolist()):
        if 0 <= e < experts:
            lists[e].append(s)
    offsets, order = [0], []
    for l in lists:
        order += l
        offsets.append(len(order))
    place = [-1] * (t * top)
    for at, s in enumerate(order):
        place[s] = at
    order += [-1] * (t * top - len(order))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(order), i32(place).view(t, top)


# -------------------------------------------------------------------- experts

def rows16(size):
    """The rounding of a slot's row: half a step of fp16, or of fp16's smallest
    at the scale of the row's largest (2^-25 in 2^14)."""
    return HALF_F16 * size + 2.0 ** -38 * size.amax(1, keepdim=True)


def moe(x, wg, wu, wd, chosen, share, kind, dy=None):
    """y and, with dy, (dx, dw_gate, dw_up, dw_down, dshare) of float64 inputs,
    each as (value, bound)."""
    t, d = x.shape
    e, f, _ = wg.shape
    zero = lambda v: torch.zeros_like(v)  # noqa: E731
    y, ye, dx, dxe = (zero(x) for _ in range(4))
    dwg, dwge, dwu, dwue = (zero(wg) for _ in range(4))
    dwd, dwde = zero(wd), zero(wd)
    ds, dse = zero(share), zero(share)
    for i in range(e):
        row, j = torch.nonzero(chosen == i, as_tuple=True)
        if not len(row):
            continue
        X, G, U, W, p = x[row], wg[i], wu[i], wd[i], share[row, j].unsqueeze(1)
        s = 1.01 * HALF_F32
        g, u = X @ G.t(), X @ U.t()
        ge, ue = d * s * (X.abs() @ G.abs().t()), d * s * (X.abs() @ U.abs().t())
        a, da = act(g, kind)
        h = a * u
        # before it is rounded (act and its derivative are Lipschitz with constants below 1.13 and 1.2)
        he = 1.13 * ge * (u.abs() + ue) + a.abs() * ue + FAST * (a.abs() + g.abs() * 2.0 ** -4) * u.abs()
        hr = HALF_BF16 * (h.abs() + he) + he
        rows = h @ W.t()
        re = hr @ W.abs().t() + f * s * ((h.abs() + hr) @ W.abs().t())
        re = re + rows16(rows.abs() + re)
        y.index_add_(0, row, p * rows)
        ye.index_add_(0, row, p.abs() * (re + 40 * HALF_F32 * (rows.abs() + re)))
        if dy is None:
            continue
        D = dy[row]
        dh = D @ W
        dhe = d * s * (D.abs() @ W.abs())
        ds[row, j] = (dh * h).sum(1)
        dse[row, j] = (dhe * (h.abs() + he) + dh.abs() * he).sum(1) + f * s * (dh.abs() * h.abs()).sum(1)
        ph = p * h
        phe = HALF_BF16 * ph.abs() + 1.01 * p.abs() * he + 2 * HALF_F32 * ph.abs()
        dwd[i], dwde[i] = D.t() @ ph, D.abs().t() @ phe + len(row) * s * (D.abs().t() @ (ph.abs() + phe))
        du, dg = p * dh * a, p * dh * u * da
        due = HALF_BF16 * du.abs() + 1.01 * p.abs() * (dhe * a.abs() + (dh.abs() + dhe) * (
            1.13 * ge + FAST * (a.abs() + g.abs() * 2.0 ** -4)))
        dge = HALF_BF16 * dg.abs() + 1.01 * p.abs() * (dhe * u.abs() * da.abs() + (dh.abs() + dhe) * (
            ue * da.abs() + (u.abs() + ue) * 1.2 * ge + FAST * u.abs() * (da.abs() + 1)))
        back = dg @ G + du @ U
        be = dge @ G.abs() + due @ U.abs() + 2 * f * s * ((dg.abs() + dge) @ G.abs() + (du.abs() + due) @ U.abs())
        be = be + rows16(back.abs() + be)
        dx.index_add_(0, row, back)
        dxe.index_add_(0, row, be + 40 * HALF_F32 * (back.abs() + be))
        for v, ve, out, oute in ((dg, dge, dwg, dwge), (du, due, dwu, dwue)):
            out[i], oute[i] = v.t() @ X, ve.t() @ X.abs() + len(row) * s * ((v.abs() + ve).t() @ X.abs())
    final = lambda v, e: (v, HALF_BF16 * (v.abs() + e) + e + 1e-38)  # noqa: E731
    if dy is None:
        return final(y, ye)
    return final(y, ye), (final(dx, dxe), final(dwg, dwge), final(dwu, dwue), final(dwd, dwde), (ds, dse + 1e-38))
