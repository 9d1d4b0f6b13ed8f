"""A decoder layer's operators at the ends of what their documentation allows:
no tokens, sizes whose offsets pass 32 bits, masked experts with NaN, two calls
at once, offsets that are no routing's at the most slots there may be."""
import math

import pytest
import torch

import layer_reference as ref
import sharded_optimizer_step_adamw_amd as z
from train_reference import inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


@pytest.mark.parametrize("style", ["half", "pairs"])
def test_no_tokens(style):
    q, k, w, cs = randn(0, 4, 64, seed=1), randn(0, 2, 64, seed=2), randn(64, seed=3), z.rope_table(8, 64)
    yq, yk = z.qk_norm_rope(q, k, cs, None, w, w, style=style)
    assert yq.shape == q.shape and yk.shape == k.shape
    dw = [torch.full((64,), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    got = z.qk_norm_rope_backward(q, k, q, k, cs, None, w, w, style=style, dw_q=dw[0], dw_k=dw[1])
    assert got[0].shape == q.shape and got[1].shape == k.shape
    assert not dw[0].any() and not dw[1].any()
    assert z.rope_table(0, 64).shape == (0, 32, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 2])
def test_a_masked_expert_is_not_there_whatever_its_logit(score, groups):
    """... nor with a bias of -inf, where its logit is NaN (the logistic's; a softmax is NaN whole)."""
    x = torch.zeros((4, 6), device=DEV)
    x[:, 0], x[:, 1] = 1.0, -math.inf
    x[1, 4] = math.inf if score == "sigmoid" else 3.0
    x[2:, 4] = math.nan if score == "sigmoid" else 50.0
    bias = torch.tensor([0.0, 5.0, 0.0, 0.0, -math.inf, 0.0], device=DEV)
    r = z.moe_route(x, 6, score=score, bias=bias, groups=groups, top_groups=groups)
    assert r.experts.tolist() == [[0, 2, 3, 5, -1, -1]] * 4
    assert r.offsets.tolist() == [0, 4, 4, 8, 12, 12, 16]
    assert torch.isfinite(r.weights).all() and not r.weights[:, 4:].any()


def test_logits_past_32_bits():
    """Rows of logits more than 2^32 bytes apart."""
    t, experts, top, gap = 4, 24, 3, (1 << 30) + 64
    flat = torch.zeros(3 * gap + experts, device=DEV)
    x = flat.as_strided((t, experts), (gap, 1))
    src = randn(t, experts, seed=4, dtype=torch.float32)
    x.copy_(src)
    dw = randn(t, top, seed=5, dtype=torch.float32)
    for kw in (dict(), dict(score="sigmoid", bias=0.1 * src[0], groups=4, top_groups=2)):
        want, got = z.moe_route(src, top, **kw), z.moe_route(x, top, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        score = kw.get("score", "softmax")
        grad = z.moe_route_backward(dw, src, want, score=score, renormalise=False)
        assert torch.equal(z.moe_route_backward(dw, x, got, score=score, renormalise=False), grad)
    z.moe_route_backward(dw, src, want, score=score, renormalise=False, out=x)
    assert torch.equal(x, grad) and not flat[experts:gap].any()


def test_slots_past_32_bits():
    """2^20 tokens, whose rows of h, dg and du are 4.8 GB each: every result of
    four stretches, and the weights' gradients whole."""
    t, d, f, e = 1 << 20, 16, 2304, 3
    x, dy = randn(t, d, seed=6), randn(t, d, seed=7)
    wg, wu, wd = (randn(e, a, b, seed=8 + i) / b ** 0.5 for i, (a, b) in enumerate(((f, d), (f, d), (d, f))))
    chosen = torch.randint(0, e, (t, 1), generator=torch.Generator().manual_seed(11)).to(torch.int32).to(DEV)
    share = randn(t, 1, seed=12, dtype=torch.float32)
    route = z.moe_plan(chosen, share, e)
    y, grads = z.moe_forward(x, wg, wu, wd, route), z.moe_backward(dy, x, wg, wu, wd, route)
    step, sums = 1 << 16, [[0.0, 0.0] for _ in range(3)]
    wide = [w.double() for w in (wg, wu, wd)]
    for k in range(0, t, step):
        at = slice(k, k + step)
        (ry, ey), back = ref.moe(x[at].double(), *wide, chosen[at], share[at].double(), "silu", dy[at].double())
        if k // step in (0, 5, 10, 15):
            inside(y[at], ry, ey, f"rows {k} y")
            inside(grads[0][at], *back[0], f"rows {k} dx")
            inside(grads[4][at], *back[4], f"rows {k} dweights")
        for s, v in zip(sums, back[1:4]):
            s[0], s[1] = s[0] + v[0], s[1] + v[1]
        del ry, ey, back
    for name, got, (want, bound) in zip(("dw_gate", "dw_up", "dw_down"), grads[1:4], sums):
        # (each stretch's bound counts its own terms; a sum over all adds the others' half steps)
        inside(got, want, bound * (t // step), name)


def test_two_calls_at_once():
    def layer(seed, t, experts):
        q, k, w = randn(t, 6, 64, seed=seed), randn(t, 2, 64, seed=seed + 1), randn(64, seed=seed + 2)
        x, cs = randn(t, experts, seed=seed + 3, dtype=torch.float32), z.rope_table(t, 64)
        dw = randn(t, 4, seed=seed + 4, dtype=torch.float32)

        def run():
            r = z.moe_route(x, 4, score="sigmoid", bias=x[0], groups=2, top_groups=1)
            return (*z.qk_norm_rope(q, k, cs, None, w, w), *z.qk_norm_rope_backward(q, k, q, k, cs, None, w, w), *r,
                    z.moe_route_backward(dw, x, r, score="sigmoid"), *z.moe_plan(r.experts, r.weights, experts))
        return run

    calls = [layer(20, 3000, 64), layer(30, 1111, 200)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in calls], []
    for _ in range(3):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(c())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_offsets_that_are_none_over_the_most_slots():
    """2^30 slots, every second expert with all of them: counts past 32 bits."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 180 GiB")
    t, top, e, d = 1 << 25, 32, 1024, 8
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[1::2] = t * top
    none = torch.zeros((t, top), dtype=torch.int32, device=DEV)
    route = z.Route(none, none.view(torch.float32), offsets, none.view(-1), none)
    x, w = randn(t, d, seed=40), [randn(e, d, d, seed=41 + k) for k in range(3)]
    y = z.moe_forward(x, *w, route)
    assert y.shape == (t, d)
    grads = z.moe_backward(x, x, *w, route)
    torch.cuda.synchronize()
    assert grads[0].shape == (t, d) and torch.equal(offsets[1::2], torch.full_like(offsets[1::2], t * top))
    del y, grads, none, route, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("e", [63, 64, 65])
def test_experts_around_a_wave(e):
    """Up to 64 the forward products find each expert's rows themselves, beyond by a list: the same results."""
    t, top, d, f = 500, 4, 72, 96
    x, dy = randn(t, d, seed=50), randn(t, d, seed=51)
    wg, wu, wd = randn(e, f, d, seed=52), randn(e, f, d, seed=53), randn(e, d, f, seed=54)
    g = torch.Generator().manual_seed(e)
    chosen = (torch.rand((t, top), generator=g) ** 3 * (e + 2)).to(torch.int32) - 1  # (some none, most the first ones)
    chosen[chosen == 5] = -1  # one without tokens
    share = torch.rand((t, top), generator=g).to(DEV)
    route = z.moe_plan(chosen.to(DEV), share, e)
    y, grads = z.moe_forward(x, wg, wu, wd, route), z.moe_backward(dy, x, wg, wu, wd, route)
    at = torch.where((chosen >= 0) & (chosen < e), chosen, -1).to(DEV)
    (ry, ey), back = ref.moe(x.double(), wg.double(), wu.double(), wd.double(), at, share.double(), "silu", dy.double())
    inside(y, ry, ey, "y")
    for name, got, (want, bound) in zip(("dx", "dw_gate", "dw_up", "dw_down", "dweights"), grads, back):
        inside(got, want, bound, name)
