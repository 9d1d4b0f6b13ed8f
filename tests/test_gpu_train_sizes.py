"""The gradient operators at sizes that take the larger tiles, split and
leftover reductions, several pieces and long strides, and at drawn sizes,
against 64-bit references on the GPU with the bounds of the small tests."""
import random

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
import test_gpu_glu as tg
import test_gpu_xent as tx
from train_reference import HALF_BF16, HALF_F32, inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def run_xent(t, d, v, seed, mean=True, scale=0.5):
    x, w, y = (a.to(DEV) for a in tx.inputs(t, d, v, seed, ignored=0.2, lean=12.0))
    got = z.linear_xent_grad(x, w, y, mean=mean, grad_scale=scale)
    tx.check(x, w, y, mean, scale, got, f"{t}x{d}x{v}")
    loss, row = z.linear_xent_loss(x, w, y, mean=mean)
    assert torch.equal(loss, got[0]) and torch.equal(row, got[1])


def run_glu(t, d, f, seed, kind):
    x, wg, wu, dh = (a.to(DEV) for a in tg.inputs(t, d, f, seed))
    g, u, ge, ue = tg.products(x, wg, wu)
    h, (cg, cu) = z.glu_forward(x, wg, wu, act=kind, checkpoint=True)
    tg.check_h(h, g, u, ge, ue, kind, f"{t}x{d}x{f} h")
    assert torch.equal(h, z.glu_forward(x, wg, wu, act=kind))
    got = z.glu_backward(dh, x, wg, wu, act=kind)
    tg.check_back(got, dh, x.double(), g, u, ge, ue, wg, wu, kind, f"{t}x{d}x{f}")
    xc = z.act8_pack(x)
    kg, ku = z.act8_unpack(cg).double(), z.act8_unpack(cu).double()
    zero = torch.zeros_like(kg)
    got = z.glu_backward(dh, xc, wg, wu, act=kind, checkpoint=(cg, cu))
    tg.check_back(got, dh, z.act8_unpack(xc).double(), kg, ku, zero, zero, wg, wu, kind, f"{t}x{d}x{f} act8")


def run_wgrad(t, n, d, seed):
    g = torch.Generator().manual_seed(seed)
    dy = (torch.randn((t, n), generator=g) * 1e-3).to(torch.bfloat16).to(DEV)
    a = z.act8_pack(torch.randn((t, d), generator=g).to(torch.bfloat16).to(DEV))
    values = z.act8_unpack(a).double()
    ref = dy.double().t() @ values
    terms = dy.double().abs().t() @ values.abs()
    inside(z.act8_wgrad(dy, a), ref, HALF_BF16 * ref.abs() + 1.01 * t * HALF_F32 * terms, f"dw {t} {n} {d}")


# 256 x 256, 256 x 128, 128 x 128 and 64 x 64 tiles; whole, split, and split only where tiles are left over
@pytest.mark.parametrize("t,d,v", [(2560, 712, 33000), (3000, 1000, 20000), (2100, 136, 8200), (1000, 520, 6000),
                                   (100, 2000, 3000), (8, 4096, 500), (4200, 72, 16500)])
def test_xent(t, d, v):
    run_xent(t, d, v, t + v)


@pytest.mark.parametrize("t,d,f", [(3000, 2000, 4300), (4100, 136, 5000), (1000, 520, 1500), (40, 4000, 200),
                                   (9000, 64, 300)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_glu(t, d, f, kind):
    run_glu(t, d, f, t + f, kind)


@pytest.mark.parametrize("t,n,d", [(4000, 520, 776), (1030, 2056, 2600), (300, 4200, 4100), (1500, 33000, 700),
                                   (2050, 5000, 3100)])
def test_wgrad(t, n, d):
    run_wgrad(t, n, d, t + n)


@pytest.mark.parametrize("seed", range(6))
def test_drawn_sizes(seed):
    r = random.Random(seed)
    size = lambda lo, hi: int(round(lo * (hi / lo) ** r.random()))  # noqa: E731
    run_xent(size(1, 3000), size(1, 1200), size(2, 12000), seed, mean=r.random() < 0.5)
    run_glu(size(1, 3000), size(1, 1200), size(1, 3000), seed, r.choice(["silu", "gelu"]))
    run_wgrad(size(1, 5000), size(1, 2000), size(1, 2000), seed)


def test_offsets_past_32_bits():
    """A vocabulary projection of more than 2^32 bytes whose last rows matter,
    rows far apart in x, and exponentials of more than 2^31 bytes."""
    t, d, v = 300, 1100, 2_000_000
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.zeros((v, d), dtype=torch.bfloat16, device=DEV)
    w[-700:] = (torch.randn((700, d), generator=g, device=DEV) / 32).to(torch.bfloat16)
    wide = torch.empty((t, 4_000_000), dtype=torch.bfloat16, device=DEV)  # 2.4 GB: rows 8 MB apart
    x = wide[:, 3_998_000:3_998_000 + d]
    x.copy_(torch.randn((t, d), generator=g, device=DEV).to(torch.bfloat16) * 4)
    y = torch.randint(v - 700, v, (t,), generator=g, device=DEV)
    loss, row, dx, dw = z.linear_xent_grad(x, w, y, mean=False)
    zz = x.double() @ w[-700:].double().t()  # every other logit is 0
    rest = float(v - 700)
    top = zz.amax(1, keepdim=True).clamp(min=0)
    total = torch.exp(zz - top).sum(1, keepdim=True) + rest * torch.exp(-top)
    p = torch.exp(zz - top) / total
    lse = (top + torch.log(total))[:, 0]
    own = zz.gather(1, (y - (v - 700)).unsqueeze(1))[:, 0]
    size = (x.double().abs() @ w[-700:].double().abs().t()).amax(1)
    inside(row, lse - own, 2.02 * d * HALF_F32 * size + 2.0 ** -20 * (lse + 1), "row_loss")
    onehot = torch.zeros_like(p)
    onehot.scatter_(1, (y - (v - 700)).unsqueeze(1), 1.0)
    m = p - onehot
    X = x.double()
    # P is bf16 of values off by 2^-11 and the logits' errors; 300 rows are summed
    bound = (2.02 * HALF_BF16 + 2.0 ** -10) * (m.abs().t() @ X.abs()) + 2.0 ** -24 * X.abs().sum(0)
    ref = m.t() @ X
    inside(dw[-700:], ref, HALF_BF16 * ref.abs() + bound, "dw, last rows")
    each = (rest and torch.exp(-top) / total)  # the probability of any other word
    ref = (each.t() @ X)[0]
    bound = (2.02 * HALF_BF16 + 2.0 ** -10) * (each.t() @ X.abs())[0] + 2.0 ** -24 * X.abs().sum(0)
    for r in (0, 1, 1_000_003, v - 701):
        inside(dw[r], ref, HALF_BF16 * ref.abs() + bound, f"dw, row {r}")
    assert bool(torch.isfinite(dx.float()).all())
