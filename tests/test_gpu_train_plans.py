"""Every kind of tile of the gradient operators' products, whole, split and
with both kinds in one launch, at odd sizes, against 64-bit references with the
bounds of the small tests; and the sums of dw over several pieces of rows."""
import math

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
import test_gpu_glu as tg
import test_gpu_xent as tx
from forced_plan import SPLITS, TILES, forced
from train_reference import HALF_BF16, HALF_F16, HALF_F32, inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
IGN = -100
kinds = pytest.mark.parametrize("tile", TILES)
splits = pytest.mark.parametrize("split", SPLITS, ids=["whole", "split", "both"])


# (every product: several tiles each way, ending inside one, and a reduction of an odd length)
@kinds
@splits
@pytest.mark.parametrize("t,d,v", [(301, 333, 779), (520, 264, 1288)])
def test_xent(tile, split, t, d, v):
    x, w, y = (a.to(DEV) for a in tx.inputs(t, d, v, t + d, ignored=0.2, lean=10.0))
    with forced(tile, *split):
        got = z.linear_xent_grad(x, w, y, grad_scale=0.5)
        tx.check(x, w, y, True, 0.5, got, f"tile {tile} {split} {t}x{d}x{v}")
        dx = z.linear_xent_grad(x, w, y, grad_scale=0.5, want_dw=False)[2]
        dw = z.linear_xent_grad(x, w, y, grad_scale=0.5, want_dx=False)[3]
        assert torch.equal(dx, got[2]) and torch.equal(dw, got[3])
        loss, row = z.linear_xent_loss(x, w, y)
        assert torch.equal(loss, got[0]) and torch.equal(row, got[1])


@kinds
@splits
@pytest.mark.parametrize("t,d,f,kind", [(301, 333, 779, "silu"), (520, 264, 520, "gelu")])
def test_glu(tile, split, t, d, f, kind):
    x, wg, wu, dh = (a.to(DEV) for a in tg.inputs(t, d, f, t + f))
    g, u, ge, ue = tg.products(x, wg, wu)
    what = f"tile {tile} {split} {t}x{d}x{f}"
    with forced(tile, *split):
        h, (cg, cu) = z.glu_forward(x, wg, wu, act=kind, checkpoint=True)
        assert torch.equal(h, z.glu_forward(x, wg, wu, act=kind))
        tg.check_h(h, g, u, ge, ue, kind, f"{what} h")
        hb = torch.empty_like(h)
        got = z.glu_backward(dh, x, wg, wu, act=kind, h=hb)
        assert torch.equal(h, hb)
        tg.check_back(got, dh, x.double(), g, u, ge, ue, wg, wu, kind, what)
        xc = z.act8_pack(x)
        kg, ku = z.act8_unpack(cg).double(), z.act8_unpack(cu).double()
        for name, k, ref, e in (("g", kg, g, ge), ("u", ku, u, ue)):
            # e4m3 within 2^-4, or 2^-10 of twice the scale: 448 2^(b - 127) is at most twice the block's largest
            big = torch.nn.functional.pad(ref.abs(), (0, -f % 32)).view(t, -1, 32).amax(2).repeat_interleave(32, 1)[:, :f]
            inside(k, ref, torch.maximum(2.0 ** -4 * ref.abs(), big * (2.0 ** -8 / 448)) + 1.07 * e, f"{what} {name}")
        zero = torch.zeros_like(kg)
        got = z.glu_backward(dh, xc, wg, wu, act=kind, checkpoint=(cg, cu))
        tg.check_back(got, dh, z.act8_unpack(xc).double(), kg, ku, zero, zero, wg, wu, kind, f"{what} act8")


@kinds
@splits
@pytest.mark.parametrize("t,n,d", [(333, 301, 779), (520, 1288, 264)])
def test_wgrad(tile, split, t, n, d):
    g = torch.Generator().manual_seed(t)
    dy = (torch.randn((t, n), generator=g) * 1e-3).to(torch.bfloat16).to(DEV)
    a = z.act8_pack(torch.randn((t, d), generator=g).to(torch.bfloat16).to(DEV))
    v = z.act8_unpack(a).double()
    with forced(tile, *split):
        got = z.act8_wgrad(dy, a)
    ref = dy.double().t() @ v
    inside(got, ref, HALF_BF16 * ref.abs() + 1.01 * t * HALF_F32 * (dy.double().abs().t() @ v.abs()), f"tile {tile} {split}")


@kinds
@splits
def test_targets_at_any_element(tile, split):
    """Next-token targets, tokens[1:]: 8 bytes past an address of 16."""
    x, w, y = (a.to(DEV) for a in tx.inputs(301, 72, 300, 5, ignored=0.1))
    tokens = torch.cat([y[:1], y])
    assert tokens[1:].data_ptr() % 16 == 8
    with forced(tile, *split):
        want = z.linear_xent_grad(x, w, y)
        got = z.linear_xent_grad(x, w, tokens[1:])
    tx.check(x, w, y, True, 1.0, want, "targets")
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ----------------------------------------------- dw over several pieces of rows

T, D, V = 3000, 33, 700_003  # 2^30 exponentials a piece: three of 1024, 1024 and 952 rows


@pytest.fixture(scope="module")
def pieces():
    """Inputs and the 64-bit reference with its bounds, by rows."""
    g = torch.Generator(device=DEV).manual_seed(2)
    w = (torch.randn((V, D), generator=g, device=DEV) / D ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    x = torch.randn((T, D), generator=g, device=DEV)
    r = w[y].float()
    x = (x + r * (16 * torch.rand((T, 1), generator=g, device=DEV) / r.square().sum(1, keepdim=True))).to(torch.bfloat16)
    y = torch.where(torch.rand((T,), generator=g, device=DEV) < 0.2, IGN, y)
    X, W = x.double(), w.double()
    scale = 0.5 / int((y != IGN).sum())
    row, rbound = torch.zeros(T, device=DEV).double(), torch.zeros(T, device=DEV).double()
    dx, dxb = torch.zeros_like(X), torch.zeros_like(X)
    dw, dwb = torch.zeros_like(W), torch.zeros_like(W)
    for a in range(0, T, 300):
        s = slice(a, a + 300)
        zz = X[s] @ W.t()
        # (as in the small tests: the logits' error, and the hardware's exponentials and logarithms)
        zerr = 1.01 * D * HALF_F32 * (X[s].abs() @ W.abs().t()).amax(1)
        keep = (y[s] != IGN).double()
        rb = (2 * zerr + 2.0 ** -21 * (zz.abs().amax(1) + math.log(V) + 1)) * keep
        lse = torch.logsumexp(zz, 1)
        at = y[s].clamp(min=0).unsqueeze(1)
        row[s] = (lse - zz.gather(1, at)[:, 0]) * keep
        rbound[s] = rb
        q = zz.sub_(lse[:, None]).exp_().mul_(keep[:, None])
        own = q.gather(1, at)
        # |P| and its error: bf16 of itself, e's 11 bits and the logits' error of the softmax, and below fp16's normals
        size = q.clone().scatter_(1, at, (keep[:, None] - own).abs())
        perr = 1.01 * HALF_BF16 * size + (1.01 * HALF_F16 + 2 * rb[:, None]) * q + 2.0 ** -25 * keep[:, None]
        p = q.scatter_add_(1, at, -keep[:, None])
        dx[s] = p @ W
        dxb[s] = perr @ W.abs() + 1.01 * V * HALF_F32 * (size @ W.abs())
        dw += p.t() @ X[s]
        dwb += perr.t() @ X[s].abs() + 1.01 * T * HALF_F32 * (size.t() @ X[s].abs())
    dx, dw = scale * dx, scale * dw
    return dict(x=x, w=w, y=y, row=row, rbound=rbound, loss=row.sum() * scale / 0.5, lbound=rbound.sum() * scale / 0.5,
                dx=dx, dxb=HALF_BF16 * dx.abs() + 1.01 * scale * dxb + 1e-38, dw=dw,
                dwb=HALF_BF16 * dw.abs() + 1.01 * scale * dwb + 1e-38)


@pytest.mark.parametrize("tile,split", [(0, (1, 0))] + [(k, s) for k in TILES for s in SPLITS])
def test_pieces(pieces, tile, split):
    p = pieces
    with forced(tile, *split):
        loss, row, dx, dw = z.linear_xent_grad(p["x"], p["w"], p["y"], grad_scale=0.5)
    inside(row, p["row"], p["rbound"], "row_loss")
    inside(loss[0], p["loss"], p["lbound"] + 4 * HALF_F32 * p["loss"], "loss")
    inside(dx, p["dx"], p["dxb"], "dx")
    inside(dw, p["dw"], p["dwb"], "dw")


def test_pieces_into_a_flat_gradient(pieces):
    """dw at an odd offset, the neighbours left alone; dw alone is the same."""
    p = pieces
    flat = torch.full((V * D + 9,), 5.0, dtype=torch.bfloat16, device=DEV)
    want = z.linear_xent_grad(p["x"], p["w"], p["y"])
    z.linear_xent_grad(p["x"], p["w"], p["y"], want_dx=False, dw=flat[5:5 + V * D].view(V, D))
    assert torch.equal(flat[5:5 + V * D].view(V, D), want[3])
    assert bool((flat[:5] == 5).all() and (flat[5 + V * D:] == 5).all())
