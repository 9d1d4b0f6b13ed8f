"""Rows far apart and matrices of gigabytes: operands read in place with row
strides up to the longest, outputs with rows past 2^32 bytes, a vocabulary
projection of more than 2^32 bytes, 8-bit checkpoints past 2^27 values.

What lies between the rows of a wide operand is NaN, so that a read beside a
row shows; the reference is the same call on the operand's contiguous copy
(which the small tests hold to 64 bits), and equality, since sizes alone
decide how a product is divided."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
import test_gpu_glu as tg
import test_gpu_xent as tx
from forced_plan import TILES, forced
from train_reference import HALF_BF16, HALF_F16, HALF_F32, act8_bytes, inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
LONGEST = (1 << 22) - 8  # elements: the longest stride that is read in place
tiles = pytest.mark.parametrize("tile", TILES)


def wide(a, ld, at=0):
    """a as columns [at, at + cols) of a matrix of NaN with rows of ld."""
    rows, cols = a.shape
    buf = torch.full((rows * ld,), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = buf.as_strided((rows, cols), (ld, 1), at)
    v.copy_(a)
    return v


@pytest.fixture(autouse=True)
def gigabytes_are_returned():
    yield
    torch.cuda.empty_cache()


@tiles
@pytest.mark.parametrize("ld", [LONGEST, LONGEST + 8])
def test_xent_rows_far_apart(tile, ld):
    x, w, y = (a.to(DEV) for a in tx.inputs(300, 72, 280, 1, ignored=0.1))
    with forced(tile):
        want = z.linear_xent_grad(x, w, y)
        xw = wide(x, ld, ld - 72)
        got = z.linear_xent_grad(xw, w, y, want_dw=False)
        assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))
        assert torch.equal(z.linear_xent_grad(xw, w, y)[3], want[3])
        del xw
        ww = wide(w, ld, 8)
        got = z.linear_xent_grad(x, ww, y)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    tx.check(x, w, y, True, 1.0, want, f"tile {tile}")


@tiles
@pytest.mark.parametrize("ld", [LONGEST, LONGEST + 8])
def test_glu_rows_far_apart(tile, ld):
    x, wg, wu, dh = (a.to(DEV) for a in tg.inputs(300, 72, 280, 2))
    with forced(tile):
        h = z.glu_forward(x, wg, wu)
        want = z.glu_backward(dh, x, wg, wu)
        xw, gw, uw = wide(x, ld, ld - 72), wide(wg, ld, 16), wide(wu, ld, ld - 72)
        assert torch.equal(z.glu_forward(xw, gw, uw), h)
        got = z.glu_backward(wide(dh, ld, 3), xw, gw, uw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g, u, ge, ue = tg.products(x, wg, wu)
    tg.check_back(want, dh, x.double(), g, u, ge, ue, wg, wu, "silu", f"tile {tile}")


@tiles
@pytest.mark.parametrize("ld", [LONGEST, LONGEST + 8])
def test_wgrad_rows_far_apart(tile, ld):
    g = torch.Generator().manual_seed(3)
    dy = torch.randn((300, 280), generator=g).to(torch.bfloat16).to(DEV)
    a = z.act8_pack(torch.randn((300, 72), generator=g).to(torch.bfloat16).to(DEV))
    with forced(tile):
        assert torch.equal(z.act8_wgrad(wide(dy, ld, 8), a), z.act8_wgrad(dy, a))


@tiles
def test_outputs_with_rows_far_apart(tile):
    """Row strides of 2^23 + 3 elements: 280 rows span 4.7e9 bytes."""
    ld = (1 << 23) + 3
    x, w, y = (a.to(DEV) for a in tx.inputs(280, 40, 270, 4))
    dh = torch.randn((280, 270), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)

    def out(rows, cols):
        buf = torch.full((rows * ld,), 5.0, dtype=torch.bfloat16, device=DEV)
        return buf, buf.as_strided((rows, cols), (ld, 1), 2)

    def same(pair, want):
        buf, v = pair
        assert torch.equal(v, want)
        beside = buf.as_strided((v.shape[0], 2), (ld, 1), 0), buf.as_strided((v.shape[0] - 1, 2), (ld, 1), 2 + v.shape[1])
        assert all(bool((b == 5).all()) for b in beside)

    with forced(tile):
        want = z.linear_xent_grad(x, w, y)
        dx, dw = out(280, 40), out(270, 40)
        z.linear_xent_grad(x, w, y, dx=dx[1], dw=dw[1])
        same(dx, want[2])
        same(dw, want[3])
        h, hb = out(280, 270), out(280, 270)
        z.glu_forward(x, w, w, out=h[1])
        same(h, z.glu_forward(x, w, w))
        want = z.glu_backward(dh, x, w, w)
        z.glu_backward(dh, x, w, w, dx=dx[1], dw_gate=dw[1], h=hb[1])
        same(dx, want[0])
        same(dw, want[1])
        assert torch.equal(hb[1], h[1])


def test_projection_past_32_bits():
    """w of 4.4e9 bytes, read in place along and across its rows, whose last
    700 rows alone are not zero."""
    t, d, v, n = 300, 1104, 2_000_000, 700
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.zeros((v, d), dtype=torch.bfloat16, device=DEV)
    w[-n:] = (torch.randn((n, d), generator=g, device=DEV) / 32).to(torch.bfloat16)
    x = (torch.randn((t, d), generator=g, device=DEV) * 4).to(torch.bfloat16)
    y = torch.randint(v - n, v, (t,), generator=g, device=DEV)
    _, row, dx, _ = z.linear_xent_grad(x, w, y, mean=False, want_dw=False)
    X, W = x.double(), w[-n:].double()
    zz = X @ W.t()  # every other logit is 0
    total = torch.exp(zz).sum(1, keepdim=True) + float(v - n)  # (logits below 40: nothing overflows)
    at = (y - (v - n)).unsqueeze(1)
    want = torch.log(total[:, 0]) - zz.gather(1, at)[:, 0]
    size = (X.abs() @ W.abs().t()).amax(1)
    rbound = 2.02 * d * HALF_F32 * size + 2.0 ** -21 * (zz.abs().amax(1) + 16)
    inside(row, want, rbound, "row_loss")
    q = torch.exp(zz) / total
    p = q.scatter_add(1, at, torch.full_like(at, -1.0, dtype=q.dtype))
    ref = p @ W
    # P is bf16 of values off by e's 11 bits and the logits' errors; of a row's sum only n terms are not 0
    perr = 1.01 * HALF_BF16 * p.abs() + (1.01 * HALF_F16 + 2 * rbound[:, None]) * q + 2.0 ** -25
    inside(dx, ref, HALF_BF16 * ref.abs() + 1.01 * (perr @ W.abs() + 1.01 * n * HALF_F32 * (p.abs() @ W.abs())), "dx")


def test_checkpoints_of_large_matrices():
    """Above 2^27 bytes the 16-bit side goes past the caches: the same codes as
    in slabs below, contiguous, strided and at odd addresses, and read back."""
    rows, cols = 9001, 8195
    g = torch.Generator(device=DEV).manual_seed(6)
    base = torch.randn((rows, cols + 6), generator=g, device=DEV)
    base *= 2.0 ** torch.randint(-30, 31, (rows, 1), generator=g, device=DEV).float()
    base = base.to(torch.bfloat16)
    base[5000, 77] = float("nan")
    for x in (base[:, :cols].contiguous(), base[:, 3:3 + cols], base[:, 1:1 + 8192], base[:, :8192].contiguous()):
        assert x.numel() * 2 > 1 << 27
        a = z.act8_pack(x)
        out = torch.full((rows, x.shape[1] + 5), 5.0, dtype=torch.bfloat16, device=DEV)
        back = z.act8_unpack(a, out=out[:, 3:3 + x.shape[1]])
        for r in range(0, rows, 1000):
            s = z.act8_pack(x[r:r + 1000])
            assert torch.equal(a.q[r:r + 1000].view(torch.uint8), s.q.view(torch.uint8))
            assert torch.equal(a.scale[r:r + 1000], s.scale)
            assert torch.equal(back[r:r + 1000].view(torch.int16), z.act8_unpack(s).view(torch.int16))
        assert bool((out[:, :3] == 5).all() and (out[:, 3 + x.shape[1]:] == 5).all())
        for r in (0, 4999, rows - 1):
            want, byte = act8_bytes(x[r:r + 1].cpu().double())
            assert torch.equal(a.scale[r].cpu().long(), byte[0]) and torch.equal(back[r].cpu().double(), want[0])
