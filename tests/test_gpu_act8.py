"""8-bit activation checkpoints against the format's definition in 64 bits:
the codes and scale bytes are equal, reading back is exact, the weight
gradient lies within its roundings."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
from train_reference import HALF_BF16, HALF_E4M3, HALF_F32, act8_bytes, inside

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def special(rows, cols, seed):
    """Values over bf16's whole range, with blocks of zeros, of one value, of
    values at the border of a power of two, subnormal and not finite."""
    x = bf16((rows, cols), seed).float()
    x *= 2.0 ** torch.randint(-40, 41, (rows, 1), generator=torch.Generator().manual_seed(seed + 1)).float()
    flat = x.view(-1)
    for k, v in enumerate([0.0, -0.0, 448.0, 450.0, 447.0, 1.75 * 2.0 ** 100, 2.0 ** 127, 3.38e38, 2.0 ** -126,
                           2.0 ** -130, 2.0 ** -133, float("inf"), float("-inf"), float("nan")]):
        flat[(k * 37) % flat.numel()] = v
    if rows > 2:
        x[1] = 0.0
        x[2, : min(cols, 40)] = 2.0 ** -133
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 100), (33, 255), (4, 1000),
                                       (129, 96), (1000, 40)])
@pytest.mark.parametrize("kind", ["normal", "special"])
def test_pack_and_unpack_match_the_definition(rows, cols, kind):
    x = bf16((rows, cols), rows * 1000 + cols) if kind == "normal" else special(rows, cols, rows + cols)
    want, byte = act8_bytes(x.double())
    a = z.act8_pack(x.to(DEV))
    assert a.q.dtype == torch.float8_e4m3fn and tuple(a.scale.shape) == (rows, -(-cols // 32))
    assert torch.equal(a.scale.cpu().long(), byte)
    got = z.act8_unpack(a).cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    # what the format promises of a finite block
    fine = torch.isfinite(x.double()) & ~torch.isnan(want)
    step = (2.0 ** (byte.double() - 127 - 10)).repeat_interleave(32, 1)[:, :cols]
    off = (want - x.double()).abs()
    assert bool((off <= torch.maximum(HALF_E4M3 * x.double().abs(), step))[fine].all())


def test_strided_and_unaligned_views():
    base = bf16((40, 100), 5).to(DEV)
    for view in (base[:, :64], base[3:, 1:66], base[::2, 8:40], base[:1, 7:8]):
        want, byte = act8_bytes(view.cpu().double())
        a = z.act8_pack(view)
        assert torch.equal(a.scale.cpu().long(), byte)
        out = torch.full((view.shape[0] + 1, view.shape[1] + 3), 9.0, dtype=torch.bfloat16, device=DEV)
        z.act8_unpack(a, out=out[:-1, 1:-2])
        assert torch.equal(out[:-1, 1:-2].cpu().double(), want)
        assert bool((out[-1] == 9).all() and (out[:, 0] == 9).all() and (out[:, -2:] == 9).all())


def test_no_rows():
    a = z.act8_pack(torch.empty((0, 40), dtype=torch.bfloat16, device=DEV))
    assert tuple(a.q.shape) == (0, 40) and tuple(a.scale.shape) == (0, 2)
    assert tuple(z.act8_unpack(a).shape) == (0, 40)
    dw = z.act8_wgrad(torch.empty((0, 24), dtype=torch.bfloat16, device=DEV), a)
    assert tuple(dw.shape) == (24, 40) and not bool(dw.any())


@pytest.mark.parametrize("t,n,d", [(1, 1, 1), (1, 8, 8), (5, 16, 33), (31, 64, 64), (32, 65, 127), (33, 128, 128),
                                   (64, 129, 255), (127, 300, 40), (300, 77, 500), (2050, 96, 64), (1000, 256, 264),
                                   (513, 520, 776)])
def test_wgrad(t, n, d):
    dy, x = bf16((t, n), t + n, 1e-3), bf16((t, d), t + d)
    a = z.act8_pack(x.to(DEV))
    values = z.act8_unpack(a).cpu().double()
    got = z.act8_wgrad(dy.to(DEV), a).cpu()
    ref = dy.double().t() @ values
    terms = dy.double().abs().t() @ values.abs()
    inside(got, ref, HALF_BF16 * ref.abs() + 1.01 * t * HALF_F32 * terms, f"dw {t} {n} {d}")


def test_wgrad_strided_views_and_neighbours():
    dy = bf16((200, 90), 1).to(DEV)[::2, 5:71]
    x = bf16((100, 50), 2)
    a = z.act8_pack(x.to(DEV))
    flat = torch.full((66 * 50 + 7,), 5.0, dtype=torch.bfloat16, device=DEV)
    out = flat[3:3 + 66 * 50].view(66, 50)  # a place in a flat gradient vector, at an odd offset
    assert z.act8_wgrad(dy, a, out=out) is out
    v = z.act8_unpack(a).cpu().double()
    ref = dy.cpu().double().t() @ v
    inside(out.cpu(), ref, HALF_BF16 * ref.abs() + 1.01 * 100 * HALF_F32 * (dy.cpu().double().abs().t() @ v.abs()),
           "dw")
    assert bool((flat[:3] == 5).all() and (flat[3 + 66 * 50:] == 5).all())


def test_wgrad_is_linear_in_dy():
    """Differences: the gradient of <dw, c> with respect to dy is x^ c^T."""
    t, n, d = 48, 24, 40
    a = z.act8_pack(bf16((t, d), 3).to(DEV))
    v = z.act8_unpack(a).cpu().double()
    dy = torch.zeros((t, n), dtype=torch.bfloat16, device=DEV)
    dy[7, 5] = 1.0
    got = z.act8_wgrad(dy, a).cpu().double()
    assert torch.equal(got[5], v[7]) and not bool(got[:5].any()) and not bool(got[6:].any())


def test_another_stream():
    x = bf16((500, 320), 8).to(DEV)
    dy = bf16((500, 64), 9).to(DEV)
    want = z.act8_wgrad(dy, z.act8_pack(x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = z.act8_pack(x, stream=s)
    got = z.act8_wgrad(dy, a, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
