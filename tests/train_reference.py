"""Plain 64-bit references of the gradient operators for the tests, and the
error bounds that follow from the roundings each operator makes.

HALF: half a step of each type relative to the value.  A product of K terms
accumulated in fp32 is off by at most K 2^-24 of the sum of its terms'
magnitudes; the matrix cores add in an order of their own, so no less is
assumed."""
import math

import torch

HALF_BF16, HALF_F16, HALF_F32, HALF_E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24, 2.0 ** -4


def act(g, kind):
    """The activation and its derivative, in g's type."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t * t) * k * (1 + 0.134145 * g * g)


def act8_bytes(x):
    """(values the checkpoint of x stands for, float64; scale bytes) of a
    float64 matrix on the CPU, straight from the format's definition: the
    nearest of all 8-bit codes, ties to the even code."""
    codes = torch.arange(0, 0x7F, dtype=torch.int32)  # 0 .. 448 in order; 0x7F is NaN
    e, m = (codes >> 3).double(), (codes & 7).double()
    grid = torch.where(codes >> 3 > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
    rows, cols = x.shape
    blocks = -(-cols // 32)
    out = torch.zeros(rows, blocks * 32, dtype=torch.float64)
    out[:, :cols] = x
    out = out.view(rows, blocks, 32)
    big = out.abs().amax(2)
    byte = torch.full((rows, blocks), 3, dtype=torch.int64)
    for b in range(4, 255):  # the smallest byte whose scale suffices
        byte[big > 448.0 * 2.0 ** (b - 1 - 127)] = b
    scale = 2.0 ** (byte.double() - 127)
    v = out / scale.unsqueeze(2)
    hi = torch.searchsorted(grid, v.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - v.abs(), v.abs() - grid[lo]
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    # at scale 2^120 the codes end at 240: 256 would stand for 2^128, beyond bf16
    pick = torch.where(byte.unsqueeze(2) == 247, pick.clamp(max=int((grid <= 240).sum()) - 1), pick)
    q = torch.sign(v) * grid[pick] * scale.unsqueeze(2)
    bad = ~torch.isfinite(out).all(2)
    q[bad] = math.nan
    byte[bad] = 255
    return q.view(rows, blocks * 32)[:, :cols], byte


def xent(x, w, y, ignore, mean, grad_scale):
    """(loss, row losses, dx, dw, probabilities with the target's 1 taken off,
    factor) in float64."""
    z = x @ w.t()
    keep = y != ignore
    at = torch.where(keep, y, torch.zeros_like(y)).unsqueeze(1)
    lse = torch.logsumexp(z, 1)
    row = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    n = int(keep.sum())
    share = (1.0 / n if n else 0.0) if mean else 1.0
    p = torch.exp(z - lse.unsqueeze(1))
    p.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=p.dtype))
    p[~keep] = 0
    c = share * grad_scale
    return row.sum() * share, row, c * (p @ w), c * (p.t() @ x), p, c


def inside(got, ref, bound, what):
    """Every element of got within bound of ref."""
    err = (got.double() - ref).abs()
    over = err - bound
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    worst = float((err / bound.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"{what}: worst error {worst:.3f} of its bound", flush=True)
    assert not bool((over > 0).any()), f"{what}: {worst:.3f} of its bound"
