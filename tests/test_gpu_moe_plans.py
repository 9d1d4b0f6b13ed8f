"""Every kind of tile of the experts' products, the weight gradients whole and in
parts, at odd sizes, against 64-bit references with the bounds of the small
tests."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
import test_gpu_moe as tm
from forced_moe_plan import TILES, forced

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


# (several tiles each way, ending inside one, experts of some rows, of none and of most)
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("part", [0, 64, 192], ids=["own", "64", "192"])
@pytest.mark.parametrize("t,d,f,e,top,kind", [(611, 333, 301, 5, 2, "silu"), (530, 520, 264, 4, 3, "gelu")])
def test_tiles_and_parts(tile, part, t, d, f, e, top, kind):
    data = tm.inputs(t, d, f, e, top, t + tile, skew=2.0)
    data[5][data[5] == e - 1] = -1
    with forced(tile, part):
        y, grads = tm.check(*data, kind, f"tile {tile} part {part} {t}x{d}x{f}")
        assert not any(g[e - 1].any() for g in grads[1:4])
        D = [v.to(DEV) for v in data]
        r = z.moe_plan(D[5], D[6], e)
        again = z.moe_backward(D[1], D[0], *D[2:5], r, act=kind)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("tile", TILES)
def test_one_expert_in_many_parts(tile):
    data = tm.inputs(3000, 72, 40, 3, 1, tile, skew=0.0, none=0.0)
    data[5][:2500] = 1
    with forced(tile, 64):
        tm.check(*data, "silu", f"tile {tile}")


@pytest.mark.parametrize("tile", TILES)
def test_offsets_that_are_none_with_parts(tile):
    t, d, f, e, top = 200, 64, 48, 4, 2
    D = [v.to(DEV) for v in tm.inputs(t, d, f, e, top, 3)]
    with forced(tile, 64):
        good = z.moe_plan(D[5], D[6], e)
        n = t * top
        for offsets in ([0, n, 0, n, 0], [n, n, n, n, n], [0, 0, 0, 0, 1 << 30], [5, n, 7, n, n], [-9, 3, n + 9, 0, n]):
            r = good._replace(offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV))
            z.moe_forward(D[0], *D[2:5], r)
            z.moe_backward(D[1], D[0], *D[2:5], r)
            torch.cuda.synchronize()
        tm.check(*[v.cpu() for v in D], "silu", "after")
