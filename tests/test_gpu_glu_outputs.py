"""glu_backward with some of its outputs given: a weight gradient that is a
view with longer rows, the other one left to the call, on the current stream and
on another."""
import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("f", [1, 9])
@pytest.mark.parametrize("given", ["dw_gate", "dw_up"])
def test_one_weight_gradient_given_as_a_padded_view(given, f, other):
    g = torch.Generator(device=DEV).manual_seed(f)
    x, wg, wu, dh = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
                     for s in ((5, 12), (f, 12), (f, 12), (5, f)))
    want = z.glu_backward(dh, x, wg, wu)
    buf = torch.full((f, 31), 5.0, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream() if other else None
    got = z.glu_backward(dh, x, wg, wu, **{given: buf[:, 7:19]}, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert got[1 if given == "dw_gate" else 2].data_ptr() == buf[:, 7:].data_ptr()
    assert bool((buf[:, :7] == 5).all() and (buf[:, 19:] == 5).all())


def test_two_strides_are_refused():
    x, w, dh = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((5, 12), (9, 12), (5, 9)))
    buf = torch.zeros((9, 31), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="dw_up: row stride differs"):
        z.glu_backward(dh, x, w, w, dw_gate=buf[:, :12], dw_up=torch.zeros_like(w))
    with pytest.raises(TypeError, match="dw_gate: expected a tensor"):
        z.glu_backward(dh, x, w, w, dw_gate=3)
