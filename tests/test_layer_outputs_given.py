"""An output that a call of the norms with rotation is given is written, or the call is refused."""
import math

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z
from test_layer_api import gpu

F32 = torch.float32


@pytest.mark.parametrize("kw", [dict(out_k=gpu(4, 2, 8))])
def test_forward_without_keys_refuses_their_output(kw):
    with pytest.raises(ValueError, match="given without k"):
        z.qk_norm_rope(gpu(4, 2, 8), None, gpu(4, 4, 2, dtype=F32), **kw)


@pytest.mark.parametrize("kw", [dict(dyk=gpu(4, 2, 8)), dict(dk=gpu(4, 2, 8)), dict(dw_k=gpu(8))])
def test_backward_without_keys_refuses_their_gradients(kw):
    args = dict(dyq=gpu(4, 2, 8), dyk=None, q=gpu(4, 2, 8), k=None, table=gpu(4, 4, 2, dtype=F32))
    with pytest.raises(ValueError, match="given without k"):
        z.qk_norm_rope_backward(**{**args, **kw})


@pytest.mark.gpu
def test_a_weights_gradient_that_is_given_is_written_without_weights():
    dev = torch.device("cuda:0")
    t, hq, hk, width = 70, 4, 2, 48
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(dev)  # noqa: E731
    q, k, dyq, dyk, cs = r(t, hq, width), r(t, hk, width), r(t, hq, width), r(t, hk, width), z.rope_table(t, 32)
    one = torch.ones(width, dtype=torch.bfloat16, device=dev)
    want = z.qk_norm_rope_backward(dyq, dyk, q, k, cs, None, one, one)
    for given in ((True, True), (True, False), (False, True)):
        dw = [torch.full((width,), math.nan, dtype=torch.bfloat16, device=dev) if g else None for g in given]
        got = z.qk_norm_rope_backward(dyq, dyk, q, k, cs, dw_q=dw[0], dw_k=dw[1])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for a, b, c in zip(got[2:], dw, want[2:]):
            assert a is b and (b is None or torch.equal(b, c))
    none = z.qk_norm_rope_backward(dyq, dyk, q, k, cs)
    assert none[2] is None and none[3] is None
