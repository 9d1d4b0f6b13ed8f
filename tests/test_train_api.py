"""The C ABI and the Python checks of the gradient operators without a GPU:
every refusal comes before any HIP call."""
import ctypes

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

FAKE = 0x100000  # aligned to 256 bytes; never dereferenced: every call fails validation
BIG = 1 << 21


def call(fn, args, ws=FAKE, size=1 << 62):
    n = ctypes.c_size_t(size)
    return fn(*args, ws, ctypes.byref(n), None), n.value


XENT = dict(T=8, D=16, V=32, x=FAKE, ldx=16, w=FAKE, ldw=16, target=FAKE, ignore=-100, mean=1, grad_scale=1.0,
            loss=FAKE, row_loss=FAKE, dx=FAKE, lddx=16, dw=FAKE, lddw=16)
FWD = dict(T=8, D=16, F=32, x=FAKE, ldx=16, wg=FAKE, wu=FAKE, ldw=16, act=0, h=FAKE, ldh=32, g8=FAKE, gs=FAKE,
           u8=FAKE, us=FAKE)
BWD = dict(T=8, D=16, F=32, dh=FAKE, lddh=32, x=FAKE, ldx=16, x8=None, xs=None, wg=FAKE, wu=FAKE, ldw=16, act=0,
           g8=FAKE, gs=FAKE, u8=FAKE, us=FAKE, h=FAKE, ldh=32, dx=FAKE, lddx=16, dwg=FAKE, dwu=FAKE, lddw=16)
WGRAD = dict(T=8, N=16, D=32, dy=FAKE, lddy=16, q=FAKE, scale=FAKE, dw=FAKE, lddw=32)
NULL, SIZE, HYPER = z.ZOPT_ERR_NULL, z.ZOPT_ERR_SIZE, z.ZOPT_ERR_HYPER


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(T=(1 << 30) + 1), SIZE), (dict(D=0), SIZE), (dict(D=BIG + 1), SIZE), (dict(V=0), SIZE),
    (dict(V=BIG + 1), SIZE), (dict(ldx=15), SIZE), (dict(ldw=15), SIZE), (dict(lddx=15), SIZE), (dict(lddw=15), SIZE),
    (dict(ldx=(1 << 31) + 1), SIZE), (dict(x=None), NULL), (dict(w=None), NULL), (dict(target=None), NULL),
    (dict(loss=None), NULL), (dict(mean=2), HYPER), (dict(mean=-1), HYPER), (dict(grad_scale=float("inf")), HYPER),
    (dict(grad_scale=float("nan")), HYPER)])
def test_linear_xent_rejects(kw, status):
    assert call(z.lib().zopt_linear_xent, {**XENT, **kw}.values())[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(D=0), SIZE), (dict(F=0), SIZE), (dict(F=BIG + 1), SIZE), (dict(ldx=15), SIZE),
    (dict(ldw=15), SIZE), (dict(ldh=31), SIZE), (dict(x=None), NULL), (dict(wg=None), NULL), (dict(wu=None), NULL),
    (dict(h=None), NULL), (dict(g8=None), NULL), (dict(us=None), NULL), (dict(act=2), HYPER), (dict(act=-1), HYPER)])
def test_glu_forward_rejects(kw, status):
    assert call(z.lib().zopt_glu_forward, {**FWD, **kw}.values())[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(D=0), SIZE), (dict(F=0), SIZE), (dict(lddh=31), SIZE), (dict(ldx=15), SIZE),
    (dict(lddx=15), SIZE), (dict(lddw=15), SIZE), (dict(ldh=31), SIZE), (dict(dh=None), NULL), (dict(x=None), NULL),
    (dict(x8=FAKE), NULL), (dict(wg=None), NULL), (dict(dx=None), NULL), (dict(dwg=None), NULL),
    (dict(dwu=None), NULL), (dict(g8=None), NULL), (dict(us=None), NULL), (dict(act=2), HYPER)])
def test_glu_backward_rejects(kw, status):
    assert call(z.lib().zopt_glu_backward, {**BWD, **kw}.values())[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(N=0), SIZE), (dict(D=0), SIZE), (dict(lddy=15), SIZE), (dict(lddw=31), SIZE),
    (dict(dy=None), NULL), (dict(q=None), NULL), (dict(scale=None), NULL), (dict(dw=None), NULL)])
def test_act8_wgrad_rejects(kw, status):
    assert call(z.lib().zopt_act8_wgrad, {**WGRAD, **kw}.values())[0] == status


def test_act8_pack_and_unpack_reject_and_empty_is_a_noop():
    L = z.lib()
    for fn, ok in ((L.zopt_act8_pack, (FAKE, 8, FAKE, FAKE)), (L.zopt_act8_unpack, (FAKE, FAKE, FAKE, 8))):
        assert fn(-1, 8, *ok, None) == SIZE
        assert fn(4, 0, *ok, None) == SIZE
        assert fn(4, BIG + 1, *ok, None) == SIZE
        assert fn(4, 9, *ok, None) == SIZE  # stride 8 < 9
        assert fn(0, 8, *ok, None) == z.ZOPT_OK
        for k, v in enumerate(ok):
            if v == FAKE:
                assert fn(4, 8, *ok[:k], None, *ok[k + 1:], None) == NULL


@pytest.mark.parametrize("name,args", [("zopt_linear_xent", XENT), ("zopt_glu_forward", FWD),
                                       ("zopt_glu_backward", BWD), ("zopt_act8_wgrad", WGRAD)])
def test_workspace_is_sized_and_checked(name, args):
    fn = getattr(z.lib(), name)
    st, need = call(fn, args.values(), ws=None, size=0)
    assert st == z.ZOPT_OK and need % 256 == 0
    assert (need == 0) == (name == "zopt_glu_forward")  # aligned operands, one launch
    if need:
        assert call(fn, args.values(), size=need - 1)[0] == z.ZOPT_ERR_WORKSPACE
    assert call(fn, args.values(), ws=FAKE + 128, size=need)[0] == z.ZOPT_ERR_WORKSPACE
    assert fn(*args.values(), FAKE, None, None) == NULL


def test_xent_workspace_follows_what_is_asked():
    """The exponentials (2 bytes a logit, at most 2 GiB) come with a gradient,
    the fp32 sums of dw with more than one piece, copies with odd operands."""
    fn = z.lib().zopt_linear_xent

    def need(**kw):
        st, n = call(fn, {**XENT, **kw}.values(), ws=None)
        assert st == z.ZOPT_OK
        return n

    sizes = dict(T=8192, D=4096, V=131072, ldx=4096, ldw=4096, lddx=4096, lddw=4096)
    loss = need(**sizes, dx=None, dw=None)
    only_dx = need(**sizes, dw=None)
    assert only_dx == loss + 8192 * 131072 * 2
    assert need(**sizes) == only_dx + 8192 * 4096 * 2  # x without the ignored rows
    assert need(**{**sizes, "T": 65536}) < 12 * (1 << 30)
    assert need(**sizes, dx=None, w=FAKE + 2) - need(**sizes, dx=None) == 131072 * 4096 * 2
    assert need(**{**sizes, "ldw": 4097}, dx=None) - need(**sizes, dx=None) == 131072 * 4096 * 2


def test_python_checks():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(32, 16, dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="x: dtype"):
        z.linear_xent_loss(x.float(), w, y)
    with pytest.raises(ValueError, match="x: must be a GPU tensor"):
        z.linear_xent_loss(x, w, y)
    with pytest.raises(ValueError, match="x: shape"):
        z.act8_pack(x[0])
    with pytest.raises(TypeError, match="a: expected an Act8"):
        z.act8_unpack(x)
    with pytest.raises(ValueError, match="dh: must be a GPU tensor"):
        z.glu_backward(x, x, w, w)
    with pytest.raises(ValueError, match="act:"):
        z._act_id("relu")
    with pytest.raises(TypeError, match="expected a tensor"):
        z.glu_forward(None, w, w)


def test_row_strides():
    """_need_rows on tensors that are not on a GPU stops at the device; the
    stride rules are looked at with meta tensors made to look like one."""
    class Gpu(torch.Tensor):
        @property
        def device(self):
            return torch.device("cuda:0")

    def t(*a):
        return torch.empty(32, 64, dtype=torch.bfloat16).as_strided(*a).as_subclass(Gpu)

    need = lambda v: z._need_rows(v, torch.bfloat16, None, None, "v")  # noqa: E731
    assert need(t((4, 16), (64, 1))) == 64
    assert need(t((1, 16), (3, 1))) == 16       # one row: its stride says nothing
    assert need(t((4, 1), (5, 7))) == 5
    for bad in (((4, 16), (1, 64)), ((4, 16), (0, 1)), ((4, 16), (15, 1)), ((4, 8), (32, 2))):
        with pytest.raises(ValueError, match="strides"):
            need(t(*bad))
    with pytest.raises(ValueError, match="rows are empty"):
        need(t((4, 0), (1, 1)))
