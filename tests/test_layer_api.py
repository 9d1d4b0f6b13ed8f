"""The C ABI and the Python checks of a decoder layer's operators without a
GPU: every refusal comes before any HIP call."""
import ctypes

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

FAKE = 0x100000  # aligned to 256 bytes; never dereferenced: every call fails validation
NULL, SIZE, HYPER, WORK = z.ZOPT_ERR_NULL, z.ZOPT_ERR_SIZE, z.ZOPT_ERR_HYPER, z.ZOPT_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def call(fn, args, ws=FAKE, size=1 << 62):
    n = ctypes.c_size_t(size)
    return fn(*args, ws, ctypes.byref(n), None), n.value


ROPE = dict(T=8, hq=4, hk=2, width=64, rot=32, q=FAKE, qt=512, qh=64, k=FAKE, kt=512, kh=64, table=FAKE, positions=8,
            position=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, style=0, yq=FAKE, yqt=256, yqh=64, yk=FAKE, ykt=128, ykh=64)
ROPE_BACK = dict(T=8, hq=4, hk=2, width=64, rot=32, dyq=FAKE, dyqt=256, dyqh=64, dyk=FAKE, dykt=128, dykh=64, q=FAKE,
                 qt=512, qh=64, k=FAKE, kt=512, kh=64, table=FAKE, positions=8, position=FAKE, wq=FAKE, wk=FAKE, eps=1e-6,
                 style=0, dq=FAKE, dqt=256, dqh=64, dk=FAKE, dkt=128, dkh=64, dwq=FAKE, dwk=FAKE)
ROUTE = dict(T=8, experts=16, top=4, logits=FAKE, ld=16, bf16=0, score=0, bias=FAKE, groups=4, top_groups=2,
             renormalise=1, scale=1.0, chosen=FAKE, weights=FAKE, offsets=FAKE, order=FAKE, place=FAKE)
PLAN = dict(T=8, experts=16, top=4, chosen=FAKE, offsets=FAKE, order=FAKE, place=FAKE)
ROUTE_BACK = dict(T=8, experts=16, top=4, dweights=FAKE, logits=FAKE, ld=16, bf16=0, score=0, renormalise=1, scale=1.0,
                  chosen=FAKE, dlogits=FAKE, lddl=16)
MOE = dict(T=8, D=16, F=32, experts=4, top=2, x=FAKE, ldx=16, wg=FAKE, wu=FAKE, ldw=16, we=512, wd=FAKE, ldd=32, wde=512,
           act=0, weights=FAKE, offsets=FAKE, order=FAKE, place=FAKE, y=FAKE, ldy=16)
MOE_BACK = dict(T=8, D=16, F=32, experts=4, top=2, dy=FAKE, lddy=16, x=FAKE, ldx=16, wg=FAKE, wu=FAKE, ldw=16, we=512,
                wd=FAKE, ldd=32, wde=512, act=0, weights=FAKE, offsets=FAKE, order=FAKE, place=FAKE, dx=FAKE, lddx=16,
                dwg=FAKE, dwu=FAKE, lddw=16, dwe=512, dwd=FAKE, lddd=32, dwde=512, dweights=FAKE)

SIDE = [(dict(T=-1), SIZE), (dict(T=(1 << 30) + 1), SIZE), (dict(hq=0), SIZE), (dict(hq=65537), SIZE), (dict(hk=-1), SIZE),
        (dict(width=0), SIZE), (dict(width=513, rot=0), SIZE), (dict(rot=31), SIZE), (dict(rot=66), SIZE),
        (dict(rot=-2), SIZE), (dict(positions=-1), SIZE), (dict(qt=-1), SIZE), (dict(qh=(1 << 40) + 1), SIZE),
        (dict(eps=-1.0), HYPER), (dict(eps=NAN), HYPER), (dict(eps=INF), HYPER), (dict(style=2), HYPER),
        (dict(q=None), NULL), (dict(k=None), NULL), (dict(table=None), NULL)]


@pytest.mark.parametrize("kw,status", SIDE + [
    (dict(yqh=63), SIZE), (dict(yqt=255), SIZE), (dict(ykt=127), SIZE), (dict(yqt=0), SIZE),
    (dict(yqt=64, yqh=511), SIZE), (dict(yq=None), NULL), (dict(yk=None), NULL)])
def test_qk_norm_rope_rejects(kw, status):
    assert z.lib().zopt_qk_norm_rope(*{**ROPE, **kw}.values(), None) == status


@pytest.mark.parametrize("kw,status", SIDE + [
    (dict(dqh=63), SIZE), (dict(dkt=127), SIZE), (dict(dyqt=-1), SIZE), (dict(dykh=-1), SIZE), (dict(dyq=None), NULL),
    (dict(dyk=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(hk=0), NULL)])
def test_qk_norm_rope_backward_rejects(kw, status):
    assert call(z.lib().zopt_qk_norm_rope_backward, {**ROPE_BACK, **kw}.values())[0] == status


def test_rope_table_rejects():
    f = z.lib().zopt_rope_table
    assert f(0, 64, 10000.0, None, None) == z.ZOPT_OK
    for args, status in (((-1, 64, 1e4, FAKE), SIZE), ((8, 0, 1e4, FAKE), SIZE), ((8, 63, 1e4, FAKE), SIZE),
                         ((8, 514, 1e4, FAKE), SIZE), ((8, 64, 0.0, FAKE), HYPER), ((8, 64, -1.0, FAKE), HYPER),
                         ((8, 64, NAN, FAKE), HYPER), ((8, 64, INF, FAKE), HYPER), ((8, 64, 1e4, None), NULL)):
        assert f(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(T=1 << 29), SIZE), (dict(experts=0), SIZE), (dict(experts=1025, ld=1025), SIZE),
    (dict(top=0), SIZE), (dict(top=17), SIZE), (dict(ld=15), SIZE), (dict(groups=0), SIZE), (dict(groups=3), SIZE),
    (dict(groups=32), SIZE), (dict(top_groups=0), SIZE), (dict(top_groups=5), SIZE), (dict(top=9), SIZE),
    (dict(logits=None), NULL), (dict(chosen=None), NULL), (dict(weights=None), NULL), (dict(offsets=None), NULL),
    (dict(order=None), NULL), (dict(place=None), NULL), (dict(bf16=2), HYPER), (dict(score=2), HYPER),
    (dict(score=-1), HYPER), (dict(renormalise=2), HYPER), (dict(scale=INF), HYPER), (dict(scale=NAN), HYPER)])
def test_moe_route_rejects(kw, status):
    assert call(z.lib().zopt_moe_route, {**ROUTE, **kw}.values())[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(T=1 << 29), SIZE), (dict(experts=0), SIZE), (dict(experts=1025), SIZE), (dict(top=0), SIZE),
    (dict(top=33), SIZE), (dict(chosen=None), NULL), (dict(offsets=None), NULL), (dict(order=None), NULL),
    (dict(place=None), NULL)])
def test_moe_plan_rejects(kw, status):
    assert call(z.lib().zopt_moe_plan, {**PLAN, **kw}.values())[0] == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SIZE), (dict(experts=0), SIZE), (dict(top=17), SIZE), (dict(ld=15), SIZE), (dict(lddl=15), SIZE),
    (dict(dweights=None), NULL), (dict(logits=None), NULL), (dict(chosen=None), NULL), (dict(dlogits=None), NULL),
    (dict(bf16=-1), HYPER), (dict(score=2), HYPER), (dict(renormalise=-1), HYPER), (dict(scale=NAN), HYPER)])
def test_moe_route_backward_rejects(kw, status):
    assert z.lib().zopt_moe_route_backward(*{**ROUTE_BACK, **kw}.values(), None) == status


BOTH = [(dict(T=-1), SIZE), (dict(T=1 << 30), SIZE), (dict(D=0), SIZE), (dict(F=0), SIZE), (dict(F=(1 << 21) + 1), SIZE),
        (dict(experts=0), SIZE), (dict(experts=1025), SIZE), (dict(top=0), SIZE), (dict(top=33), SIZE),
        (dict(ldx=15), SIZE), (dict(ldw=15), SIZE), (dict(ldd=31), SIZE), (dict(we=511), SIZE), (dict(wde=511), SIZE),
        (dict(ldw=17), SIZE), (dict(x=None), NULL), (dict(wg=None), NULL), (dict(wu=None), NULL), (dict(wd=None), NULL),
        (dict(weights=None), NULL), (dict(offsets=None), NULL), (dict(order=None), NULL), (dict(place=None), NULL),
        (dict(act=2), HYPER)]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(ldy=15), SIZE), (dict(y=None), NULL)])
def test_moe_forward_rejects(kw, status):
    assert call(z.lib().zopt_moe_forward, {**MOE, **kw}.values())[0] == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(lddy=15), SIZE), (dict(lddx=15), SIZE), (dict(lddw=15), SIZE), (dict(lddd=31), SIZE), (dict(dwe=511), SIZE),
    (dict(dwde=511), SIZE), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dwg=None), NULL), (dict(dwu=None), NULL),
    (dict(dwd=None), NULL), (dict(dweights=None), NULL)])
def test_moe_backward_rejects(kw, status):
    assert call(z.lib().zopt_moe_backward, {**MOE_BACK, **kw}.values())[0] == status


@pytest.mark.parametrize("name,args,least", [
    ("zopt_qk_norm_rope_backward", ROPE_BACK, 1), ("zopt_moe_route", {**ROUTE, "T": 5000}, 1), ("zopt_moe_route", ROUTE, 0),
    ("zopt_moe_plan", {**PLAN, "T": 5000}, 1), ("zopt_moe_plan", PLAN, 0), ("zopt_moe_forward", MOE, 1),
    ("zopt_moe_backward", MOE_BACK, 1)])
def test_workspace_is_sized_and_checked(name, args, least):
    fn = getattr(z.lib(), name)
    st, need = call(fn, args.values(), ws=None, size=0)
    assert st == z.ZOPT_OK and need % 256 == 0 and (need > 0) == (least > 0)
    if need:
        assert call(fn, args.values(), size=need - 1)[0] == WORK
    assert call(fn, args.values(), ws=FAKE + 128, size=need)[0] == WORK
    assert fn(*args.values(), FAKE, None, None) == NULL


def test_no_weights_no_workspace():
    assert call(z.lib().zopt_qk_norm_rope_backward, {**ROPE_BACK, "dwq": None, "dwk": None}.values(), ws=None) == (
        z.ZOPT_OK, 0)


class Gpu(torch.Tensor):
    """A tensor that says it lies on GPU 0 (nothing reads it)."""
    @property
    def device(self):
        return torch.device("cuda:0")

    def get_device(self):
        return 0


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Gpu)


I32, F32 = torch.int32, torch.float32


@pytest.mark.parametrize("kw,error,match", [
    (dict(q=gpu(4, 2, 8, dtype=F32)), TypeError, "q: dtype"), (dict(q=torch.zeros(4, 2, 8, dtype=torch.bfloat16)), ValueError,
                                                              "q: must be a GPU tensor"),
    (dict(q=gpu(4, 8)), ValueError, "q: shape"), (dict(q=None), TypeError, "q: expected a tensor"),
    (dict(k=gpu(5, 2, 8)), ValueError, "k: shape"), (dict(k=gpu(4, 0, 8)), ValueError, "k: no heads"),
    (dict(q=gpu(4, 0, 8)), ValueError, "no heads"), (dict(q=gpu(4, 2, 16)[..., ::2]), ValueError, "q: strides"),
    (dict(table=gpu(4, 4, dtype=F32)), ValueError, "table: shape"), (dict(table=gpu(4, 4, 2)), TypeError, "table: dtype"),
    (dict(table=gpu(4, 5, 2, dtype=F32)), ValueError, "turns 10"), (dict(position=gpu(4, dtype=I32)), TypeError, "position"),
    (dict(position=gpu(3, dtype=torch.int64)), ValueError, "position: shape"), (dict(w_q=gpu(7)), ValueError, "w_q: shape"),
    (dict(w_k=gpu(8, dtype=F32)), TypeError, "w_k: dtype"), (dict(style="third"), ValueError, "style")])
def test_qk_norm_rope_python_checks(kw, error, match):
    args = dict(q=gpu(4, 2, 8), k=gpu(4, 2, 8), table=gpu(4, 4, 2, dtype=F32))
    with pytest.raises(error, match=match):
        z.qk_norm_rope(**{**args, **kw})


def route(T=4, top=2, E=8):
    return z.Route(gpu(T, top, dtype=I32), gpu(T, top, dtype=F32), gpu(E + 1, dtype=I32), gpu(T * top, dtype=I32),
                   gpu(T, top, dtype=I32))


@pytest.mark.parametrize("r,error,match", [
    (None, TypeError, "r: expected a Route"), (route(T=5), ValueError, "r.experts: shape"),
    (route()._replace(weights=gpu(4, 2)), TypeError, "r.weights: dtype"),
    (route()._replace(order=gpu(4, 2, dtype=I32)), ValueError, "r.order: shape"),
    (route()._replace(place=gpu(4, 3, dtype=I32)), ValueError, "r.place: shape"),
    (route()._replace(place=gpu(2, 4, dtype=I32).t()), ValueError, "r.place"),
    (route()._replace(offsets=gpu(1, dtype=I32)), ValueError, "r.offsets: shape"),
    (route()._replace(experts=torch.zeros(4, 2, dtype=I32)), ValueError, "r.experts: must be a GPU tensor")])
def test_route_checks(r, error, match):
    with pytest.raises(error, match=match):
        z._need_route(r, 4, "r", 0)


def test_need_route_takes_what_is_right():
    E, top, _ = z._need_route(route(), 4, "r", 0)
    assert (E, top) == (8, 2)


def test_experts_strides():
    need = lambda t, e=3, r=None, c=None: z._need_experts(t, e, r, c, "w", torch.device("cuda:0"))  # noqa: E731
    assert need(gpu(3, 4, 8)) == (8, 32) and need(gpu(3, 6, 8)[:, :4]) == (8, 48) and need(gpu(3, 4, 10)[..., :8]) == (10, 40)
    assert need(gpu(1, 4, 8), 1) == (8, 32)
    for bad in (gpu(3, 8, 4).transpose(1, 2), gpu(4, 3, 8).transpose(0, 1), gpu(1, 4, 8).expand(3, 4, 8), gpu(3, 4, 16)[..., ::2]):
        with pytest.raises(ValueError, match="w: strides"):
            need(bad)
    for bad, error in ((gpu(2, 4, 8), ValueError), (gpu(3, 0, 8), ValueError), (gpu(3, 4), ValueError),
                       (gpu(3, 4, 8, dtype=F32), TypeError), (None, TypeError)):
        with pytest.raises(error, match="w: "):
            need(bad)
    with pytest.raises(ValueError, match="w: on cpu"):
        need(torch.zeros(3, 4, 8, dtype=torch.bfloat16))


def test_other_python_checks():
    for bad in (torch.float16, I32):
        with pytest.raises(TypeError, match="logits: dtype"):
            z.moe_route(gpu(4, 8, dtype=bad), 2)
    with pytest.raises(TypeError, match="expected a tensor"):
        z.moe_route([1.0], 2)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        z.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="experts: dtype"):
        z.moe_plan(gpu(4, 2, dtype=torch.int64), gpu(4, 2, dtype=F32), 8)
    with pytest.raises(ValueError, match="weights: shape"):
        z.moe_plan(gpu(4, 2, dtype=I32), gpu(4, 3, dtype=F32), 8)
    with pytest.raises(ValueError, match="num_experts"):
        z.moe_plan(gpu(4, 2, dtype=I32), gpu(4, 2, dtype=F32), 0)
    with pytest.raises(TypeError, match="weights: expected"):
        z.moe_plan(gpu(4, 2, dtype=I32), None, 8)
    with pytest.raises(ValueError, match="score"):
        z._one_of("tanh", z.SCORES, "score")
    with pytest.raises(ValueError, match="on a GPU"):
        z.rope_table(4, 8, device="cpu")
