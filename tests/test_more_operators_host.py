"""Refusals of the routing by scores, AdamW and the gradients' norm before any launch (no GPU)."""
import ctypes
import math

import pytest
import torch

from test_abi_host import _Fake, bd  # noqa: F401  (bd: the library fixture)
from test_operators_host import _by, _Holder, _ws


def _rule(bd, score=1, groups=4, topk_groups=2, group_rank=2, renormalise=1, scale=2.5):
    return bd.MoeRouterRule(score, groups, topk_groups, group_rank, renormalise, scale)


def _select(bd, T=64, E=16, k=3):
    f = _Fake(bd)
    F32, I32, U8 = bd.MOE_DT_F32, bd.MOE_DT_I32, bd.MOE_DT_U8
    return f, {"logits": f.t((T, E), F32), "bias": f.t((E,), F32), "mask": f.t((T,), U8), "idx": f.t((T, k), I32), "w": f.t((T, k), F32),
               "dw": f.t((T, k), F32), "dl": f.t((T, E), F32)}


def _fwd(bd, a, rule):
    return bd.LIB.moe_router_select_fwd(*[_by(a[n]) for n in ("logits", "bias", "mask", "idx", "w")], _by(rule), None)


def _bwd(bd, a, rule, accumulate=0):
    return bd.LIB.moe_router_select_bwd(*[_by(a[n]) for n in ("logits", "idx", "w", "dw", "dl")], _by(rule), accumulate, None)


@pytest.mark.parametrize("name,shape,dt,code,both", [
    ("logits", (63, 16), "F32", "MOE_ERR_SHAPE", True), ("logits", (64, 16), "I32", "MOE_ERR_DTYPE", True),
    ("logits", (64, 2048), "F32", "MOE_ERR_UNSUPPORTED", True), ("logits", (64, 18), "F32", "MOE_ERR_SHAPE", True),
    ("idx", (64, 33), "I32", "MOE_ERR_UNSUPPORTED", True), ("idx", (64, 9), "I32", "MOE_ERR_SHAPE", True), ("idx", (64, 3), "F32", "MOE_ERR_DTYPE", True),
    ("w", (64, 2), "F32", "MOE_ERR_SHAPE", True), ("w", (64, 3), "BF16", "MOE_ERR_DTYPE", True), ("bias", (15,), "F32", "MOE_ERR_SHAPE", False),
    ("bias", (16,), "BF16", "MOE_ERR_DTYPE", False), ("mask", (63,), "U8", "MOE_ERR_SHAPE", False), ("mask", (64,), "I32", "MOE_ERR_DTYPE", False)])
def test_select_refuses_bad_tensors(bd, name, shape, dt, code, both):  # noqa: F811
    f, a = _select(bd)
    a[name] = f.t(shape, getattr(bd, "MOE_DT_" + dt))
    assert _fwd(bd, a, _rule(bd)) == bd.ERR[code]
    if both:
        assert _bwd(bd, a, _rule(bd)) == bd.ERR[code]


@pytest.mark.parametrize("kw,code", [
    ({"score": 2}, "UNSUPPORTED"), ({"score": -1}, "UNSUPPORTED"), ({"groups": 0}, "UNSUPPORTED"), ({"groups": 33}, "UNSUPPORTED"), ({"groups": 3}, "SHAPE"),
    ({"topk_groups": 0}, "SHAPE"), ({"topk_groups": 5}, "SHAPE"), ({"group_rank": 0}, "UNSUPPORTED"), ({"group_rank": 3}, "UNSUPPORTED"),
    ({"scale": 0.0}, "UNSUPPORTED"), ({"scale": -1.0}, "UNSUPPORTED"), ({"scale": math.nan}, "UNSUPPORTED"), ({"scale": math.inf}, "UNSUPPORTED"),
    ({"groups": 16, "topk_groups": 2}, "SHAPE")])
def test_select_refuses_bad_rules(bd, kw, code):  # noqa: F811
    f, a = _select(bd)
    assert _fwd(bd, a, _rule(bd, **kw)) == bd.ERR["MOE_ERR_" + code]
    assert _bwd(bd, a, _rule(bd, **kw)) == bd.ERR["MOE_ERR_" + code]


def test_select_refuses_layouts_and_missing_tensors(bd):  # noqa: F811
    E = bd.ERR
    for name in ("logits", "idx", "w"):
        f, a = _select(bd)
        a[name] = None
        assert _fwd(bd, a, _rule(bd)) == E["MOE_ERR_NULL"] and _bwd(bd, a, _rule(bd)) == E["MOE_ERR_NULL"]
    for name in ("dw", "dl"):
        f, a = _select(bd)
        a[name] = None
        assert _bwd(bd, a, _rule(bd)) == E["MOE_ERR_NULL"]
    f, a = _select(bd)
    assert _fwd(bd, a, None) == E["MOE_ERR_NULL"] and _bwd(bd, a, None) == E["MOE_ERR_NULL"]
    a["logits"] = f.t((64, 16), bd.MOE_DT_F32, contiguous=False)
    assert _fwd(bd, a, _rule(bd)) == E["MOE_ERR_LAYOUT"] and _bwd(bd, a, _rule(bd)) == E["MOE_ERR_LAYOUT"]
    f, a = _select(bd)
    a["bias"] = f.t((16,), bd.MOE_DT_F32, misalign=4)
    assert _fwd(bd, a, _rule(bd)) == E["MOE_ERR_ALIGN"]
    f, a = _select(bd)
    a["dl"] = f.t((64, 16), bd.MOE_DT_BF16)
    assert _bwd(bd, a, _rule(bd), accumulate=1) == E["MOE_ERR_UNSUPPORTED"]
    a["dl"] = f.t((64, 16), bd.MOE_DT_I32)
    assert _bwd(bd, a, _rule(bd)) == E["MOE_ERR_DTYPE"]


def test_bias_step_refusals(bd):  # noqa: F811
    E, f = bd.ERR, _Fake(bd)
    step = lambda c, b, r=1e-3: bd.LIB.moe_router_bias_step(_by(c), _by(b), r, None)  # noqa: E731
    counts, bias = f.t((2, 8), bd.MOE_DT_I32), f.t((8,), bd.MOE_DT_F32)
    assert step(None, bias) == E["MOE_ERR_NULL"] and step(counts, None) == E["MOE_ERR_NULL"]
    assert step(f.t((8,), bd.MOE_DT_I32), bias) == E["MOE_ERR_SHAPE"]
    assert step(f.t((2, 9), bd.MOE_DT_I32), bias) == E["MOE_ERR_SHAPE"]
    assert step(f.t((2, 2000), bd.MOE_DT_I32), f.t((2000,), bd.MOE_DT_F32)) == E["MOE_ERR_UNSUPPORTED"]
    assert step(f.t((2, 8), bd.MOE_DT_F32), bias) == E["MOE_ERR_DTYPE"]
    for rate in (-1.0, math.nan, math.inf):
        assert step(counts, bias, rate) == E["MOE_ERR_UNSUPPORTED"]


def _adamw(bd, n=1000, count=3, state="F32"):
    f = _Fake(bd)
    F32, B16 = bd.MOE_DT_F32, bd.MOE_DT_BF16
    st = getattr(bd, "MOE_DT_" + state)
    a = {"p": [f.t((n,), F32) for _ in range(count)], "g": [f.t((n,), (F32, B16)[i % 2]) for i in range(count)],
         "m": [f.t((n,), st) for _ in range(count)], "v": [f.t((n,), st) for _ in range(count)],
         "ms": [f.t((-(-n // 256),), F32) for _ in range(count)], "vs": [f.t((-(-n // 256),), F32) for _ in range(count)],
         "copy": [f.t((n,), B16) for _ in range(count)]}
    return f, a


def _step(bd, a, count=None, lr_at=None, step_at=None, scale=None, **kw):
    o = bd.MoeAdamwOptions(*[kw.get(n, d) for n, d in (("lr", 1e-3), ("beta1", 0.9), ("beta2", 0.999), ("eps", 1e-8), ("decay", 0.1), ("step", 1), ("seed", 0))])
    for name, t in (("lr_on_device", lr_at), ("step_on_device", step_at), ("grad_scale", scale)):
        if t is not None:
            setattr(o, name, ctypes.pointer(t))
    arrays = [None if a[n] is None else (bd.MoeTensor * len(a[n]))(*a[n]) for n in ("p", "g", "m", "v", "ms", "vs", "copy")]
    return bd.LIB.moe_adamw_step(len(a["p"]) if count is None else count, *arrays, ctypes.byref(o), None)


@pytest.mark.parametrize("kw", [{"lr": -1.0}, {"lr": math.nan}, {"lr": math.inf}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0}, {"beta2": math.nan}, {"eps": 0.0},
                                {"eps": 2.0}, {"decay": -1.0}, {"decay": math.nan}])
def test_adamw_refuses_numbers(bd, kw):  # noqa: F811
    _, a = _adamw(bd)
    assert _step(bd, a, **kw) == bd.ERR["MOE_ERR_UNSUPPORTED"]


def test_adamw_refuses_steps_and_counts(bd):  # noqa: F811
    E = bd.ERR
    f, a = _adamw(bd)
    assert _step(bd, a, step=0) == E["MOE_ERR_SHAPE"] and _step(bd, a, step=-5) == E["MOE_ERR_SHAPE"]
    assert _step(bd, a, count=-1) == E["MOE_ERR_SHAPE"] and _step(bd, a, count=65537) == E["MOE_ERR_UNSUPPORTED"]
    assert _step(bd, a, count=0) == 0
    assert bd.LIB.moe_adamw_step(0, *[None] * 7, None, None) == E["MOE_ERR_NULL"]
    for bad, code in ((f.t((2,), bd.MOE_DT_F32), "SHAPE"), (f.t((1,), bd.MOE_DT_I32), "DTYPE"), (f.t((1,), bd.MOE_DT_F32, misalign=2), "ALIGN")):
        assert _step(bd, a, lr_at=bad) == E["MOE_ERR_" + code] and _step(bd, a, scale=bad) == E["MOE_ERR_" + code]
    assert _step(bd, a, step_at=f.t((1,), bd.MOE_DT_F32)) == E["MOE_ERR_DTYPE"]


@pytest.mark.parametrize("state", ["F32", "U8", "E4M3"])
@pytest.mark.parametrize("name,change,code", [
    ("p", lambda f, bd: f.t((1000,), bd.MOE_DT_BF16), "DTYPE"), ("p", lambda f, bd: f.t((999,), bd.MOE_DT_F32), "SHAPE"),
    ("p", lambda f, bd: f.t((10, 100), bd.MOE_DT_F32, contiguous=False), "LAYOUT"), ("p", lambda f, bd: f.t((1000,), bd.MOE_DT_F32, misalign=4), "ALIGN"),
    ("g", lambda f, bd: f.t((1000,), bd.MOE_DT_I32), "DTYPE"), ("g", lambda f, bd: f.t((1001,), bd.MOE_DT_BF16), "SHAPE"),
    ("g", lambda f, bd: f.t((1000,), bd.MOE_DT_BF16, misalign=8), "ALIGN"), ("m", lambda f, bd: f.t((1000,), bd.MOE_DT_BF16), "DTYPE"),
    ("v", lambda f, bd: f.t((1000,), bd.MOE_DT_I32), "DTYPE"), ("v", lambda f, bd: f.t((500,), bd.MOE_DT_F32), "SHAPE DTYPE"),
    ("copy", lambda f, bd: f.t((1000,), bd.MOE_DT_F32), "DTYPE"), ("copy", lambda f, bd: f.t((998,), bd.MOE_DT_BF16), "SHAPE")])
def test_adamw_refuses_tensors(bd, state, name, change, code):  # noqa: F811
    f, a = _adamw(bd, state=state)
    a[name][2] = change(f, bd)                       # the last of the list: nothing of it is launched
    assert _step(bd, a) in [bd.ERR["MOE_ERR_" + c] for c in code.split()]


def test_adamw_refuses_mixtures_scales_and_the_same_parameter_twice(bd):  # noqa: F811
    E = bd.ERR
    f, a = _adamw(bd, state="E4M3")
    a["m"][1] = f.t((1000,), bd.MOE_DT_F32)
    assert _step(bd, a) == E["MOE_ERR_DTYPE"]
    for name in ("ms", "vs"):
        f, a = _adamw(bd, state="U8")
        a[name][0] = f.t((3,), bd.MOE_DT_F32)
        assert _step(bd, a) == E["MOE_ERR_SHAPE"]
        a[name] = None
        assert _step(bd, a) == E["MOE_ERR_NULL"]
    for count in (2, 300, 2000):
        f, a = _adamw(bd, n=64, count=count)
        a["p"][count - 1] = a["p"][0]
        assert _step(bd, a) == E["MOE_ERR_UNSUPPORTED"]
    f, a = _adamw(bd)
    a["p"][1].data = None
    assert _step(bd, a) == E["MOE_ERR_NULL"]
    f, a = _adamw(bd)
    a["g"] = None
    assert _step(bd, a) == E["MOE_ERR_NULL"]
    huge = f.t((1,), bd.MOE_DT_F32)
    huge.ndim, huge.shape[0], huge.shape[1], huge.shape[2] = 3, 1 << 40, 1 << 40, 1 << 40      # its product is beyond 64 bits
    f, a = _adamw(bd)
    a["p"][0] = huge
    assert _step(bd, a) == E["MOE_ERR_SHAPE"]


def test_norm_refusals(bd):  # noqa: F811
    E, f = bd.ERR, _Fake(bd)
    need = bd.moe_grad_norm_workspace_bytes(3000, 3)
    grads = [f.t((1000,), bd.MOE_DT_F32), f.t((10, 100), bd.MOE_DT_BF16), f.t((1000,), bd.MOE_DT_F32)]
    out = f.t((2,), bd.MOE_DT_F32, misalign=4)

    def norm(grads, out, ws, most=1.0, count=None):
        return bd.LIB.moe_grad_norm(len(grads) if count is None else count, (bd.MoeTensor * max(len(grads), 1))(*grads), _by(out), most, _by(ws), None)
    assert norm(grads, out, _ws(bd, need - 1)) == E["MOE_ERR_SCRATCH"]
    assert norm(grads, out, _ws(bd, need, 64)) == E["MOE_ERR_SCRATCH"]
    assert norm(grads, out, None) == E["MOE_ERR_NULL"] and norm(grads, None, _ws(bd, need)) == E["MOE_ERR_NULL"]
    assert norm(grads, f.t((1,), bd.MOE_DT_F32), _ws(bd, need)) == E["MOE_ERR_SHAPE"]
    assert norm(grads, f.t((2,), bd.MOE_DT_I32), _ws(bd, need)) == E["MOE_ERR_DTYPE"]
    assert norm(grads, out, _ws(bd, need), count=-1) == E["MOE_ERR_SHAPE"] and norm(grads, out, _ws(bd, need), count=70000) == E["MOE_ERR_UNSUPPORTED"]
    for most in (-1.0, math.nan, math.inf):
        assert norm(grads, out, _ws(bd, need), most) == E["MOE_ERR_UNSUPPORTED"]
    used = _ws(bd, need)
    used.state[0] = 1
    assert norm(grads, out, used) == E["MOE_ERR_STATE"]
    for bad, code in ((f.t((5,), bd.MOE_DT_U8), "DTYPE"), (f.t((4, 5), bd.MOE_DT_F32, contiguous=False), "LAYOUT"), (f.t((5,), bd.MOE_DT_F32, misalign=4), "ALIGN")):
        assert norm(grads + [bad], out, _ws(bd, 1 << 20)) == E["MOE_ERR_" + code]
    size = bd.moe_grad_norm_workspace_bytes
    assert 0 < size(0, 0) <= size(1000, 1) < size(10 ** 6, 1) and size(10 ** 12, 65536) < 1 << 24
    for bad in ((-1, 1), (1 << 41, 1), (10, -1), (10, 65537)):
        assert size(*bad) == 0


def test_binding_refuses_other_kinds_of_arguments(bd):  # noqa: F811
    """Off the GPU, of other types, of unlike lengths: an exception, nothing else."""
    F = torch.zeros
    rule = bd.RouterRule(score="sigmoid")
    with pytest.raises(bd.MoeError, match="UNSUPPORTED"):
        bd.RouterRule(score="tanh")
    idx, w = F(4, 2, dtype=torch.int32), F(4, 2)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_router_select_fwd(F(4, 8), idx, w, rule, stream=0)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_router_select_bwd(F(4, 8), idx, w, w, F(4, 8), rule, stream=0)
    with pytest.raises(bd.MoeError, match="DTYPE"):
        bd.moe_router_select_fwd(F(4, 8).half(), idx, w, rule, stream=0)
    with pytest.raises(TypeError):
        bd.moe_router_select_fwd([1.0], idx, w, rule, stream=0)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_router_bias_step(F(1, 8, dtype=torch.int32), F(8), 0.1, stream=0)
    with pytest.raises(TypeError):
        bd.moe_router_bias_step(F(1, 8, dtype=torch.int32), F(8), "x", stream=0)
    p, m = F(10), F(10)
    step = lambda *a, **k: bd.moe_adamw_step(*a, stream=0, **k)  # noqa: E731
    with pytest.raises(bd.MoeError, match="NULL"):
        step([p], [p], [m], [m], 1)
    with pytest.raises(bd.MoeError, match="DTYPE"):
        step([p.double()], [p], [m], [m], 1)
    with pytest.raises(bd.MoeError, match="LAYOUT"):
        step([F(10, 4).t()], [F(4, 10)], [F(4, 10)], [F(4, 10)], 1)
    with pytest.raises(ValueError):
        step([p, p], [p], [m], [m], 1)
    for bad in ([p, "x"], 5, [None]):
        with pytest.raises(TypeError):
            step([p], bad, [m], [m], 1)
    for kw in ({"lr": "x"}, {"betas": ("a", 0.9)}, {"eps": None}, {"seed": 1.5}):
        with pytest.raises(TypeError):
            step([p], [p], [m], [m], 1, **kw)
    with pytest.raises((TypeError, OverflowError)):
        step([p], [p], [m], [m], 2 ** 80)
    with pytest.raises(bd.MoeError, match="SHAPE"):
        step([p], [p], [m], [m], 0)
    step([], [], [], [], 1)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_grad_norm([p], F(2), _Holder(bd), stream=0)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_grad_norm([F(5)], None, _Holder(bd), stream=0)
