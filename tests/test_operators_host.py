"""Refusals of moe_balance_fwd / moe_balance_bwd and moe_orthogonalise before any launch (no GPU)."""
import ctypes

import pytest

from test_abi_host import _Fake, bd  # noqa: F401  (bd: the library fixture)


def _ws(bd, n, misalign=0):
    s = bd.MoeScratch()
    s.data, s.bytes = (1 << 40) + misalign, n
    return s


def _by(t):
    return None if t is None else ctypes.byref(t)


def _balance(bd, T=64, E=16, k=2, B=3):
    f = _Fake(bd)
    F32, I32, U8 = bd.MOE_DT_F32, bd.MOE_DT_I32, bd.MOE_DT_U8
    return f, {"logits": f.t((T, E), F32), "idx": f.t((T, k), I32), "w": f.t((T, k), F32), "dw": f.t((T, k), F32),
               "mask": f.t((T,), U8), "off": f.t((B + 1,), I32), "counts": f.t((B, E), I32), "tokens": f.t((B,), I32),
               "loss": f.t((B, 2), F32), "dl": f.t((T, E), F32)}


def _fwd(bd, a, ws):
    return bd.LIB.moe_balance_fwd(*[_by(a[n]) for n in ("logits", "idx", "mask", "off", "counts", "tokens", "loss")], _by(ws),
                                  None)


def _bwd(bd, a):
    return bd.LIB.moe_balance_bwd(*[_by(a[n]) for n in ("logits", "idx", "w", "dw", "mask", "off", "counts", "tokens", "loss",
                                                        "dl")], None)


@pytest.mark.parametrize("name,shape,dt,code", [
    ("logits", (64, 17), "F32", "MOE_ERR_SHAPE"), ("logits", (64, 16), "BF16", "MOE_ERR_DTYPE"),
    ("logits", (64, 2048), "F32", "MOE_ERR_UNSUPPORTED"), ("idx", (63, 2), "I32", "MOE_ERR_SHAPE"),
    ("idx", (64, 33), "I32", "MOE_ERR_UNSUPPORTED"), ("idx", (64, 17), "I32", "MOE_ERR_UNSUPPORTED"),
    ("idx", (64, 2), "F32", "MOE_ERR_DTYPE"), ("mask", (63,), "U8", "MOE_ERR_SHAPE"), ("mask", (64,), "I32", "MOE_ERR_DTYPE"),
    ("off", (3,), "I32", "MOE_ERR_SHAPE"), ("off", (4,), "F32", "MOE_ERR_DTYPE"), ("counts", (3, 15), "I32", "MOE_ERR_SHAPE"),
    ("counts", (3, 16), "F32", "MOE_ERR_DTYPE"), ("tokens", (2,), "I32", "MOE_ERR_SHAPE"),
    ("tokens", (3,), "F32", "MOE_ERR_DTYPE"), ("loss", (3, 1), "F32", "MOE_ERR_SHAPE"), ("loss", (3, 2), "BF16", "MOE_ERR_DTYPE"),
])
def test_balance_refuses_bad_tensors(bd, name, shape, dt, code):  # noqa: F811
    f, a = _balance(bd)
    a[name] = f.t(shape, getattr(bd, "MOE_DT_" + dt))
    ws = _ws(bd, 1 << 30)
    assert _fwd(bd, a, ws) == bd.ERR[code]
    assert _bwd(bd, a) == bd.ERR[code]


def test_balance_refuses_layouts_workspaces_and_halves(bd):  # noqa: F811
    E = bd.ERR
    need = bd.moe_balance_workspace_bytes(64, 16, 3)
    f, a = _balance(bd)
    assert _fwd(bd, a, _ws(bd, need - 1)) == E["MOE_ERR_SCRATCH"]
    assert _fwd(bd, a, _ws(bd, need, 64)) == E["MOE_ERR_SCRATCH"]
    assert _fwd(bd, a, None) == E["MOE_ERR_NULL"]
    used = _ws(bd, need)
    used.state[0] = 1                     # moe_orthogonalise has left data there
    assert _fwd(bd, a, used) == E["MOE_ERR_STATE"]
    for name in ("logits", "idx", "counts", "tokens", "loss"):
        f, a = _balance(bd)
        a[name] = None
        assert _fwd(bd, a, _ws(bd, need)) == E["MOE_ERR_NULL"], name
    f, a = _balance(bd)
    a["off"] = None                       # several segments need their bounds
    assert _fwd(bd, a, _ws(bd, need)) == E["MOE_ERR_SHAPE"]
    f, a = _balance(bd)
    a["dw"] = None                        # weights without their gradient
    assert _bwd(bd, a) == E["MOE_ERR_NULL"]
    f, a = _balance(bd)
    a["dw"] = f.t((64, 3), bd.MOE_DT_F32)
    assert _bwd(bd, a) == E["MOE_ERR_SHAPE"]
    f, a = _balance(bd)
    a["dl"] = f.t((64, 16), bd.MOE_DT_F32, contiguous=False)
    assert _bwd(bd, a) == E["MOE_ERR_LAYOUT"]
    f, a = _balance(bd)
    a["logits"] = f.t((64, 16), bd.MOE_DT_F32, misalign=4)
    assert _fwd(bd, a, _ws(bd, need)) == E["MOE_ERR_ALIGN"]
    assert _bwd(bd, a) == E["MOE_ERR_ALIGN"]


def test_balance_workspace_sizes(bd):  # noqa: F811
    size = bd.moe_balance_workspace_bytes
    assert 0 < size(0, 8, 1) <= size(1, 8, 1) < size(100000, 8, 1) < size(100000, 128, 1) < size(100000, 128, 50)
    for bad in [(-1, 8, 1), (1 << 30, 8, 1), (10, 0, 1), (10, 1025, 1), (10, 8, 0), (10, 8, 65536)]:
        assert size(*bad) == 0, bad


def _ortho(bd, G, O, ws, steps=5, coeffs=None, eps=1e-7):
    co = None if coeffs is None else (ctypes.c_float * len(coeffs))(*coeffs)
    return bd.LIB.moe_orthogonalise(_by(G), _by(O), steps, co, eps, _by(ws), None)


def test_orthogonalise_refusals(bd):  # noqa: F811
    E = bd.ERR
    f = _Fake(bd)
    F32, B16, I32 = bd.MOE_DT_F32, bd.MOE_DT_BF16, bd.MOE_DT_I32
    need = bd.moe_orthogonalise_workspace_bytes(2, 48, 100)
    G, O, ws = f.t((2, 48, 100), F32), f.t((2, 48, 100), B16), _ws(bd, need)
    assert _ortho(bd, f.t((48, 100), F32), O, ws) == E["MOE_ERR_SHAPE"]
    assert _ortho(bd, f.t((2, 0, 100), F32), f.t((2, 0, 100), B16), ws) == E["MOE_ERR_SHAPE"]
    assert _ortho(bd, G, f.t((2, 100, 48), B16), ws) == E["MOE_ERR_SHAPE"]
    assert _ortho(bd, G, f.t((2, 48, 100), F32), ws) == E["MOE_ERR_DTYPE"]
    assert _ortho(bd, f.t((2, 48, 100), I32), O, ws) == E["MOE_ERR_DTYPE"]
    assert _ortho(bd, f.t((2, 48, 100), F32, contiguous=False), O, ws) == E["MOE_ERR_LAYOUT"]
    assert _ortho(bd, f.t((2, 48, 100), F32, misalign=8), O, ws) == E["MOE_ERR_ALIGN"]
    assert _ortho(bd, G, O, _ws(bd, need - 1)) == E["MOE_ERR_SCRATCH"]
    assert _ortho(bd, G, O, _ws(bd, need, 128)) == E["MOE_ERR_SCRATCH"]
    assert _ortho(bd, G, O, None) == E["MOE_ERR_NULL"]
    assert _ortho(bd, None, O, ws) == E["MOE_ERR_NULL"]
    assert _ortho(bd, G, O, ws, steps=0) == E["MOE_ERR_SHAPE"]
    for kw in ({"steps": 17}, {"eps": 0.0}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": 2.0},
               {"coeffs": [17.0, 0, 0] * 5}, {"coeffs": [0, float("nan"), 0] * 5}):
        assert _ortho(bd, G, O, ws, **kw) == E["MOE_ERR_UNSUPPORTED"], kw
    for bad in [(65536, 4, 4), (1, 32769, 4), (1, 4, 32769), (65535, 32768, 32768), (-1, 4, 4), (1, 0, 4)]:
        assert bd.moe_orthogonalise_workspace_bytes(*bad) == 0, bad


class _Holder:
    def __init__(self, bd):
        self.handle = bd.MoeScratch()
        self.handle.data, self.handle.bytes = 1 << 40, 1 << 40
        self.address = ctypes.addressof(self.handle)


def test_orthogonalise_coefficient_lists(bd):  # noqa: F811
    """The binding takes one triple or one for each step, nothing else."""
    import torch
    G = torch.zeros(1, 4, 4)
    for bad in ([(1, 1, 1)] * 4, (1.0, 2.0), [(1, 1)] * 5):
        with pytest.raises(bd.MoeError, match="SHAPE"):
            bd.moe_orthogonalise(G, G, _Holder(bd), steps=5, coeffs=bad, stream=0)
    with pytest.raises(bd.MoeError, match="UNSUPPORTED"):
        bd.moe_orthogonalise(G, G, _Holder(bd), steps=17, coeffs=(1, 1, 1), stream=0)


def test_tensors_off_the_gpu_and_other_things_are_refused(bd):  # noqa: F811
    import torch
    ws = _Holder(bd)
    G, O = torch.zeros(1, 4, 4), torch.zeros(1, 4, 4, dtype=torch.bfloat16)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_orthogonalise(G, O, ws, stream=0)
    with pytest.raises(bd.MoeError, match="DTYPE"):
        bd.moe_orthogonalise(G.double(), O, ws, stream=0)
    with pytest.raises(bd.MoeError, match="SHAPE"):
        bd.moe_orthogonalise(G[0], O[0], ws, stream=0)
    with pytest.raises(bd.MoeError, match="SHAPE"):
        bd.moe_orthogonalise(G[None], O[None], ws, stream=0)
    with pytest.raises(TypeError):
        bd.moe_orthogonalise([1.0], O, ws, stream=0)
    logits, idx = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32)
    counts, tokens, loss = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_balance_fwd(logits, idx, counts, tokens, loss, ws, stream=0)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_balance_bwd(logits, idx, None, None, counts, tokens, loss, torch.zeros(6, 4), stream=0)
    with pytest.raises(bd.MoeError, match="DTYPE"):
        bd.moe_balance_fwd(logits.half(), idx, counts, tokens, loss, ws, stream=0)
