"""Lists of tensors follow them (no GPU): a tensor that has changed in place is what the next call sees, whatever its address."""
import pytest
import torch

from test_abi_host import bd  # noqa: F401  (bd: the library fixture)

NAMES = ("p", "g", "m", "v", "ms", "vs", "copy")
TYPES = {"p": torch.float32, "g": torch.float32, "m": torch.uint8, "v": torch.uint8, "ms": torch.float32, "vs": torch.float32, "copy": torch.bfloat16}


def _tensors(shape=(4, 10)):
    return {n: torch.zeros((1,) if n in ("ms", "vs") else shape, dtype=TYPES[n]) for n in NAMES}


def _step(bd, lists):  # noqa: F811
    bd.moe_adamw_step(lists["p"], lists["g"], lists["m"], lists["v"], 1, m_scales=lists["ms"], v_scales=lists["vs"], copies=lists["copy"], stream=0)


def _to_ints(t):
    t.data = t.data.view(torch.int16 if t.element_size() == 2 else torch.int32 if t.element_size() == 4 else torch.int8)


def _turn(t):
    t.data = t.data.t()


# (what a call says of tensors off the GPU is said tensor by tensor: no values are right, then the next; else there is no data)
@pytest.mark.parametrize("name", ["p", "g", "m", "v"])
@pytest.mark.parametrize("change,code", [(_to_ints, "DTYPE"), (_turn, "LAYOUT")])
def test_type_and_order_at_the_same_address(bd, name, change, code):  # noqa: F811
    t = _tensors()
    for n in NAMES[:NAMES.index(name)]:
        t[n] = torch.empty(0, dtype=TYPES[n])                    # empty ones before it are passed over
    lists = {n: bd.TensorList([x]) for n, x in t.items()}
    with pytest.raises(bd.MoeError, match="NULL"):
        _step(bd, lists)
    at = t[name].data_ptr()
    change(t[name])
    assert t[name].data_ptr() == at
    with pytest.raises(bd.MoeError, match=code):
        _step(bd, lists)


def test_size_at_the_same_address(bd):  # noqa: F811
    t = _tensors()
    t["g"] = torch.zeros(4, 10, dtype=torch.int32)               # comes to light as soon as p is passed over
    lists = {n: bd.TensorList([x]) for n, x in t.items()}
    with pytest.raises(bd.MoeError, match="NULL"):
        _step(bd, lists)
    t["p"].resize_(0)
    with pytest.raises(bd.MoeError, match="DTYPE"):
        _step(bd, lists)
    t["p"].resize_(40)
    with pytest.raises(bd.MoeError, match="NULL"):
        _step(bd, lists)


def test_one_of_many(bd):  # noqa: F811
    t = _tensors((5, 2))
    lists = {n: bd.TensorList([torch.empty(0, dtype=TYPES[n]) for _ in range(300)] + [x]) for n, x in t.items()}
    for change, code in ((lambda: None, "NULL"), (lambda: _turn(t["p"]), "LAYOUT"), (lambda: _to_ints(t["p"]), "DTYPE")):
        change()
        with pytest.raises(bd.MoeError, match=code):
            _step(bd, lists)


def test_a_norm_whose_workspace_is_on_another_device(bd):  # noqa: F811
    """The call runs on the gradients' device, which would write to another one's memory."""
    ws = bd.Workspace(1024, device="cpu")
    with pytest.raises(ValueError, match="devices"):
        bd.moe_grad_norm([], torch.empty(2, device="meta"), ws, stream=0)
    with pytest.raises(bd.MoeError, match="NULL"):               # here nothing is on a GPU
        bd.moe_grad_norm([], torch.empty(2), ws, stream=0)
