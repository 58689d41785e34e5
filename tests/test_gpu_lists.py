"""Lists whose tensors change between calls: each call steps what they are by then, and nothing beside it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 256


def _state(n, state, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"p": torch.randn(n, generator=g, device="cuda"), "g": torch.randn(n, generator=g, device="cuda")}
    for k in ("m", "v"):
        t[k] = torch.zeros(n, device="cuda", dtype=torch.uint8 if state == 8 else torch.float32)
    for k in ("ms", "vs"):
        t[k] = torch.zeros(-(-n // BLOCK), device="cuda")
    t["copy"] = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    return t


def _step(moe, lists, state, step=1):
    moe.moe_adamw_step(lists["p"], lists["g"], lists["m"], lists["v"], step, m_scales=lists["ms"] if state == 8 else None,
                       v_scales=lists["vs"] if state == 8 else None, copies=lists["copy"], seed=step)


@pytest.mark.parametrize("state", [32, 8])
def test_tensors_that_shrink_and_grow_at_their_address(cuda_lib, state):
    n, some = 5000, 1000
    t, want = _state(n, state), _state(n, state)
    whole = {k: x.data for k, x in t.items()}
    lists = {k: cuda_lib.TensorList([x]) for k, x in t.items()}
    _step(cuda_lib, lists, state)
    _step(cuda_lib, {k: [x] for k, x in want.items()}, state)
    for step, size in ((2, some), (3, n)):
        before = {k: x.clone() for k, x in whole.items()}
        for k, x in t.items():
            at, m = x.data_ptr(), -(-size // BLOCK) if k in ("ms", "vs") else size
            x.data = whole[k][:m]
            assert x.data_ptr() == at
        _step(cuda_lib, lists, state, step)
        _step(cuda_lib, {k: [x[:t[k].numel()]] for k, x in want.items()}, state, step)
        for k in whole:
            m = t[k].numel()
            assert torch.equal(whole[k][m:].view(torch.uint8), before[k][m:].view(torch.uint8))
            assert torch.equal(whole[k].view(torch.uint8), want[k].view(torch.uint8))


def test_gradients_of_another_type_at_their_address(cuda_lib):
    n = 3000
    t = _state(n, 32)
    room = t["g"].data
    lists = {k: cuda_lib.TensorList([x]) for k, x in t.items()}
    ws, out = cuda_lib.Workspace(cuda_lib.moe_grad_norm_workspace_bytes(n, 1)), torch.empty(2, device="cuda")
    _step(cuda_lib, lists, 32)
    half = room.to(torch.bfloat16)
    t["g"].data = room.view(torch.bfloat16)[:n]
    t["g"].copy_(half)
    want = {k: x.clone() for k, x in t.items()}
    _step(cuda_lib, lists, 32, 2)
    _step(cuda_lib, {k: [x] for k, x in want.items()}, 32, 2)
    for k in ("p", "m", "v", "copy"):
        assert torch.equal(t[k], want[k])
    cuda_lib.moe_grad_norm(lists["g"], out, ws)
    # (64 squares and their sums in 32 bits, half of that in the root, a rounding)
    want_norm = float(half.double().square().sum().sqrt())
    assert abs(float(out[0]) - want_norm) <= 34 * 2.0 ** -24 * want_norm


def test_tensors_that_come_to_the_gpu(cuda_lib):
    t = {k: x.cpu() for k, x in _state(700, 32).items()}
    lists = {k: cuda_lib.TensorList([x]) for k, x in t.items()}
    with pytest.raises(cuda_lib.MoeError, match="NULL"):
        _step(cuda_lib, lists, 32)
    for x in t.values():
        x.data = x.data.cuda()
    want = {k: x.clone() for k, x in t.items()}
    _step(cuda_lib, lists, 32)
    _step(cuda_lib, {k: [x] for k, x in want.items()}, 32)
    for k in ("p", "m", "v", "copy"):
        assert torch.equal(t[k], want[k])


@pytest.mark.parametrize("most", [1e-30, 1e-44, 1e-50, 1e-300])
def test_a_norm_clipped_to_next_to_nothing(cuda_lib, most):
    """A max_norm below the numbers of fp32 still clips; only 0 does not.  The factor is most / 4, off by a rounding of the
    quotient and of max_norm: 2^-23 of it, or two of the smallest steps, 2^-148."""
    grads = [torch.ones(16, device="cuda")]
    ws, out = cuda_lib.Workspace(cuda_lib.moe_grad_norm_workspace_bytes(16, 1)), torch.empty(2, device="cuda")
    cuda_lib.moe_grad_norm(grads, out, ws, max_norm=most)
    assert float(out[0]) == 4 and abs(float(out[1]) - most / 4) <= 2.0 ** -23 * most / 4 + 2.0 ** -148
    cuda_lib.moe_grad_norm(grads, out, ws, max_norm=0.0)
    assert out.tolist() == [4.0, 1.0]
