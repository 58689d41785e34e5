"""8-bit AdamW states over many steps."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 256


def _zeros(n):
    codes = [torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    return codes + [torch.zeros(-(-n // BLOCK), device="cuda") for _ in range(2)]


def _decode(code, scale):
    return code.double() * scale.double().repeat_interleave(BLOCK)[:code.numel()]


@pytest.mark.parametrize("on_device", [False, True])
def test_states_move_without_a_seed(cuda_lib, on_device):
    """v follows its gradients up and down where no seed is given.  Bounds as with one (test_gpu_adamw.py): v gains the variance of
    its root's rounding, 1.25 times it and under 1.5, and may be 5 % lower by chance."""
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    p = [torch.zeros(n, device="cuda") for _ in range(2)]
    m8, v8, ms, vs = _zeros(n)
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    number, step = torch.zeros(1, dtype=torch.int32, device="cuda"), 0
    for level, steps in ((1.0, 3000), (0.25, 2000)):
        for _ in range(steps):
            step += 1
            number.add_(1)
            grad = torch.randn(n, generator=g, device="cuda") * level
            cuda_lib.moe_adamw_step([p[0]], [grad], [m], [v], step, lr=1e-4)
            cuda_lib.moe_adamw_step([p[1]], [grad], [m8], [v8], number if on_device else step, lr=1e-4, m_scales=[ms], v_scales=[vs])
        assert 0.95 < float((_decode(v8, vs) ** 2).mean() / v.double().mean()) < 1.5


def test_without_a_seed_a_step_is_the_same_from_the_host_and_the_device(cuda_lib):
    n = 3001
    grad = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    codes = []
    for step in (41, torch.tensor([41], dtype=torch.int32, device="cuda"), 42):
        m8, v8, ms, vs = _zeros(n)
        cuda_lib.moe_adamw_step([torch.zeros(n, device="cuda")], [grad], [m8], [v8], step, m_scales=[ms], v_scales=[vs])
        codes.append([x.view(torch.uint8) for x in (m8, v8)])
    assert all(torch.equal(a, b) for a, b in zip(codes[0], codes[1]))
    assert not any(torch.equal(a, b) for a, b in zip(codes[0], codes[2]))


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("number", [0, -1, -2 ** 31])
def test_no_step_below_the_first(cuda_lib, state, number):
    """A step's number on the device cannot be refused by the call: it leaves everything as it is."""
    n = 1000
    g = torch.Generator(device="cuda").manual_seed(4)
    t = {k: torch.randn(n, generator=g, device="cuda") for k in ("p", "g")}
    m, v, ms, vs = _zeros(n)
    if state == 32:
        m, v = torch.rand(n, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    t.update(m=m, v=v, ms=ms, vs=vs, copy=torch.full((n,), 3.0, dtype=torch.bfloat16, device="cuda"))
    before = {k: x.clone() for k, x in t.items()}
    step = torch.tensor([number], dtype=torch.int32, device="cuda")
    cuda_lib.moe_adamw_step([t["p"]], [t["g"]], [m], [v], step, m_scales=[ms] if state == 8 else None, v_scales=[vs] if state == 8 else None,
                            copies=[t["copy"]])
    for k in t:
        assert torch.equal(before[k].view(torch.uint8), t[k].view(torch.uint8))
