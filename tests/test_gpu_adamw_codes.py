"""8-bit AdamW states bit for bit: codes and scales against the formulas, restated with numpy's correctly rounded 32-bit
products, sums, quotients and roots, a code as a whole number of steps, and the noise in whole numbers.  Nothing is
within a tolerance here: every operation is a single rounding to nearest, or exact."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 256
F = np.float32


def noise(seed, ordinal, n):
    """32 bits for each value of the list's tensor `ordinal`."""
    low = np.uint64(0xFFFFFFFF)
    place = np.arange(n, dtype=np.uint64)
    h = (place * np.uint64(0x9E3779B1) + np.uint64((seed ^ (seed >> 32)) & 0xFFFFFFFF) + np.uint64((ordinal + 1) * 0x85EBCA77)) & low
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        h = ((h ^ (h >> np.uint64(shift))) * np.uint64(factor)) & low
    return h ^ (h >> np.uint64(16))


def values(code):
    """E4M3: sign, four bits of exponent (bias 7), three of mantissa."""
    e, f = ((code >> 3) & 15).astype(np.int64), (code & 7).astype(np.float64)
    x = np.where(e > 0, np.ldexp(1 + f / 8, e - 7), f / 512)
    return np.where(code & 128, -x, x).astype(F)


def blocks(x):
    return np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK)


def steps(t):
    """How many codes t is above 0, with 20 bits behind the point: those that fp32's mantissa has past E4M3's three, and under
    2^-6, where codes are 2^-9 apart, t rounded to as many."""
    t = t.astype(np.float64)
    e = np.floor(np.log2(np.maximum(t, 2.0 ** -20)))
    large = (e + 7) * 8 + (t / 2.0 ** e - 1) * 8
    return np.where(t >= 2.0 ** -6, large, np.rint(t * 2.0 ** 29) / 2.0 ** 20)


def encode(x, bits, least):
    """Codes without a sign, and scales, of x >= 0 by the 16 bits for each value."""
    most = blocks(x).max(1)
    most = np.where(most < F(1e-35), F(0), most)
    with np.errstate(divide="ignore"):
        up = np.where(most > 0, (F(1) / most) * F(448), F(0))
    t = x * np.repeat(up, BLOCK)[:len(x)]
    code = np.floor(steps(t) + (bits.astype(np.float64) * 16 + 8) / 2.0 ** 20).clip(least, 126).astype(np.uint8)
    return np.where(np.repeat(up, BLOCK)[:len(x)] > 0, code, np.uint8(0)), most * (F(1) / F(448)), np.repeat(up, BLOCK)[:len(x)] > 0


def step(g, scale, m, ms, v, vs, ordinal, seed, b1=0.9, b2=0.999):
    n = len(g)
    g = g * F(scale)
    m = (values(m) * np.repeat(ms, BLOCK)[:n]) * F(b1) + g * F(1 - b1)
    r = values(v) * np.repeat(vs, BLOCK)[:n]
    r = np.sqrt((r * r) * F(b2) + (g * g) * F(1 - b2))
    assert m.dtype == r.dtype == F
    h = noise(seed, ordinal, n)
    cm, ms, some = encode(np.abs(m), h & np.uint64(0xFFFF), 0)
    cv, vs, _ = encode(r, h >> np.uint64(16), 1)
    return np.where(some & np.signbit(m), cm | 128, cm).astype(np.uint8), ms, cv, vs


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seed", [1, 2 ** 32 - 1, 5 + (9 << 33)])
def test_codes_and_scales(cuda_lib, grad, seed):
    """Three steps of several tensors, whole and partial blocks, uneven sizes of gradients, blocks of zeros and next to nothing,
    a factor of the gradients; each step starts from what the one before has left."""
    rng = np.random.default_rng(seed % 1000)
    sizes = [1, 255, 256, 1000, 0, 5000, 70_001]
    t = {"p": [torch.zeros(n, device="cuda") for n in sizes], "m": [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes],
         "v": [torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda").view(torch.uint8) for n in sizes]}
    for k in ("ms", "vs"):
        t[k] = [torch.zeros(-(-n // BLOCK), device="cuda") for n in sizes]
    factor = torch.tensor([0.37], device="cuda")
    want = [(np.zeros(n, np.uint8), np.zeros(-(-n // BLOCK), F)) * 2 for n in sizes]
    for number in (1, 2, 3):
        grads = []
        for i, n in enumerate(sizes):
            level = np.repeat(10.0 ** rng.uniform(-6, 3, -(-n // BLOCK)), BLOCK)[:n]
            g = rng.standard_normal(n) * level * np.exp(rng.standard_normal(n))
            if i == 5:
                g[:BLOCK], g[BLOCK:2 * BLOCK], g[2 * BLOCK:3 * BLOCK:2] = 0, 1e-37, 0
            grads.append(torch.tensor(g, dtype=torch.float32).to(grad).cuda())
        cuda_lib.moe_adamw_step(t["p"], grads, t["m"], t["v"], number, m_scales=t["ms"], v_scales=t["vs"], grad_scale=factor, seed=seed)
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            want[i] = step(grads[i].float().cpu().numpy(), 0.37, *want[i], i, seed)
            for k, x in zip(("m", "ms", "v", "vs"), want[i]):
                assert np.array_equal(t[k][i].cpu().numpy(), x), (number, i, k)
    moved = want[6][0]
    assert len(np.unique(moved)) > 200 and len(np.unique(want[6][2])) > 100      # most codes of either sign come up
