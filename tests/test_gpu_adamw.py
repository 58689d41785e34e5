"""AdamW over many tensors and the norm of their gradients, against formulas in 64 bits.

Bounds.  m' is two products and a sum: each rounds by half a last place (2^-24) of its size, so 2^-24 (2 |b1 m| + 2 |c1 g|)
covers them and b1's, c1's own rounding adds as much again; v' likewise, with the square's rounding: 2^-24 of 5 terms.
p' rounds once, 2^-24 |p'|, and its step u = mhat / (root + eps) carries m's relative error, v's half, those of the two
factors (rounded to fp32) and of a quotient of 2 last places: 12 x 2^-24 of (|b1 m| + |c1 g|) / (root + eps), and lr's and
decay's roundings 3 x 2^-24 of lr (|u| + decay |p|).  The scale of gradients adds a rounding of g.  bf16: 2^-8.
8 bits: a decoded state is code x scale with one rounding; a code is off by less than one step of E4M3, 2^-3 of the value
or 2^-9 of 448ths of the largest, and the scale by 2^-23."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 256
U = 2.0 ** -24


def make(sizes, grad, copy, seed, state=32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"p": [], "g": [], "m": [], "v": [], "copy": [], "ms": [], "vs": []}
    for i, n in enumerate(sizes):
        level = 10.0 ** (-(i % 4))
        t["p"].append(torch.randn(n, generator=g, device="cuda") * 0.05)
        kind = grad if grad != "both" else ("f32", "bf16")[i % 2]
        t["g"].append((torch.randn(n, generator=g, device="cuda") * level).to(torch.bfloat16 if kind == "bf16" else torch.float32))
        m, v = torch.randn(n, generator=g, device="cuda") * 0.3 * level, (torch.rand(n, generator=g, device="cuda") * level).square()
        if state == 8:
            for x, c, s in ((m, "m", "ms"), (v.sqrt(), "v", "vs")):
                rows = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
                scale = rows.abs().amax(1) / 448
                code = (rows / scale.clamp(min=1e-30)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1)[:n]
                t[c].append(code.contiguous())
                t[s].append(scale.contiguous())
        else:
            t["m"].append(m)
            t["v"].append(v)
        t["copy"].append(torch.empty(n, dtype=torch.bfloat16, device="cuda"))
    if not copy:
        t["copy"] = None
    return t


def decode(code, scale):
    n = code.numel()
    return code.double().cpu() * scale.double().cpu().repeat_interleave(BLOCK)[:n]


def step64(p, g, m, v, h):
    """p', m', v' and bounds of p', m', v' for one tensor; everything in 64 bits."""
    b1, b2 = h["betas"]
    g = g.double().cpu() * h.get("scale", 1.0)
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    um, uv = 4 * U * ((b1 * m).abs() + ((1 - b1) * g).abs()), 6 * U * (b2 * v + (1 - b2) * g * g) + 1e-44
    root = torch.sqrt(v2 / (1 - b2 ** h["step"])) + h["eps"]
    u = m2 / (1 - b1 ** h["step"]) / root
    p2 = p - h["lr"] * (u + h["weight_decay"] * p)
    size = ((b1 * m).abs() + ((1 - b1) * g).abs()) / (1 - b1 ** h["step"]) / root
    up = U * p2.abs() + h["lr"] * U * (14 * size + 4 * h["weight_decay"] * p.abs() + 2 * u.abs()) + 1e-44
    return p2, m2, v2, up, um, uv


def run(moe, t, h, state, **kw):
    moe.moe_adamw_step(t["p"], t["g"], t["m"], t["v"], kw.pop("step", h["step"]), lr=kw.pop("lr", h["lr"]), betas=h["betas"], eps=h["eps"],
                       weight_decay=h["weight_decay"], m_scales=t["ms"] if state == 8 else None, v_scales=t["vs"] if state == 8 else None,
                       copies=t["copy"], **kw)


H = {"lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1, "step": 7}
LISTS = [[1], [255, 256, 257], [0, 3, 0, 1000, 0], [4097] * 5, [70_001, 5, 260, 1], list(range(1, 60)), [33] * 400, [1 + (i * 37) % 700 for i in range(900)]]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("grad", ["f32", "bf16", "both"])
@pytest.mark.parametrize("copy", [False, True])
def test_states_in_32_bits(cuda_lib, sizes, grad, copy):
    t = make(sizes, grad, copy, len(sizes))
    before = [[x.double().cpu() for x in t[n]] for n in "pmv"]
    for h in (H, {**H, "step": 1, "lr": 0.02, "betas": (0.0, 0.9), "eps": 1e-3, "weight_decay": 0.0}):
        run(cuda_lib, t, h, 32)
        for i, n in enumerate(sizes):
            p2, m2, v2, up, um, uv = step64(before[0][i], t["g"][i], before[1][i], before[2][i], h)
            p = t["p"][i].double().cpu()
            assert ((t["m"][i].double().cpu() - m2).abs() <= um).all()
            assert ((t["v"][i].double().cpu() - v2).abs() <= uv).all()
            assert ((p - p2).abs() <= up).all()
            if copy:
                assert torch.equal(t["copy"][i], t["p"][i].to(torch.bfloat16))
        before = [[x.double().cpu() for x in t[n]] for n in "pmv"]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("grad", ["f32", "both"])
def test_states_in_8_bits(cuda_lib, sizes, grad):
    t = make(sizes, grad, True, 3 + len(sizes), state=8)
    for step in (1, 2):
        h = {**H, "step": step}
        p0 = [x.double().cpu() for x in t["p"]]
        m0 = [decode(c, s) for c, s in zip(t["m"], t["ms"])]
        r0 = [decode(c, s) for c, s in zip(t["v"], t["vs"])]
        run(cuda_lib, t, h, 8, seed=step)
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            # (decoding rounds once: 2^-24 of m, twice that of v, and of its square)
            p2, m2, v2, up, um, uv = step64(p0[i], t["g"][i], m0[i], r0[i] ** 2, h)
            assert ((t["p"][i].double().cpu() - p2).abs() <= 1.5 * up).all()
            assert torch.equal(t["copy"][i], t["p"][i].to(torch.bfloat16))
            r2 = v2.sqrt()
            for x, ux, code, scale, least in ((m2, um, t["m"][i], t["ms"][i], 0), (r2, uv / (2 * r2.clamp(min=1e-22)) + 2 * U * r2, t["v"][i], t["vs"][i], 1)):
                # a block's largest value is as far off as its values are, which where b1 m and c1 g cancel is more than its
                # own last places (um: 2^-24 of the terms); r = sqrt(v) has half of v's relative error and a rounding; then two
                # roundings of the scale
                rows = lambda y: torch.nn.functional.pad(y, (0, -n % BLOCK)).view(-1, BLOCK).abs().amax(1)  # noqa: E731
                most = rows(x)
                assert ((scale.double().cpu() * 448 - most).abs() <= rows(ux) + 4 * U * most).all()
                got = decode(code, scale)
                per = (most / 448).repeat_interleave(BLOCK)[:n]
                y = x.abs() / per
                grid = torch.maximum(2.0 ** (torch.floor(torch.log2(y.clamp(min=2.0 ** -9))) - 3), torch.tensor(2.0 ** -9, dtype=torch.float64))
                slack = torch.maximum(grid, torch.full_like(grid, least * 2.0 ** -9)) * (1 + 1e-5) + 1e-5 * y
                assert ((got - x).abs() <= slack * per + ux + rows(ux).repeat_interleave(BLOCK)[:n]).all()
                assert (code.view(torch.uint8) & 127 != 127).all()
                if least:
                    assert (code.view(torch.uint8) >= 1).all()


def test_rounding_is_exact_in_the_mean(cuda_lib):
    """Over many seeds codes average to the value: the mean of N roundings of a step q is off by 5 standard errors,
    5 q / (2 sqrt N), at most (16 bits of noise add 2^-17 q)."""
    n, N = 2048, 600
    g = torch.Generator(device="cuda").manual_seed(1)
    grad = torch.randn(n, generator=g, device="cuda")
    sums = [torch.zeros(n, dtype=torch.float64) for _ in range(2)]
    for seed in range(N):
        p = torch.zeros(n, device="cuda")
        m, v = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
        ms, vs = torch.zeros(n // BLOCK, device="cuda"), torch.zeros(n // BLOCK, device="cuda")
        cuda_lib.moe_adamw_step([p], [grad], [m], [v], 1, m_scales=[ms], v_scales=[vs], seed=seed)
        for s, c, sc in zip(sums, (m, v), (ms, vs)):
            s += decode(c.view(torch.float8_e4m3fn), sc)
    for s, x in zip(sums, (0.1 * grad.double().cpu(), math.sqrt(0.001) * grad.double().cpu().abs())):
        per = x.view(-1, BLOCK).abs().amax(1).repeat_interleave(BLOCK) / 448
        y = x.abs() / per
        q = torch.maximum(2.0 ** (torch.floor(torch.log2(y.clamp(min=1e-9))) - 3), torch.tensor(2.0 ** -9, dtype=torch.float64))
        low = y < 2.0 ** -9        # (r's smallest code)
        assert (((s / N - x).abs() <= per * q * (5 / (2 * math.sqrt(N)) + 2e-5) + 1e-6 * x.abs()) | low).all()


def test_8_bit_states_follow_32_bit_ones(cuda_lib):
    """v grows and falls with its gradients, as it could not by rounding to nearest (3000 steps of level 1, 2000 of 0.25).
    Rounding leaves r's mean as it is and adds its variance q^2 f (1 - f) <= q d to v, q <= r / 8 a code's step and d how
    far r has come from a code: r came from one, and v's decay, the gradient and the block's scale move it against the codes
    by about 0.0005 r each in the mean, so v gains at most 0.0002 v a step where its memory is 0.001: 1 / (1 - 0.2) = 1.25
    times v, and with r's own spread under 1.5.  The mean over 4096 values has 1.6 % of a value's deviation, which is under
    its size: below 1 it may be by 5 %."""
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    p = [torch.zeros(n, device="cuda") for _ in range(2)]
    m8, v8 = (torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(n // BLOCK, device="cuda") for _ in range(2))
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    step = 0
    for level, steps in ((1.0, 3000), (0.25, 2000)):
        for _ in range(steps):
            step += 1
            grad = torch.randn(n, generator=g, device="cuda") * level
            cuda_lib.moe_adamw_step([p[0]], [grad], [m], [v], step, lr=1e-4)
            cuda_lib.moe_adamw_step([p[1]], [grad], [m8], [v8], step, lr=1e-4, m_scales=[ms], v_scales=[vs], seed=step)
        r8, r = decode(v8, vs), v.sqrt().double().cpu()
        ratio = float((r8 ** 2).mean() / (r ** 2).mean())
        print('level', level, 'v in 8 bits over v in 32:', ratio)
        assert 0.95 < ratio < 1.5


def test_noise_repeats_and_depends_on_the_seed_alone(cuda_lib):
    outs = []
    for seed in (5, 5, 6, 5 + (1 << 33)):
        t = make([1000, 300, 4000], "f32", True, 9, state=8)
        run(cuda_lib, t, H, 8, seed=seed)
        outs.append([x.clone() for n in ("p", "m", "v", "ms", "vs", "copy") for x in t[n]])
    same = lambda a, b: all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))  # noqa: E731
    assert same(outs[0], outs[1]) and not same(outs[0], outs[2]) and not same(outs[0], outs[3])


@pytest.mark.parametrize("state", [32, 8])
def test_scale_and_numbers_on_the_device(cuda_lib, state):
    h = {**H, "scale": 0.37}
    t, other = make([5000, 17], "both", True, 4, state), make([5000, 17], "both", True, 4, state)
    scale = torch.tensor([1.0, 0.37], device="cuda")[1:]
    run(cuda_lib, t, H, state, grad_scale=scale, seed=10)
    run(cuda_lib, other, H, state, grad_scale=scale, seed=3, step=torch.tensor([7], dtype=torch.int32, device="cuda"),
        lr=torch.tensor(1e-3, device="cuda"))
    for i in range(2):
        m0 = make([5000, 17], "both", True, 4, state)
        m, v = ((decode(m0["m"][i], m0["ms"][i]), decode(m0["v"][i], m0["vs"][i]) ** 2) if state == 8 else (m0["m"][i].double().cpu(), m0["v"][i].double().cpu()))
        h["scale"] = float(scale[0])
        p2, m2, v2, up, um, uv = step64(m0["p"][i].double().cpu(), m0["g"][i], m, v, h)
        assert ((t["p"][i].double().cpu() - p2).abs() <= 1.5 * up).all()
        # 1 - b^t from fp32's expm1: a few more last places in the step
        assert ((other["p"][i].double().cpu() - p2).abs() <= 1.5 * up + 8 * U * (p2 - m0["p"][i].double().cpu()).abs()).all()
        assert torch.equal(t["m"][i].view(torch.uint8), other["m"][i].view(torch.uint8))   # (3 + 7 is the other's seed)


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_no_step_without_a_finite_scale(cuda_lib, state, bad):
    t = make([1000, 3], "f32", True, 5, state)
    for c in t["copy"]:
        c.fill_(3)
    before = {n: [x.clone() for x in t[n]] for n in t}
    run(cuda_lib, t, H, state, grad_scale=torch.tensor([bad], device="cuda"))
    for n in t:
        for a, b in zip(before[n], t[n]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_blocks_of_nan_zeros_and_tiny_values(cuda_lib):
    n = 4 * BLOCK + 40
    g = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    g[300] = math.nan
    g[2 * BLOCK:3 * BLOCK] = 0
    g[3 * BLOCK:4 * BLOCK] = 1e-36
    p, m, v = torch.ones(n, device="cuda"), torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda")
    ms, vs = torch.zeros(5, device="cuda"), torch.zeros(5, device="cuda")
    for step in (1, 2):
        cuda_lib.moe_adamw_step([p], [g], [m], [v], step, m_scales=[ms], v_scales=[vs], seed=step)
        assert ms.isnan().tolist() == [False, True, False, False, False] and vs.isnan().tolist() == ms.isnan().tolist()
        assert ms[2] == 0 and ms[3] == 0 and vs[2] == 0 and (m.view(torch.uint8)[2 * BLOCK:4 * BLOCK] == 0).all()
        assert p[300].isnan() and torch.isfinite(p[2 * BLOCK:]).all() and torch.isfinite(p[:BLOCK]).all()
        assert torch.isfinite(decode(m, ms)[:BLOCK]).all()
        if step == 2:   # by then the whole block's states are lost
            assert p[BLOCK:2 * BLOCK].isnan().all()


def test_what_lies_between_the_tensors(cuda_lib):
    """Views of a few buffers with odd lengths: what is not theirs stays."""
    sizes, start = [1, 255, 257, 511, 40], [0, 64, 512, 1024, 2048]
    for state in (32, 8):
        flat = {"p": torch.full((4096,), 9.0, device="cuda"), "g": torch.full((4096,), 0.5, device="cuda"), "copy": torch.full((4096,), 9.0, device="cuda", dtype=torch.bfloat16)}
        for n in "mv":
            flat[n] = torch.full((4096,), 9, device="cuda", dtype=torch.uint8 if state == 8 else torch.float32)
        flat["ms"], flat["vs"] = torch.full((32,), 9.0, device="cuda"), torch.full((32,), 9.0, device="cuda")
        t = {n: [flat[n][a:a + k] for a, k in zip(start, sizes)] for n in ("p", "g", "m", "v", "copy")}
        t["ms"] = [flat["ms"][5 * i + 1:5 * i + 1 + -(-k // BLOCK)] for i, k in enumerate(sizes)]
        t["vs"] = [flat["vs"][5 * i + 1:5 * i + 1 + -(-k // BLOCK)] for i, k in enumerate(sizes)]
        run(cuda_lib, t, H, state)
        theirs = torch.zeros(4096, dtype=torch.bool, device="cuda")
        for a, k in zip(start, sizes):
            theirs[a:a + k] = True
        for n in ("p", "copy", "m", "v"):
            assert (flat[n][~theirs] == 9).all()
        if state == 8:
            of = torch.zeros(32, dtype=torch.bool, device="cuda")
            for i, k in enumerate(sizes):
                of[5 * i + 1:5 * i + 1 + -(-k // BLOCK)] = True
            assert (flat["ms"][~of] == 9).all() and (flat["vs"][~of] == 9).all() and (flat["ms"][of] != 9).all()


def test_lists_follow_their_tensors(cuda_lib):
    """A TensorList whose tensor has got other memory writes there."""
    p = torch.zeros(1000, device="cuda")
    g, m, v = torch.ones(1000, device="cuda"), torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda")
    lists = [cuda_lib.TensorList([x]) for x in (p, g, m, v)]
    cuda_lib.moe_adamw_step(*lists, 1, lr=0.5)
    old = p.data
    kept = old.clone()
    p.data = torch.full((1000,), 2.0, device="cuda")
    cuda_lib.moe_adamw_step(*lists, 2, lr=0.5)
    assert torch.equal(old, kept) and (p < 2).all()


@pytest.mark.parametrize("sizes", LISTS + [[3_000_000, 17, 1]], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("grad", ["f32", "both"])
def test_norm(cuda_lib, sizes, grad):
    """64 squares in 32 bits: at most 2^-24 (64 + 1) of their sum, half of it in the root, then the rounding."""
    t = make(sizes, grad, False, 8)
    elements = sum(sizes)
    ws = cuda_lib.Workspace(cuda_lib.moe_grad_norm_workspace_bytes(elements, len(sizes)))
    out = torch.empty(2, device="cuda")
    want = math.sqrt(sum(float(x.double().square().sum()) for x in t["g"]))
    got = []
    for most in (0.0, want / 3, want * 2):
        cuda_lib.moe_grad_norm(t["g"], out, ws, max_norm=most)
        norm, factor = out.tolist()
        assert abs(norm - want) <= 34 * U * want
        assert abs(factor - (1.0 if most == 0 else min(1.0, most / want))) <= 36 * U
        got.append(norm)
    assert got[0] == got[1] == got[2]
    assert cuda_lib.moe_read_device_status(ws) == 0


def test_norms_that_are_none(cuda_lib):
    ws = cuda_lib.Workspace(cuda_lib.moe_grad_norm_workspace_bytes(2000, 2))
    out = torch.empty(2, device="cuda")
    for value in (math.nan, math.inf, 1e25):
        g = torch.ones(1000, device="cuda")
        g[777] = value
        cuda_lib.moe_grad_norm([torch.ones(5, device="cuda"), g], out, ws, max_norm=1.0)
        assert out[1].isnan() and not torch.isfinite(out[0])
    cuda_lib.moe_grad_norm([], out, ws, max_norm=1.0)
    assert out.tolist() == [0.0, 1.0]
    cuda_lib.moe_grad_norm([torch.zeros(100, device="cuda")], out, ws, max_norm=1.0)
    assert out.tolist() == [0.0, 1.0]
    cuda_lib.moe_grad_norm([torch.empty(0, device="cuda")], out, ws)
    assert out.tolist() == [0.0, 1.0]


def test_workspaces_of_other_calls(cuda_lib):
    ws = cuda_lib.Workspace(1 << 20)
    out = torch.empty(2, device="cuda")
    logits, idx = torch.randn(100, 8, device="cuda"), torch.zeros(100, 2, dtype=torch.int32, device="cuda")
    counts, tokens, loss = torch.empty(1, 8, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, 2, device="cuda")
    cuda_lib.moe_balance_fwd(logits, idx, counts, tokens, loss, ws)        # leaves zeros
    cuda_lib.moe_grad_norm([torch.ones(16, device="cuda")], out, ws)
    assert out[0] == 4
    with pytest.raises(cuda_lib.MoeError, match="STATE"):
        cuda_lib.moe_balance_fwd(logits, idx, counts, tokens, loss, ws)
    cuda_lib.moe_orthogonalise(torch.randn(1, 8, 8, device="cuda"), torch.empty(1, 8, 8, dtype=torch.bfloat16, device="cuda"), ws)
    with pytest.raises(cuda_lib.MoeError, match="STATE"):
        cuda_lib.moe_grad_norm([torch.ones(16, device="cuda")], out, ws)


@pytest.mark.parametrize("state", [32, 8])
def test_clipped_step_on_a_stream_and_in_a_graph(cuda_lib, state):
    """Norm and step as a training loop has them: eager, on another stream, replayed."""
    moe = cuda_lib
    sizes = [4000, 1, 300, 50_000]
    results = []
    for way in ("eager", "stream", "graph"):
        t = make(sizes, "both", True, 11, state)
        names = ("p", "g", "m", "v") + (("ms", "vs") if state == 8 else ())
        lists = {n: moe.TensorList(t[n]) for n in names}
        ws, out = moe.Workspace(moe.moe_grad_norm_workspace_bytes(sum(sizes), 4)), torch.empty(2, device="cuda")
        step = torch.zeros(1, dtype=torch.int32, device="cuda")

        def once():
            step.add_(1)
            moe.moe_grad_norm(lists["g"], out, ws, max_norm=1.0)
            moe.moe_adamw_step(lists["p"], lists["g"], lists["m"], lists["v"], step, lr=1e-2, m_scales=lists.get("ms"), v_scales=lists.get("vs"),
                               copies=t["copy"], grad_scale=out[1:], seed=77)
        torch.cuda.synchronize()
        if way == "eager":
            for _ in range(3):
                once()
        elif way == "stream":
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                for _ in range(3):
                    once()
            side.synchronize()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                once()
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        results.append([x.clone().view(torch.uint8) for n in names + ("copy",) for x in t[n]] + [out.clone().view(torch.uint8)])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)


def test_long_tensor(cuda_lib):
    """Positions past 2^31 bytes and 2^29 values, both ends looked at."""
    n = (1 << 29) + 1001
    p, g, m, v = torch.full((n,), 0.5, device="cuda"), torch.full((n,), 2.0, device="cuda", dtype=torch.bfloat16), torch.zeros(n, device="cuda", dtype=torch.uint8), torch.zeros(n, device="cuda", dtype=torch.uint8)
    ms, vs = torch.zeros(-(-n // BLOCK), device="cuda"), torch.zeros(-(-n // BLOCK), device="cuda")
    cuda_lib.moe_adamw_step([p], [g], [m], [v], 1, lr=0.125, m_scales=[ms], v_scales=[vs])
    ws, out = cuda_lib.Workspace(cuda_lib.moe_grad_norm_workspace_bytes(n, 1)), torch.empty(2, device="cuda")
    cuda_lib.moe_grad_norm([g], out, ws)
    # the step of a first gradient is lr exactly but for eps and roundings
    assert float((p - 0.375).abs().max()) < 1e-6
    assert (m == 126).all() and (v == 126).all()
    assert abs(float(out[0]) - 2 * math.sqrt(n)) <= 36 * U * 2 * math.sqrt(n)
