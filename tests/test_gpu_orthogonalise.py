"""Newton-Schulz orthogonalisation against the same steps in 64 bits.

Bar: 5e-3 relative 2-norm for a matrix: three times bf16's own rounding of the result (1.7e-3); the
fp16 operands (unit roundoff 4.9e-4) enter A, B and X once a step each and the last step's a, b, c
weigh them with about 3, which adds as much again."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAR = 5e-3
MUON = (3.4445, -4.7750, 2.0315)


def exact(G, steps=5, coeffs=MUON, eps=1e-7):
    """fp64, one matrix at a time; coeffs one triple or one for each step."""
    G = G.detach().double().cpu()
    per = [coeffs] * steps if not hasattr(coeffs[0], "__len__") else coeffs
    out = []
    for g in G:
        x = g / (g.norm() + eps)
        x = x.T if g.shape[0] > g.shape[1] else x
        for a, b, c in per:
            A = x @ x.T
            x = a * x + b * (A @ x) + c * (A @ (A @ x))
        out.append(x.T if g.shape[0] > g.shape[1] else x)
    return torch.stack(out)


def run(bd, G, O=None, **kw):
    O = torch.full(G.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if O is None else O
    ws = bd.Workspace(bd.moe_orthogonalise_workspace_bytes(*G.shape))
    ws.buffer[256:].fill_(0xFF)                  # NaNs wherever a kernel might read what it did not write
    bd.moe_orthogonalise(G, O, ws, **kw)
    assert bd.moe_read_device_status(ws) == 0
    return O


def errors(O, ref):
    o = O.double().cpu()
    return [float((a - b).norm() / max(float(b.norm()), 1e-300)) for a, b in zip(o, ref)]


def gauss(N, R, C, dtype, seed=0, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(N, R, C, generator=g)).to(dtype).cuda()


SHAPES = [(1, 1, 1), (2, 1, 5), (2, 3, 1), (3, 2, 200), (1, 16, 16), (2, 24, 40), (9, 52, 100), (1, 64, 64), (2, 100, 300),
          (1, 128, 128), (1, 128, 2048), (3, 129, 127), (2, 127, 1000), (2, 130, 257), (1, 192, 640), (1, 640, 192),
          (2, 256, 256), (1, 257, 255), (1, 384, 385), (5, 256, 128), (1, 777, 300), (1, 1030, 520), (40, 8, 70),
          (1, 60, 1500), (2, 2048, 100), (1, 1025, 128), (2, 100, 2100), (1, 2056, 24), (70, 260, 300),
          (330, 150, 140), (1, 128, 4096), (2, 3000, 65), (1, 4104, 30), (90, 100, 600), (2, 16, 2048), (2, 10, 2049),
          (3, 7, 20000), (2, 32, 1000), (1, 32, 16000), (1, 33, 1030), (2, 64, 512), (2, 5000, 61), (1, 17, 257), (1, 1, 32768)]


@pytest.mark.parametrize("N,R,C", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random_matrices(cuda_lib, N, R, C, dtype):
    G = gauss(N, R, C, dtype, seed=R * 7 + C)
    assert max(errors(run(cuda_lib, G), exact(G))) < BAR


@pytest.mark.parametrize("R,C", [(200, 320), (512, 300)])
@pytest.mark.parametrize("kind", ["rank", "decay"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_of_low_rank(cuda_lib, R, C, kind, dtype):
    """Few tokens (rank 24 and noise) and singular values that fall as 1 / i."""
    g = torch.Generator().manual_seed(3)
    if kind == "rank":
        G = torch.randn(2, R, 24, generator=g) @ torch.randn(2, 24, C, generator=g) + 0.02 * torch.randn(2, R, C, generator=g)
    else:
        m = min(R, C)
        U = torch.linalg.qr(torch.randn(2, R, m, generator=g))[0]
        V = torch.linalg.qr(torch.randn(2, C, m, generator=g))[0]
        G = U * (1 / torch.arange(1, m + 1.0)) @ V.transpose(1, 2)
    G = G.to(dtype).cuda()
    assert max(errors(run(cuda_lib, G), exact(G))) < BAR


def test_singular_values_and_flip(cuda_lib):
    G = gauss(2, 160, 400, torch.float32, 5)
    O, F = run(cuda_lib, G), run(cuda_lib, G.transpose(1, 2).contiguous())
    sv = torch.linalg.svdvals(O.double().cpu())
    assert float(sv.min()) > 0.5 and float(sv.max()) < 1.35
    assert max(errors(F.transpose(1, 2), O.double().cpu())) < 2 * BAR


@pytest.mark.parametrize("steps", [1, 2, 3, 12])
def test_steps_and_coefficients(cuda_lib, steps):
    """(3/2, -1/2, 0) converges to the nearest orthogonal matrix; coefficients of each step's own."""
    G = gauss(2, 96, 150, torch.float32, 6)
    cubic = (1.5, -0.5, 0.0)
    assert max(errors(run(cuda_lib, G, steps=steps, coeffs=cubic), exact(G, steps, cubic))) < BAR
    mixed = [(3.4445 - 0.1 * (i % 4), -4.7750 + 0.2 * (i % 4), 2.0315 - 0.1 * (i % 4)) for i in range(min(steps, 3))]
    assert max(errors(run(cuda_lib, G, steps=len(mixed), coeffs=mixed), exact(G, len(mixed), mixed))) < BAR


@pytest.mark.parametrize("scale", [1e-12, 1e-7, 1.0, 1e10])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,C", [(70, 90), (140, 150)])
def test_scales(cuda_lib, scale, dtype, R, C):
    """Down to norms that eps outweighs, and up."""
    G = gauss(2, R, C, dtype, 7, scale)
    assert max(errors(run(cuda_lib, G), exact(G))) < BAR
    assert max(errors(run(cuda_lib, G, eps=1e-3), exact(G, eps=1e-3))) < BAR


@pytest.mark.parametrize("R,C", [(80, 200), (300, 200)])
def test_zero_nan_and_infinite_matrices_stay_apart(cuda_lib, R, C):
    G = gauss(6, R, C, torch.float32, 8)
    G[1] = 0
    G[2, 5, 6] = float("nan")
    G[3, 0, 0] = float("inf")
    G[4] *= 1e25                                 # its squared norm leaves fp32
    O = run(cuda_lib, G)
    assert not O[1].float().abs().max()
    for i in (2, 3, 4):
        assert torch.isnan(O[i].float()).all()
    keep = [0, 5]
    assert max(errors(O[keep], exact(G[keep]))) < BAR


@pytest.mark.parametrize("R,C", [(60, 300), (300, 260)])
def test_in_place(cuda_lib, R, C):
    G = gauss(3, R, C, torch.bfloat16, 9)
    ref = exact(G)
    assert max(errors(run(cuda_lib, G, O=G), ref)) < BAR


def test_one_large_entry(cuda_lib):
    """The largest fp16 values: a matrix whose whole norm is one entry."""
    G = torch.zeros(1, 150, 170, device="cuda")
    G[0, 149, 0] = -3.0
    assert max(errors(run(cuda_lib, G), exact(G))) < BAR


def test_weights_of_the_layer(cuda_lib):
    """W13's gate and up halves as matrices of their own, by a view."""
    W = gauss(3, 2 * 128, 256, torch.float32, 10)
    O = torch.empty(3, 256, 256, dtype=torch.bfloat16, device="cuda")
    run(cuda_lib, W.view(6, 128, 256), O=O.view(6, 128, 256))
    assert max(errors(O.view(6, 128, 256), exact(W.view(6, 128, 256)))) < BAR


def test_no_matrices(cuda_lib):
    bd = cuda_lib
    ws = bd.Workspace(max(256, bd.moe_orthogonalise_workspace_bytes(0, 8, 8)))
    bd.moe_orthogonalise(torch.empty(0, 8, 8, device="cuda"), torch.empty(0, 8, 8, dtype=torch.bfloat16, device="cuda"), ws)


@pytest.mark.parametrize("N,R,C", [(2, 100, 140), (3, 300, 520), (70, 260, 300), (40, 700, 385), (9, 1000, 1300)])
def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph(cuda_lib, N, R, C):
    bd = cuda_lib
    G = gauss(N, R, C, torch.float32, 11)
    one = run(bd, G)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        two = run(bd, G)
    torch.cuda.synchronize()
    assert torch.equal(one, two)
    for _ in range(4):                           # tiles of one phase read by the next: the same bits however they fall
        assert torch.equal(one, run(bd, G))
    ws, O = bd.Workspace(bd.moe_orthogonalise_workspace_bytes(N, R, C)), torch.empty_like(one)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.moe_orthogonalise(G, O, ws)
    G.copy_(gauss(N, R, C, torch.float32, 12))
    g.replay()
    torch.cuda.synchronize()
    assert max(errors(O, exact(G))) < BAR


@pytest.mark.parametrize("N,R,C", [(2, 100, 140), (2, 300, 520)])
def test_waits_are_bounded(cuda_lib, N, R, C):
    """With no operand loads every wait runs out: a status code, and the next call works."""
    bd = cuda_lib
    G = gauss(N, R, C, torch.float32, 13)
    O = torch.empty(N, R, C, dtype=torch.bfloat16, device="cuda")
    ws = bd.Workspace(bd.moe_orthogonalise_workspace_bytes(N, R, C))
    ws.set_wait_limit(200000, bd.MOE_TEST_WITHHOLD_LOADS)
    bd.moe_orthogonalise(G, O, ws)
    assert bd.moe_read_device_status(ws) == bd.MOE_DEV_TIMEOUT
    ws.set_wait_limit()
    bd.moe_orthogonalise(G, O, ws)
    assert bd.moe_read_device_status(ws) == 0
    assert max(errors(O, exact(G))) < BAR


@pytest.mark.parametrize("N,R,C", [(5, 7, 513), (3, 513, 7), (4, 33, 255), (9, 255, 33), (3, 127, 771), (7, 1, 3), (7, 3, 1),
                                   (2, 5, 2), (11, 31, 33), (2, 1021, 61), (3, 65, 2047), (3, 2047, 65), (2, 131, 263)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_off_16_bytes_between_guards(cuda_lib, N, R, C, dtype):
    """Matrices and rows that begin anywhere: nothing beside O is written, and O may be G itself."""
    G, n = gauss(N, R, C, dtype, seed=R + 3 * C), N * R * C
    ref = exact(G)
    buf = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    assert max(errors(run(cuda_lib, G, O=buf[8:8 + n].view(N, R, C)), ref)) < BAR
    assert bool((buf[:8] == 7).all()) and bool((buf[8 + n:] == 7).all())
    if dtype is torch.bfloat16:
        buf[8:8 + n] = G.flatten()
        inside = buf[8:8 + n].view(N, R, C)
        assert max(errors(run(cuda_lib, inside, O=inside), ref)) < BAR
        assert bool((buf[:8] == 7).all()) and bool((buf[8 + n:] == 7).all())


@pytest.mark.parametrize("N,R,C", [(160, 40, 600), (90, 1100, 64), (2, 50, 9000), (1, 16500, 20), (140, 100, 900), (24, 128, 4000),
                                   (3, 8, 1025), (2, 9000, 8), (2, 9, 1000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_short_and_long_matrices(cuda_lib, N, R, C, dtype):
    G = gauss(N, R, C, dtype, seed=N + R + C)
    assert max(errors(run(cuda_lib, G), exact(G))) < BAR
