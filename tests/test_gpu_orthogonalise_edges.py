"""Orthogonalisation where its kernels meet their edges; formulas, inputs and bar as in test_gpu_orthogonalise.py."""
import pytest
import torch

from test_gpu_orthogonalise import BAR, errors, exact, gauss, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,R,C", [(2, 1300, 33), (2, 2501, 61), (2, 2051, 127), (5, 2101, 21), (3, 257, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clusters_with_ctas_past_the_last_column(cuda_lib, N, R, C, dtype):
    """Tall matrices off 16 bytes whose cluster has CTAs with nothing to copy."""
    G, n = gauss(N, R, C, dtype, seed=R + C), N * R * C
    buf = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    assert max(errors(run(cuda_lib, G, O=buf[8:8 + n].view(N, R, C)), exact(G))) < BAR
    assert bool((buf[:8] == 7).all()) and bool((buf[8 + n:] == 7).all())


@pytest.mark.parametrize("N,R,C", [(2, 100, 140), (1, 128, 2048), (40, 40, 300), (3, 61, 2501)])
def test_a_wait_limit_below_a_products_time(cuda_lib, N, R, C):
    """A wait may run out while its product is at work (one look at a barrier can outlast the product, so it need
    not): a status code or the right result, the product ends before its memory does, and the next call works."""
    bd = cuda_lib
    G = gauss(N, R, C, torch.float32, 21)
    ref = exact(G)
    O = torch.empty(N, R, C, dtype=torch.bfloat16, device="cuda")
    ws = bd.Workspace(bd.moe_orthogonalise_workspace_bytes(N, R, C))
    for _ in range(3):
        ws.set_wait_limit(1)
        bd.moe_orthogonalise(G, O, ws)
        status = bd.moe_read_device_status(ws)
        assert status in (0, bd.MOE_DEV_TIMEOUT)
        assert status or max(errors(O, ref)) < BAR
        ws.set_wait_limit()
        bd.moe_orthogonalise(G, O, ws)
        assert bd.moe_read_device_status(ws) == 0
        assert max(errors(O, ref)) < BAR


# The accuracy that the header states.  The kernels' roundings carried through the formulas on the host give O before
# its own rounding within 2e-3 where singular vectors are spread over many entries and, up to 128 rows, where lines
# along the longer edge hold them: 2.6e-3 with bf16's 1.7e-3, and 3e-3 leaves room for rows whose own rounding is
# worse than that.  Where few entries (past 128 rows, few lines) hold a singular vector they give up to 1e-2, and bf16
# rounds a single value by up to 3.9e-3.
SPREAD, HELD_BY_FEW = 3e-3, 1.5e-2


def lines(N, m, n, k, dtype, seed):
    """k non-zero lines of n values among m: the gradient of a router that met k experts."""
    g = torch.Generator().manual_seed(seed)
    G = torch.zeros(N, m, n)
    for i in range(N):
        G[i, torch.randperm(m, generator=g)[:k]] = torch.randn(k, n, generator=g)
    return (1e-3 * G).to(dtype).cuda()


@pytest.mark.parametrize("m,n", [(128, 1024), (40, 200), (16, 200), (100, 300)])
@pytest.mark.parametrize("k", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tall", [False, True])
def test_few_lines_up_to_128_rows(cuda_lib, m, n, k, dtype, tall):
    G = lines(24, m, n, k, dtype, m + n + k)
    if tall:
        G = G.transpose(1, 2).contiguous()
    assert max(errors(run(cuda_lib, G), exact(G))) < SPREAD


@pytest.mark.parametrize("N,m,n", [(40, 100, 1100), (2, 100, 5000), (2, 50, 9000), (2, 128, 4500)])
@pytest.mark.parametrize("k", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("tall", [False, True])
def test_few_lines_of_matrices_that_no_cluster_takes(cuda_lib, N, m, n, k, tall):
    """Long or many, so that the kernel of tiles has them."""
    G = lines(N, m, n, k, torch.float32, m + n + k)
    if tall:
        G = G.transpose(1, 2).contiguous()
    assert max(errors(run(cuda_lib, G), exact(G))) < SPREAD


@pytest.mark.parametrize("N,R,C", [(4, 40, 200), (4, 100, 300), (4, 300, 100), (2, 256, 400), (2, 600, 200), (90, 300, 520)])
@pytest.mark.parametrize("rank", [0, 8, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_spread_matrices(cuda_lib, N, R, C, rank, dtype):
    g = torch.Generator().manual_seed(R + C + rank)
    G = torch.randn(N, R, C, generator=g) if rank == 0 else torch.randn(N, R, rank, generator=g) @ torch.randn(N, rank, C, generator=g)
    G = G.to(dtype).cuda()
    assert max(errors(run(cuda_lib, G), exact(G))) < SPREAD


@pytest.mark.parametrize("R,C", [(16, 20), (100, 120), (128, 300), (150, 170), (256, 400), (400, 256), (300, 900)])
@pytest.mark.parametrize("kind", ["entry", "block 2", "block 3", "block 4", "diagonal", "lines 4", "columns 2"])
def test_matrices_held_by_few_values(cuda_lib, R, C, kind):
    g = torch.Generator().manual_seed(R + C)
    N, what, k = 16, kind.split()[0], int((kind + " 1").split()[1])
    G = torch.zeros(N, R, C)
    if what == "diagonal":
        i = torch.arange(min(R, C))
        G[:, i, i] = torch.randn(N, len(i), generator=g)
    elif what == "lines":
        G = lines(N, R, C, k, torch.float32, R).cpu()
    elif what == "columns":
        G = lines(N, C, R, k, torch.float32, C).cpu().transpose(1, 2).contiguous()
    else:
        G[:, 3:3 + k, 5:5 + k] = torch.randn(N, k, k, generator=g)
    G = G.cuda()
    assert max(errors(run(cuda_lib, G), exact(G))) < HELD_BY_FEW


@pytest.mark.parametrize("N,R,C", [(2, 100, 300), (2, 300, 90), (2, 300, 520), (2, 6, 700)])
@pytest.mark.parametrize("ratio", [1e-5, 1e-7, 1e-9, 1e-11, 1e-13])
@pytest.mark.parametrize("eps", [1e-7, 1.0])
def test_norms_far_below_eps(cuda_lib, N, R, C, ratio, eps):
    """The absolute error that the header states, 1e-9 an entry, beside the relative one."""
    G = gauss(N, R, C, torch.float32, 31, ratio * eps / (R * C) ** 0.5)
    ref = exact(G, eps=eps)
    O = run(cuda_lib, G, eps=eps).double().cpu()
    for o, r in zip(O, ref):
        assert float((o - r).norm()) <= BAR * float(r.norm()) + 1e-9 * (R * C) ** 0.5


@pytest.mark.parametrize("N,R,C", [(2, 100, 300), (2, 300, 520), (2, 6, 700)])
def test_entries_whose_squares_leave_fp32(cuda_lib, N, R, C):
    G = gauss(N, R, C, torch.float32, 32, 1e-17)
    assert max(errors(run(cuda_lib, G, eps=1e-20), exact(G, eps=1e-20))) < BAR
    if min(R, C) > 8:
        assert not run(cuda_lib, gauss(N, R, C, torch.float32, 32, 1e-26), eps=1e-20).any()


@pytest.mark.parametrize("N,R,C", [(2, 100, 300), (2, 300, 200), (2, 6, 40)])
def test_growth_between_steps(cuda_lib, N, R, C):
    """Singular values up to 7.9 between steps, and 63 for the polynomial of one; with up to 8 rows beyond that too."""
    g = torch.Generator().manual_seed(33)
    G = (torch.randn(N, R, 1, generator=g) @ torch.randn(N, 1, C, generator=g)).cuda()       # one singular value: 1
    for co in ([(7.5, 0, 0)] * 2, [(1, 6, 0), (0.5, 1.2, 0)], [(-7, 0, 0), (16, -1.5, 0.02)]):
        assert max(errors(run(cuda_lib, G, steps=2, coeffs=co), exact(G, 2, co))) < BAR
    far = [(9, 0, 0)] * 2                        # 81 in A's one entry where one entry is all there is
    G[:, 1:] = 0
    G[:, :, 1:] = 0
    O = run(cuda_lib, G, steps=2, coeffs=far)
    if min(R, C) <= 8:
        assert max(errors(O, exact(G, 2, far))) < BAR
    else:
        assert not O.isfinite().all()


@pytest.mark.parametrize("N,R,C", [(1, 16, 32768), (2, 12, 20001), (3, 20, 9000), (2, 9000, 40), (1, 9, 16500)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clusters_whose_ctas_add_few_rows(cuda_lib, N, R, C, dtype):
    """Short, long matrices: down to one row of A, and four threads, for each CTA of sixteen."""
    G = gauss(N, R, C, dtype, seed=R * C % 1000)
    assert max(errors(run(cuda_lib, G), exact(G))) < BAR
