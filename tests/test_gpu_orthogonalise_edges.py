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
