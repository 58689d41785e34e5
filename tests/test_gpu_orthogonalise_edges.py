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
