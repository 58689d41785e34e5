"""The balance loss where its kernels meet their edges; formulas and bar as in test_gpu_balance.py."""
import numpy as np
import pytest

from test_gpu_balance import check, losses, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,B", [(65, 128, 8, 1), (64, 128, 8, 1), (700, 40, 4, 2), (16384, 128, 8, 3), (5000, 1000, 2, 1)])
def test_picks_of_improbable_experts(cuda_lib, T, E, k, B):
    """A biased or forced router: the picked experts have p of about 1e-11, in one block of tokens or in several.  A
    block's sum of p, 1e-9, is held to 2^-48 or finer where blocks are joined: 2e-6 of it, less when they add up."""
    logits, _, w, dw = make(T, E, k, seed=T)
    logits[:, :k] = -20 + 0.1 * logits[:, :k]
    idx = np.broadcast_to(np.arange(k, dtype=np.int32), (T, k)).copy()
    offsets = None if B == 1 else np.linspace(0, T, B + 1).astype(np.int32)
    d = losses(B, 40)
    check(run(cuda_lib, logits, idx, w, dw, d, None, offsets), reference(logits, idx, w, dw, d, None, offsets))
