"""Routing by scores at biases of the type's ends, against the plain form in 64 bits (bounds: test_gpu_select.py)."""
import itertools

import pytest
import torch

from test_gpu_select import check

pytestmark = pytest.mark.gpu

LEAST, MOST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max


# (few and many tokens; experts of the groups at the border up to 32 and more; groups even and odd; fewer groups left than kept)
@pytest.mark.parametrize("T,E,G,kept,k", [(64, 8, 4, 3, 5), (64, 8, 4, 4, 7), (60, 64, 8, 6, 30), (3000, 64, 16, 10, 8), (2600, 256, 8, 5, 8), (50, 45, 9, 6, 20),
                                          (40, 1000, 20, 12, 9), (3000, 32, 32, 20, 18)])
@pytest.mark.parametrize("score,rank", list(itertools.product(["softmax", "sigmoid"], [1, 2])))
def test_whole_groups_at_the_least_bias(cuda_lib, T, E, G, kept, k, score, rank):
    """Masked by the type's lowest value, which is no exclusion: where groups kept reach into those, their sums are compared as
    they are in 64 bits (two of them are beyond 32), and their experts are picked behind the others."""
    g = torch.Generator().manual_seed(E + k)
    logits = torch.randn(T, E, generator=g)
    for spread in (0.0, 0.1):
        bias = spread * torch.randn(E, generator=g)
        bias[E // 2:] = LEAST
        idx, _, _ = check(cuda_lib, logits.cuda(), k, bias=bias.cuda(), score=score, G=G, kept=kept, rank=rank)
        assert (idx >= 0).all()
        bias[:E // G] = LEAST                                   # the first group too, all but one expert
        bias[0] = 0.5
        bias[-2 * (E // G):-(E // G)] = -float("inf")           # and one that is out
        check(cuda_lib, logits.cuda(), min(k, (kept - 1) * (E // G)), bias=bias.cuda(), score=score, G=G, kept=kept, rank=rank)


@pytest.mark.parametrize("T,E,G,kept,k", [(64, 16, 1, 1, 12), (64, 16, 4, 3, 10), (2600, 128, 1, 1, 8), (2600, 128, 8, 3, 20), (30, 999, 3, 2, 31)])
@pytest.mark.parametrize("score,rank", list(itertools.product(["softmax", "sigmoid"], [1, 2])))
@pytest.mark.parametrize("high", [1e31, 1e35, MOST])
def test_biases_further_apart_than_fp32_reaches(cuda_lib, T, E, G, kept, k, score, rank, high):
    """The least bias less a large one is -inf in 32 bits, which is no exclusion either."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(T, E, generator=g)
    bias = 0.1 * torch.randn(E, generator=g)
    bias[1::2] = LEAST
    bias[3] = LEAST / 2
    bias[0], bias[E // 2] = high, high / 4
    bias[5] = -float("inf")
    idx, _, _ = check(cuda_lib, logits.cuda(), k, bias=bias.cuda(), score=score, G=G, kept=kept, rank=rank)
    assert (idx >= 0).all() and (idx != 5).all()
