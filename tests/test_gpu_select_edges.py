"""Routing by scores at biases of the type's ends, against the plain form in 64 bits (bounds: test_gpu_select.py)."""
import itertools

import pytest
import torch

from test_gpu_select import W_REL, W_REL_ROW, check, choose64, grad64, run

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


@pytest.mark.parametrize("T,E,k,G,kept", [(120, 40, 6, 1, 1), (1300, 64, 8, 8, 2), (50, 33, 32, 1, 1), (700, 999, 31, 3, 2), (300, 160, 8, 1, 1)])
@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [True, False])))
@pytest.mark.parametrize("biased,out", [(False, torch.float32), (True, torch.float32), (True, torch.bfloat16)])
def test_gradients_of_masked_and_short_rows(cuda_lib, T, E, k, G, kept, score, renorm, biased, out):
    """Rows that leave fewer than k picks, one or none, by -inf logits or biases, and logits at the least number, beside padded
    tokens that hold NaN; also joined to a gradient that stands there.  Against autograd in 64 bits at the picks, with -inf as the
    least logit of a score that is 0 there; bounds as test_gpu_select.py's."""
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=g)
    logits[0] = -float("inf")
    logits[1, 1:] = -float("inf")
    logits[2, k // 2:] = -float("inf")
    logits[3] = LEAST
    logits[4, 3:] = LEAST
    logits[5:60, ::3] = -float("inf")
    mask = torch.rand(T, generator=g) < 0.8
    mask[:5] = True
    logits[~mask] = float("nan")
    bias = None
    if biased:
        bias = 0.1 * torch.randn(E, generator=g)
        bias[torch.randperm(E, generator=g)[:E // 5]] = -float("inf")
        bias = bias.cuda()
    dw = torch.randn(T, k, generator=g).cuda()
    rule = dict(score=score, G=G, kept=kept, rank=2, renorm=renorm, scale=2.5)
    idx, w, d = run(cuda_lib, logits.cuda(), k, bias, mask.cuda(), dw, out, **rule)
    ri, rw = choose64(logits, k, bias=bias, mask=mask, **rule)
    assert torch.equal(idx.cpu().long(), ri) and (ri[mask] < 0).any() and (ri[mask] >= 0).any()
    # (a row without any finite logit has no scores to differentiate: its picks' gradients are 0, or there are none)
    safe = torch.where(logits == -float("inf"), torch.full_like(logits, LEAST), logits)
    safe = torch.where(mask[:, None] & (ri >= 0).any(1, keepdim=True), safe, torch.zeros_like(safe))
    # (autograd's sigmoid has infinity times 0 at LEAST; at -600 score and slope are under 1e-260 as well)
    rd = grad64(safe.clamp(min=-600.0), ri, dw, score, renorm, 2.5)
    if renorm and score == "sigmoid":   # scores of LEAST are 0 in 64 bits: picks of those alone weigh the same, slope w (dw - D / scale)
        low = (ri >= 0) & (safe.gather(1, ri.clamp(min=0)) == LEAST)
        for t in ((low | (ri < 0)).all(1) & low.any(1)).nonzero().flatten().tolist():
            at = ri[t][ri[t] >= 0]
            wt, dt = rw[t][:len(at)], dw[t].cpu().double()[:len(at)]
            rd[t] = 0
            rd[t, at] = wt * (dt - (wt * dt).sum() / 2.5)
    rel = W_REL_ROW if score == "softmax" and not renorm else W_REL
    size = (rw * dw.cpu().double()).abs().sum(1, keepdim=True)
    bound = 4 * rel * size + (2 ** -8 * rd.abs() if out == torch.bfloat16 else 0) + 1e-37
    assert ((d.cpu().double() - rd).abs() <= bound).all()
    assert (d[~mask.cuda()] == 0).all() and (d[0] == 0).all()
    if out == torch.float32:
        there = torch.randn(T, E, generator=g).cuda()
        both = run(cuda_lib, logits.cuda(), k, bias, mask.cuda(), dw, accumulate=there, **rule)[2]
        # With r = -s D of the row (|r| <= size) and q = w dw of the pick, d = fl(q + r) and both = fl(fl(there + r) + q), in either of
        # which r may stand unrounded (a fused product): 2^-24 (2 |r| + |d| + |there + r| + |both|), at most the following.  (Where
        # one pick has all of a row's score r and q cancel, and d says nothing of their size.)
        assert ((both.double() - there.double() - d.double()).abs() <= 2 ** -23 * (there.abs() + d.abs() + both.abs()) + 2 ** -22 * size.cuda()).all()


@pytest.mark.parametrize("T,E,G,kept,k", [(300, 16, 4, 2, 6), (2600, 16, 4, 3, 3), (2600, 128, 1, 1, 8), (60, 1000, 20, 7, 9), (2600, 256, 8, 4, 8), (40, 64, 1, 1, 8)])
@pytest.mark.parametrize("score,rank", list(itertools.product(["softmax", "sigmoid"], [1, 2])))
@pytest.mark.parametrize("biases", [None, (0.0,), (0.0, 1e-40, -1e-40), (0.0, 3e-39, 1e-38)])
def test_scores_below_the_numbers_of_fp32(cuda_lib, T, E, G, kept, k, score, rank, biases):
    """Scores under 1e-38 are 0 in the forward's 32 bits; groups and sums with biases as small are told apart all the same."""
    g = torch.Generator().manual_seed(E + k + T)
    logits = -84 - 20 * torch.rand(T, E, generator=g)
    if score == "softmax":   # beside one that has nearly all of the sum
        logits[:, E // 3] = 1.0
    bias = None if biases is None else torch.tensor(biases)[torch.randint(0, len(biases), (E,), generator=g)].cuda()
    check(cuda_lib, logits.cuda(), k, bias=bias, score=score, G=G, kept=kept, rank=rank)
