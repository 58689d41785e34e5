"""Routing by scores against a plain implementation in 64 bits: picks exactly, weights and gradients by derived bounds.

Bounds.  A weight is a product of an exponential, a quotient and a scale in fp32, relative to a sum of at most 32 of them:
expf and the division give 2 + 2 half units in the last place, a softmax over all experts adds its sum's (ex2.approx 2^-22,
an argument rounded by 2^-24 of at most some 30, and as many roundings as the sum has levels), so 2e-6 relative covers
the renormalised and sigmoid weights and 6e-6 the others; the rounding of an exponent z adds 2^-24 |z|, taken as 2^-23 |ln w|.  A gradient w (dw - D) (1 - s) adds the weight's error on each
side of the difference: 4 x that of max |w dw| over the row, D included.  bf16 outputs add half a step, 2^-8 relative.
Picks are compared exactly."""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

W_REL, W_REL_ROW = 2e-6, 6e-6


def scores64(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    z = torch.exp(x - x.amax(1, keepdim=True))
    return z / z.sum(1, keepdim=True)


def choose64(logits, k, score="softmax", G=1, kept=1, rank=1, renorm=True, scale=1.0, bias=None, mask=None):
    """Picks and weights of each token: stable sorts in 64 bits, so that equal ones keep the order of their index."""
    T, E = logits.shape
    x = logits.double().cpu()
    s = scores64(x.cuda(), score).cpu()   # (the GPU's 64-bit exponential: sums that are equal but for its last bit are in no other order)
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    above = lambda v: torch.where(v.isnan(), math.inf, v)  # noqa: E731  (NaN ranks highest; no test has infinities beside it)
    out = (x == -math.inf) | (b == -math.inf)
    c = above(s + b).masked_fill(out, -math.inf)
    if kept < G:
        best = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :rank]
        value = torch.where(best == -math.inf, 0.0, best).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        first = value.sort(dim=1, descending=True, stable=True)
        stays = torch.zeros(T, G, dtype=torch.bool).scatter_(1, first.indices[:, :kept], first.values[:, :kept] > -math.inf)
        out = out | ~stays.repeat_interleave(E // G, 1)
    if mask is not None:
        out = out | ~mask.bool()[:, None]
    key = (above(x) if bias is None else c).masked_fill(out, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    idx = torch.where(out.gather(1, idx), -1, idx)
    z, at = x.gather(1, idx.clamp(min=0)), idx >= 0
    if renorm:   # relative to the largest, so that small scores count too
        z = (z if score == "softmax" else torch.nn.functional.logsigmoid(z)).masked_fill(~at, -math.inf)
        w = torch.softmax(z, 1).masked_fill(~at, 0.0)
    else:
        w = s.gather(1, idx.clamp(min=0)).masked_fill(~at, 0.0)
    return idx, w * scale


def grad64(logits, idx, dw, score, renorm, scale):
    """By autograd in 64 bits at the given picks."""
    x = logits.double().cpu().requires_grad_(True)
    live = (idx >= 0).double()
    u = scores64(x, score).gather(1, idx.clamp(min=0)) * live
    if renorm:
        u = u / u.sum(1, keepdim=True).clamp(min=1e-300)
    (u * scale * dw.double().cpu() * live).sum().backward()
    return x.grad


def run(moe, logits, k, bias=None, mask=None, dw=None, out=None, accumulate=None, **rule):
    T, E = logits.shape
    names = {"G": "groups", "kept": "topk_groups", "rank": "group_rank", "renorm": "renormalise"}
    r = moe.RouterRule(**{names.get(n, n): v for n, v in rule.items()})
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), math.nan, device="cuda")
    moe.moe_router_select_fwd(logits, idx, w, r, bias=bias, mask=mask)
    if dw is None:
        return idx, w
    d = accumulate.clone() if accumulate is not None else torch.full((T, E), math.nan, device="cuda", dtype=out or logits.dtype)
    moe.moe_router_select_bwd(logits, idx, w, dw, d, r, accumulate=accumulate is not None)
    return idx, w, d


def check(moe, logits, k, bias=None, mask=None, seed=0, out=None, **rule):
    g = torch.Generator().manual_seed(seed)
    T, E = logits.shape
    dw = torch.randn(T, k, generator=g).cuda()
    idx, w, d = run(moe, logits, k, bias, mask, dw, out, **rule)
    ri, rw = choose64(logits, k, bias=bias, mask=mask, **rule)
    assert torch.equal(idx.cpu().long(), ri)
    dense = rule.get("score", "softmax") == "softmax" and not rule.get("renorm", True)
    rel = W_REL_ROW if dense else W_REL
    assert ((w.cpu().double() - rw).abs() <= (rel + 2 ** -23 * rw.clamp(min=1e-37).log().abs()) * rw + 1e-37).all()
    safe = logits if mask is None else torch.where(mask.bool()[:, None], logits, torch.zeros_like(logits))
    rd = grad64(safe, ri, dw, rule.get("score", "softmax"), rule.get("renorm", True), rule.get("scale", 1.0))
    size = (rw * dw.cpu().double()).abs().sum(1, keepdim=True)
    bound = 4 * rel * size + (2 ** -8 * rd.abs() if d.dtype == torch.bfloat16 else 0) + 1e-37
    assert d.dtype == (out or logits.dtype)
    assert ((d.cpu().double() - rd).abs() <= bound).all()
    return idx, w, d


SHAPES = [(2500, 128, 8, 1, 1), (2600, 256, 8, 8, 4), (5000, 512, 8, 1, 1), (10_000, 64, 4, 4, 2), (1, 1, 1, 1, 1), (3, 2, 1, 1, 1), (7, 8, 2, 1, 1), (33, 16, 16, 1, 1), (70, 24, 5, 3, 2), (64, 256, 8, 8, 4), (50, 100, 7, 1, 1),
          (40, 1000, 32, 20, 9), (20, 1024, 32, 32, 8), (31, 999, 31, 3, 2), (29, 1023, 9, 31, 17), (45, 60, 13, 12, 5), (130, 127, 6, 1, 1),
          (66, 384, 8, 1, 1), (1230, 48, 6, 4, 2), (1220, 512, 8, 1, 1), (1220, 700, 3, 7, 3), (1290, 20, 3, 5, 4), (1220, 1020, 5, 17, 4),
          (1300, 128, 8, 1, 1), (1300, 256, 8, 8, 4), (1250, 31, 4, 31, 9)]


@pytest.mark.parametrize("T,E,k,G,kept", SHAPES)
@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [True, False])))
def test_picks_weights_and_gradients(cuda_lib, T, E, k, G, kept, score, renorm):
    g = torch.Generator().manual_seed(T * E + k)
    logits = (2 * torch.randn(T, E, generator=g)).cuda()
    bias = None if (T + k) % 2 else (0.1 * torch.randn(E, generator=g)).cuda()
    check(cuda_lib, logits, k, bias=bias, score=score, G=G, kept=kept, rank=1 + E % 2, renorm=renorm, scale=1.0 + (k == 8) * 1.5)


@pytest.mark.parametrize("T,E,k,G,kept", [(200, 64, 8, 8, 3), (1300, 128, 8, 1, 1), (90, 100, 10, 1, 1), (1300, 96, 5, 6, 2)])
@pytest.mark.parametrize("score,biased", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_bf16_logits_and_ties(cuda_lib, T, E, k, G, kept, score, biased):
    """bf16 logits meet each other exactly in most rows; equal sums go to the lower index."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(T, E, generator=g).to(torch.bfloat16)
    logits[::3] = (logits[::3].float() * 4).round().div(4).to(torch.bfloat16)
    bias = (0.25 * torch.randint(-1, 2, (E,), generator=g)).cuda() if biased else None
    for out in (torch.bfloat16, torch.float32):
        check(cuda_lib, logits.cuda(), k, bias=bias, score=score, G=G, kept=kept, rank=2, out=out)
    check(cuda_lib, logits.float().cuda(), k, bias=bias, score=score, G=G, kept=kept, rank=2, out=torch.bfloat16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,G,kept", [(64, 1, 1), (1000, 1, 1), (96, 8, 3)])
def test_all_experts_equal(cuda_lib, score, biased, E, G, kept):
    """A router that starts from zero: every sum the same, the lowest indices."""
    bias = torch.zeros(E, device="cuda") if biased else None
    idx, _, _ = check(cuda_lib, torch.zeros(40, E, device="cuda"), 6, bias=bias, score=score, G=G, kept=kept, rank=2)
    assert torch.equal(idx.cpu(), torch.arange(6, dtype=torch.int32).expand(40, 6))


def test_sums_within_fp32_of_each_other(cuda_lib):
    """Sums that fp32 cannot tell apart: bias = target - sigmoid(l), rounded to fp32, of few targets."""
    g = torch.Generator().manual_seed(5)
    for T, E, k, G, kept in [(300, 128, 8, 1, 1), (1300, 64, 6, 4, 2), (40, 300, 20, 1, 1)]:
        logits = torch.randn(1, E, generator=g).expand(T, E).clone()
        logits[1::2] += 1e-6 * torch.randn(T // 2, E, generator=g)
        target = 1.0 + 0.125 * torch.randint(0, 3, (E,), generator=g)
        bias = (target - torch.sigmoid(logits[0].double())).float()
        for score in ("sigmoid", "softmax"):
            if score == "softmax":
                bias = (target - torch.softmax(logits[0].double(), 0)).float()
            check(cuda_lib, logits.cuda(), k, bias=bias.cuda(), score=score, G=G, kept=kept, rank=2)
    # one that is larger behind equal ones, by less than fp32 or a key can tell, with and without a bias
    x = torch.full((100, 64), 0.5)
    x[torch.arange(100), torch.randint(0, 64, (100,), generator=g)] += 2.0 ** -24 * 2
    x[torch.arange(100), torch.randint(0, 64, (100,), generator=g)] += 2.0 ** -24 * 4
    for bias in (None, torch.full((64,), 0.25).cuda()):
        check(cuda_lib, x.cuda(), 6, bias=bias, score="sigmoid")
        check(cuda_lib, x.repeat(13, 1).cuda(), 6, bias=bias)
    # logits a last bit apart, without a bias
    base = torch.full((200, 96), 1.5)
    base += torch.randint(0, 5, (200, 96), generator=g) * 2.0 ** -23
    check(cuda_lib, base.cuda(), 7)
    check(cuda_lib, -base.cuda(), 7, score="sigmoid", G=8, kept=3, rank=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rank,biased", [(1, False), (2, False), (1, True), (2, True)])
def test_groups_within_fp32_of_each_other(cuda_lib, score, rank, biased):
    """Sums of groups that fp32 cannot tell apart at the border, in few and in many tokens, groups with one expert or none left."""
    g = torch.Generator().manual_seed(15)
    for T, E, G, kept, k in [(200, 64, 8, 3, 5), (1300, 128, 8, 4, 8), (1300, 96, 12, 5, 6), (60, 1000, 20, 7, 9), (1300, 256, 4, 1, 4)]:
        base = torch.randn(T, 1, E // G, generator=g).expand(T, G, E // G).reshape(T, E).clone()     # every group the same, in another order
        order = torch.stack([torch.randperm(E // G, generator=g) + i * (E // G) for i in range(G)]).flatten()
        logits = base[:, order]
        logits[1::3] += 2e-7 * torch.randn(logits[1::3].shape, generator=g)
        logits[2::3] += 1e-3 * torch.randn(logits[2::3].shape, generator=g)
        bias = None
        if biased:
            bias = 0.25 * torch.randint(0, 2, (E,), generator=g).float()
            bias[:E // G] = -math.inf
            bias[0] = 0.25                                                                # one left in the first group
            bias[E // G:2 * (E // G)] = -math.inf
        check(cuda_lib, logits.cuda(), k, bias=None if bias is None else bias.cuda(), score=score, G=G, kept=kept, rank=rank)


def test_sums_that_a_large_bias_makes_equal(cuda_lib):
    """s + b in 64 bits loses what s has under 2^-50 of b: such sums are equal, and the lower index comes first, groups too."""
    g = torch.Generator().manual_seed(16)
    for T, E, G, kept, k in [(300, 6, 6, 2, 1), (300, 32, 32, 7, 7), (1500, 12, 4, 2, 5), (1500, 64, 1, 1, 6), (100, 13, 13, 4, 4)]:
        logits = -30 + 0.003 * torch.randn(T, E, generator=g)
        logits[::3, E // 2] = 40.0
        for b in (7.25, 0.0):
            check(cuda_lib, logits.cuda(), k, bias=torch.full((E,), b).cuda(), score="sigmoid", G=G, kept=kept, rank=2, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,G,kept,dtype", [(40, 100, 1, 1, torch.float32), (3000, 387, 1, 1, torch.bfloat16), (60, 96, 3, 2, torch.float32)])
def test_biases_that_are_equal_less_the_largest(cuda_lib, score, T, E, G, kept, dtype):
    # equal logits, biases one step of 32 bits apart, the larger at the higher index; 0.5 above them both, they are the same number
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, E, generator=g)
    bias = torch.rand(E, generator=g) * 1e-2
    b = torch.tensor(-1.5e-5)
    for e in (5, 9, 14, 30):
        x[:, e] = 4.0
        bias[e] = b
        b = torch.nextafter(b, torch.tensor(0.0))
    bias[E - 1] = 0.5
    x[:, E - 1] = -30.0 if score == "sigmoid" else -3.0
    assert len({float(bias[e]) for e in (5, 9, 14, 30)}) == 4 and len({float(bias[e] - bias[E - 1]) for e in (5, 9, 14, 30)}) == 1
    idx, _, _ = check(cuda_lib, x.to(dtype).cuda(), 8, bias=bias.cuda(), score=score, G=G, kept=kept)
    order = [e for e in idx[0].tolist() if e in (5, 9, 14, 30)]
    assert G > 1 or order == [30, 14, 9, 5]


def test_saturated_scores(cuda_lib):
    """Logits so large that scores are 1 in 64 bits: ordered by the logits without a bias, equal with one."""
    g = torch.Generator().manual_seed(6)
    x = 40 + 30 * torch.rand(100, 64, generator=g)
    check(cuda_lib, x.cuda(), 5, score="sigmoid")
    check(cuda_lib, x.cuda(), 5, score="sigmoid", bias=torch.zeros(64).cuda())
    check(cuda_lib, x.cuda(), 5, score="sigmoid", G=8, kept=3, rank=2)          # groups tie, their experts do not
    check(cuda_lib, x.cuda(), 5, score="sigmoid", G=8, kept=3, rank=1, bias=(0.25 * torch.randint(0, 2, (64,), generator=g)).cuda())
    # small scores keep their digits where weights are relative
    check(cuda_lib, (-60 - 20 * torch.rand(100, 64, generator=g)).cuda(), 5, score="sigmoid")
    check(cuda_lib, (30 * torch.randn(100, 64, generator=g)).cuda(), 5, score="softmax", bias=torch.zeros(64).cuda())


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [True, False])))
def test_masks_and_excluded_experts(cuda_lib, score, renorm):
    """Padded tokens are not read; experts at -inf are not picked; rows that leave fewer than k, one or none."""
    g = torch.Generator().manual_seed(7)
    for T, E, k, G, kept in [(120, 40, 6, 1, 1), (1300, 64, 8, 8, 2), (50, 33, 33 - 1, 1, 1)]:
        logits = torch.randn(T, E, generator=g)
        logits[0] = -math.inf
        logits[1, 1:] = -math.inf
        logits[2, k // 2:] = -math.inf
        logits[3] = torch.finfo(torch.float32).min
        logits[4, 3:] = torch.finfo(torch.float32).min
        mask = torch.rand(T, generator=g) < 0.8
        mask[:5] = True
        logits[~mask] = math.nan
        bias = 0.1 * torch.randn(E, generator=g)
        bias[torch.randperm(E, generator=g)[:E // 5]] = -math.inf
        for b in (None, bias.cuda()):
            idx, w, d = check_masked(cuda_lib, logits.cuda(), k, b, mask.cuda(), score, G, kept, renorm)
            assert (idx[~mask.cuda()] == -1).all() and (w[~mask.cuda()] == 0).all() and (d[~mask.cuda()] == 0).all()
            assert (idx[0] == -1).all() and (w[0] == 0).all()
    # nothing is left for anybody
    bias = torch.full((40,), -math.inf, device="cuda")
    idx, w = run(cuda_lib, torch.randn(9, 40, generator=g).cuda(), 4, bias=bias, score=score, renorm=renorm)
    assert (idx == -1).all() and (w == 0).all()


def check_masked(moe, logits, k, bias, mask, score, G, kept, renorm):
    dw = torch.randn(logits.shape[0], k, generator=torch.Generator().manual_seed(1)).cuda()
    idx, w, d = run(moe, logits, k, bias, mask, dw, score=score, G=G, kept=kept, rank=2, renorm=renorm)
    ri, rw = choose64(logits, k, score=score, G=G, kept=kept, rank=2, renorm=renorm, bias=bias, mask=mask.cpu())
    assert torch.equal(idx.cpu().long(), ri)
    assert ((w.cpu().double() - rw).abs() <= W_REL_ROW * rw.abs() + 1e-37).all()
    assert torch.isfinite(d).all()
    assert (d[logits.isinf() & mask[:, None]] == 0).all()
    return idx, w, d


def test_nan_and_infinite_logits(cuda_lib):
    """NaN ranks above every number and stays in its row."""
    g = torch.Generator().manual_seed(8)
    for G, kept in ((1, 1), (8, 3)):
        for biased in (False, True):
            x = torch.randn(80, 64, generator=g)
            x[3, 17] = math.nan
            x[5, [9, 4]] = math.nan
            bias = (0.1 * torch.randn(64, generator=g)).cuda() if biased else None
            idx, w = run(cuda_lib, x.cuda(), 4, bias=bias, score="sigmoid", G=G, kept=kept, rank=2)
            assert idx[3, 0] == 17 and idx[5, :2].tolist() == [4, 9]
            assert w[3].isnan().all() and w[5].isnan().all()
            rest = [t for t in range(80) if t not in (3, 5)]
            ri, rw = choose64(x[rest], 4, score="sigmoid", G=G, kept=kept, rank=2, bias=bias)
            assert torch.equal(idx[rest].cpu().long(), ri)
            idx, w = run(cuda_lib, x.cuda(), 4, bias=bias, G=G, kept=kept, rank=2)
            assert ((idx >= 0) & (idx < 64)).all() and w[3].isnan().all()
            assert torch.isfinite(w[rest]).all()
    x = torch.randn(5, 16, generator=g)
    x[2, 11] = math.inf
    idx, w = run(cuda_lib, x.cuda(), 3, score="sigmoid")
    assert idx[2, 0] == 11 and torch.isfinite(w).all()


def test_gradient_against_differences(cuda_lib):
    """The weights' derivative by central differences of the forward itself, at picks that a small step does not change.
    A step of 2^-6 leaves a third-order error of h^2 / 6 of the third derivative (at most 1 here): 5e-5, and the
    weights' rounding over 2 h, 2^-23 / 2^-5: 4e-6."""
    g = torch.Generator().manual_seed(9)
    h = 2.0 ** -6
    for score, renorm in itertools.product(["softmax", "sigmoid"], [True, False]):
        base = torch.linspace(-2, 2, 24)[torch.randperm(24, generator=g)][None].cuda()
        dw = torch.randn(1, 5, generator=g).cuda()
        rule = dict(score=score, renorm=renorm, scale=1.5)
        idx, w, d = run(cuda_lib, base, 5, dw=dw, **rule)
        for e in range(24):
            ends = []
            for sign in (1, -1):
                x = base.clone()
                x[0, e] += sign * h
                i2, w2 = run(cuda_lib, x, 5, **rule)
                assert torch.equal(i2, idx)
                ends.append(float((w2.double() * dw.double()).sum()))
            assert abs((ends[0] - ends[1]) / (2 * h) - float(d[0, e])) < 3e-4


def test_accumulate_joins_the_balance_loss(cuda_lib):
    """dlogits of the balance loss first, the selection's added to it."""
    moe = cuda_lib
    g = torch.Generator().manual_seed(10)
    for T, E, k, score, renorm in [(300, 64, 6, "sigmoid", True), (1300, 130, 4, "softmax", False), (77, 128, 8, "softmax", True)]:
        logits, dw = torch.randn(T, E, generator=g).cuda(), torch.randn(T, k, generator=g).cuda()
        there = torch.randn(T, E, generator=g).cuda()
        idx, w, d = run(moe, logits, k, dw=dw, score=score, renorm=renorm)
        both = run(moe, logits, k, dw=dw, score=score, renorm=renorm, accumulate=there)[2]
        # one rounding of the sum, and in the dense form one for the row and one for the pick
        assert ((both.double() - there.double() - d.double()).abs() <= 2 ** -23 * (there.abs() + d.abs() + both.abs())).all()


@pytest.mark.parametrize("E,G,kept,k", [(500, 1, 1, 30), (999, 3, 2, 31), (256, 8, 4, 8), (201, 3, 2, 2), (13, 13, 11, 10), (40, 8, 2, 8), (64, 1, 1, 17), (1024, 1, 1, 12), (512, 1, 1, 9)])
@pytest.mark.parametrize("score,biased", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_dense_sums(cuda_lib, E, G, kept, k, score, biased):
    """Scores so close together that most tokens have several within what a key holds, in no order of their index."""
    g = torch.Generator(device="cuda").manual_seed(E + k)
    for T, width in ((3000, 0.02), (3000, 0.002), (900, 0.01), (20000, 0.003)):
        logits = 1 + width * torch.randn(T, E, generator=g, device="cuda")
        bias = None
        if biased:   # against the scores' own spread
            bias = width * (0.2 if score == "sigmoid" else 1.0 / E) * torch.randn(E, generator=g, device="cuda")
        idx, w = run(cuda_lib, logits, k, bias=bias, score=score, G=G, kept=kept, rank=2)
        ri, rw = choose64(logits, k, bias=bias, score=score, G=G, kept=kept, rank=2)
        assert torch.equal(idx.cpu().long(), ri)
        assert ((w.cpu().double() - rw).abs() <= W_REL * rw).all()


def test_long_batches_and_many_blocks(cuda_lib):
    """More tokens than one wave of blocks, against the plain order in 64 bits on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(11)
    for T, E, k, dtype in [(60_000, 64, 8, torch.float32), (40_003, 333, 5, torch.bfloat16), (70_001, 8, 2, torch.float32)]:
        logits = torch.randn(T, E, generator=g, device="cuda").to(dtype)
        bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        dw = torch.randn(T, k, generator=g, device="cuda")
        idx, w, d = run(cuda_lib, logits, k, bias=bias, dw=dw, score="sigmoid", renorm=False)
        s = scores64(logits.double(), "sigmoid")
        want = (s + bias.double()).sort(dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(idx.long(), want)
        u = s.gather(1, want)
        assert ((w.double() - u).abs() <= W_REL * u).all()
        rd = torch.zeros_like(s).scatter_(1, want, dw.double() * u * (1 - u))
        step = 2 ** -8 if dtype == torch.bfloat16 else 0
        assert ((d.double() - rd).abs() <= 4 * W_REL * dw.double().abs().amax() + step * rd.abs()).all()


def test_repeats_streams_and_graphs(cuda_lib):
    moe = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(12)
    T, E, k = 3000, 256, 8
    logits, dw = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    rule = dict(score="sigmoid", G=8, kept=4, rank=2, scale=2.5)
    first = run(moe, logits, k, bias=bias, dw=dw, **rule)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = run(moe, logits, k, bias=bias, dw=dw, **rule)
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    r = moe.RouterRule(score="sigmoid", groups=8, topk_groups=4, group_rank=2, scale=2.5)
    idx, w, d = torch.empty_like(first[0]), torch.empty_like(first[1]), torch.empty_like(first[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_router_select_fwd(logits, idx, w, r, bias=bias)
        moe.moe_router_select_bwd(logits, idx, w, dw, d, r)
    for _ in range(2):
        idx.fill_(0), w.fill_(0), d.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, first[0]) and torch.equal(w, first[1]) and torch.equal(d, first[2])


def test_what_lies_behind_the_outputs(cuda_lib):
    """Odd sizes leave what follows the tensors as it was."""
    moe = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(13)
    for T, E, k, dtype in [(13, 7, 3, torch.bfloat16), (1301, 9, 5, torch.float32), (9, 1, 1, torch.bfloat16), (8193, 5, 2, torch.bfloat16)]:
        logits, dw = torch.randn(T, E, generator=g, device="cuda").to(dtype), torch.randn(T, k, generator=g, device="cuda")
        r = moe.RouterRule(score="sigmoid")
        room = [torch.full((n + 64,), 5, dtype=t, device="cuda") for n, t in ((T * k, torch.int32), (T * k, torch.float32), (T * E, dtype))]
        idx, w, d = room[0][:T * k].view(T, k), room[1][:T * k].view(T, k), room[2][:T * E].view(T, E)
        moe.moe_router_select_fwd(logits, idx, w, r)
        moe.moe_router_select_bwd(logits, idx, w, dw, d, r)
        for buffer, n in zip(room, (T * k, T * k, T * E)):
            assert (buffer[n:] == 5).all()
        rd = grad64(logits, idx.cpu().long(), dw, "sigmoid", True, 1.0)
        step = 2 ** -8 if dtype == torch.bfloat16 else 0
        size = (w * dw).abs().sum(1, keepdim=True).cpu().double()
        assert ((d.cpu().double() - rd).abs() <= 4 * W_REL * size + step * rd.abs() + 1e-37).all()


def test_bias_step(cuda_lib):
    g = torch.Generator().manual_seed(14)
    for B, E in [(1, 1), (1, 8), (3, 128), (7, 1000), (4000, 64), (1, 1024)]:
        counts = torch.randint(0, 50, (B, E), generator=g, dtype=torch.int32)
        counts[:, E // 2] = counts.double().mean(1).round().int()
        if B == 3:
            counts[:] = 7
        bias = 0.1 * torch.randn(E, generator=g)
        bias[0] = -math.inf if E > 1 else bias[0]
        n = counts.long().sum(0)
        want = bias + 1e-3 * torch.sign(n.sum() - n * E).float()
        got = bias.cuda()
        cuda_lib.moe_router_bias_step(counts.cuda(), got, 1e-3)
        assert torch.equal(got.cpu(), want)
    big = torch.full((1, 4), 2 ** 31 - 1, dtype=torch.int32).cuda()
    big[0, 1] = 0
    bias = torch.zeros(4).cuda()
    cuda_lib.moe_router_bias_step(big, bias, 0.5)
    assert bias.tolist() == [-0.5, 0.5, -0.5, -0.5]


def test_empty_batch(cuda_lib):
    idx, w, d = run(cuda_lib, torch.empty(0, 16, device="cuda"), 4, dw=torch.empty(0, 4, device="cuda"))
    assert idx.shape == (0, 4) and d.shape == (0, 16)
