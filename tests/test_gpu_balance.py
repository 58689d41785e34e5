"""Balance loss, z-loss, per-expert counts and their gradient against the formulas in 64 bits.

Bar: counts and tokens exact.  Losses within 1e-5 relative and dlogits within 1e-5 of the sum of the
magnitudes of the terms each entry is made of: exp of a difference of up to about 30 carries 3e-6 (the
argument's own rounding), the softmax's and the segments' sums of at most about 80 levels 5e-6."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAR = 1e-5


def make(T, E, k, seed, scale=1.0):
    r = np.random.default_rng(seed)
    logits = (scale * r.standard_normal((T, E)) + r.standard_normal((1, E))).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    w = r.random((T, k)).astype(np.float32)
    dw = r.standard_normal((T, k)).astype(np.float32)
    return logits, idx, w, dw


def members(T, B, mask, offsets):
    m = np.zeros((B, T), bool)
    for s in range(B):
        lo, hi = (0, T) if offsets is None else (offsets[s], offsets[s + 1])
        m[s, lo:hi] = True
    return m if mask is None else m & (mask != 0)[None]


def reference(logits, idx, w, dw, dloss, mask, offsets):
    """counts, tokens, loss, dlogits, and the magnitude each dlogits entry is judged against."""
    T, E = logits.shape
    k, B = idx.shape[1], dloss.shape[0]
    m = members(T, B, mask, offsets)
    counts, tokens, loss = np.zeros((B, E), np.int64), m.sum(1), np.zeros((B, 2))
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for s in range(B):
        t = np.nonzero(m[s])[0]
        if not len(t):
            continue
        x = logits[t].astype(np.float64)
        top = x.max(1, keepdims=True)
        dead = np.isneginf(top)
        z = np.where(dead, 0.0, np.exp(x - np.where(dead, 0.0, top)))
        total = np.where(dead, 1.0, z.sum(1, keepdims=True))
        p, lse = z / total, np.where(dead, 0.0, top + np.log(total))
        picks = idx[t][(idx[t] >= 0) & (idx[t] < E)]
        c = np.bincount(picks, minlength=E).astype(np.float64)
        counts[s] = c
        n = len(t)
        loss[s] = E / (k * n * n) * (c * p.sum(0)).sum(), (lse ** 2).sum() / n
        gb, gz = dloss[s, 0] * E / (k * n * n), dloss[s, 1] * 2 / n
        pc = (p * c).sum(1, keepdims=True)
        d[t] = gb * p * (c - pc) + gz * lse * p
        mag[t] = abs(gb) * p * (c + pc) + abs(gz * lse) * p
    if w is not None:
        w, dw = w.astype(np.float64), dw.astype(np.float64)
        g, gm = w * (dw - (w * dw).sum(1, keepdims=True)), w * (abs(dw) + abs(w * dw).sum(1, keepdims=True))
        for j in range(k):
            t = np.nonzero((idx[:, j] >= 0) & (idx[:, j] < E))[0]
            d[t, idx[t, j]] += g[t, j]
            mag[t, idx[t, j]] += gm[t, j]
    return counts, tokens, loss, d, mag


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(bd, logits, idx, w, dw, dloss, mask=None, offsets=None, ws=None):
    T, E = logits.shape
    B = dloss.shape[0]
    counts = torch.full((B, E), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    loss = torch.full((B, 2), float("nan"), device="cuda")
    dl = torch.full((T, E), float("nan"), device="cuda")
    lg, ix, mk, off = dev(logits), dev(idx), dev(mask), dev(offsets)
    ws = ws or bd.Workspace(bd.moe_balance_workspace_bytes(T, E, B))
    bd.moe_balance_fwd(lg, ix, counts, tokens, loss, ws, mask=mk, seg_offsets=off)
    assert not ws.buffer.any()                   # as the next call wants it
    bd.moe_balance_bwd(lg, ix, dev(w), dev(dw), counts, tokens, dev(dloss), dl, mask=mk, seg_offsets=off)
    torch.cuda.synchronize()
    return counts.cpu().numpy(), tokens.cpu().numpy(), loss.cpu().numpy(), dl.cpu().numpy()


def check(got, ref):
    np.testing.assert_array_equal(got[0], ref[0])
    np.testing.assert_array_equal(got[1], ref[1])
    np.testing.assert_allclose(got[2], ref[2], rtol=BAR, atol=1e-30)
    assert np.all(np.isfinite(got[3]))
    assert np.all(np.abs(got[3] - ref[3]) <= BAR * ref[4] + 1e-37)


def losses(B, seed):
    return (np.random.default_rng(seed).standard_normal((B, 2))).astype(np.float32)


SHAPES = [(1, 1, 1, 1), (1, 8, 2, 1), (2, 33, 1, 3), (7, 5, 3, 2), (33, 127, 8, 4), (64, 128, 8, 1), (300, 130, 8, 7),
          (1000, 1024, 32, 3), (777, 1023, 1, 65), (4096, 256, 6, 1), (2500, 512, 8, 900), (12345, 64, 4, 2),
          (40000, 8, 2, 5), (20000, 512, 4, 3), (16500, 1024, 8, 2), (40001, 132, 6, 40), (70000, 68, 2, 1)]


@pytest.mark.parametrize("T,E,k,B", SHAPES)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_formulas(cuda_lib, T, E, k, B, masked, weights):
    logits, idx, w, dw = make(T, E, k, seed=T + E)
    r = np.random.default_rng(B)
    offsets = None if B == 1 else np.sort(np.r_[0, r.integers(0, T + 1, B - 1), T]).astype(np.int32)
    mask = (r.random(T) < 0.7) if masked else None
    if not weights:
        w = dw = None
    dloss = losses(B, T)
    check(run(cuda_lib, logits, idx, w, dw, dloss, mask, offsets), reference(logits, idx, w, dw, dloss, mask, offsets))


def test_masked_rows_are_not_read(cuda_lib):
    logits, idx, w, dw = make(200, 60, 4, 1)
    mask = np.ones(200, np.uint8)
    mask[3::7] = 0
    mask[150:] = 0
    ref = reference(logits, idx, w, dw, losses(2, 1), mask, np.array([0, 90, 200], np.int32))
    bad = logits.copy()
    bad[mask == 0] = np.nan
    bad[3] = np.inf
    check(run(cuda_lib, bad, idx, w, dw, losses(2, 1), mask, np.array([0, 90, 200], np.int32)), ref)
    mask[mask != 0] = 255                        # any byte but 0 counts
    check(run(cuda_lib, bad, idx, w, dw, losses(2, 1), mask, np.array([0, 90, 200], np.int32)), ref)


def test_nothing_counts(cuda_lib):
    logits, idx, w, dw = make(70, 16, 2, 2)
    got = run(cuda_lib, np.full_like(logits, np.nan), idx, w, dw, losses(1, 3), np.zeros(70, bool))
    check(got, reference(logits, idx, w, dw, losses(1, 3), np.zeros(70, bool), None))
    assert not got[0].any() and not got[1].any() and not got[2].any()


def test_empty_and_partial_segments(cuda_lib):
    """Empty segments first, between and last; tokens before the first and past the last offset."""
    logits, idx, w, dw = make(500, 100, 5, 4)
    offsets = np.array([11, 11, 11, 40, 40, 41, 333, 333, 480, 480], np.int32)
    d = losses(9, 5)
    check(run(cuda_lib, logits, idx, w, dw, d, None, offsets), reference(logits, idx, w, dw, d, None, offsets))


def test_no_tokens(cuda_lib):
    got = run(cuda_lib, np.zeros((0, 12), np.float32), np.zeros((0, 2), np.int32), None, None, losses(3, 1), None,
              np.zeros(4, np.int32))
    assert not got[0].any() and not got[1].any() and not got[2].any()


@pytest.mark.parametrize("E", [100, 101])
def test_infinities_and_lowest_values(cuda_lib, E):
    """Experts masked out of a row by -inf or by the type's lowest value; a row masked throughout."""
    logits, idx, w, dw = make(90, E, 4, 6)
    logits[::3, 50:] = -np.inf
    logits[1::3, 50:] = np.finfo(np.float32).min
    logits[4] = -np.inf
    logits[5, 1:] = -np.inf                      # one expert left
    d = losses(1, 7)
    check(run(cuda_lib, logits, idx, w, dw, d), reference(logits, idx, w, dw, d, None, None))


def test_nan_and_positive_infinity_show(cuda_lib):
    logits, idx, w, dw = make(40, 32, 4, 8)
    logits[7, 3] = np.nan
    logits[30, 1] = np.inf
    offsets = np.array([0, 20, 25, 40], np.int32)
    d = losses(3, 9)
    got = run(cuda_lib, logits, idx, w, dw, d, None, offsets)
    assert np.isnan(got[2][[0, 2]]).all() and np.isfinite(got[2][1]).all()
    assert np.isnan(got[3][[7, 30]]).all()
    rest = [t for t in range(40) if t not in (7, 30)]
    assert np.isfinite(got[3][rest]).all()


def test_wide_logits(cuda_lib):
    """Logits of 1e4: a softmax without its maximum would overflow."""
    logits, idx, w, dw = make(64, 128, 8, 10, scale=1e4)
    d = losses(1, 11)
    check(run(cuda_lib, logits, idx, w, dw, d), reference(logits, idx, w, dw, d, None, None))


def test_dropped_picks(cuda_lib):
    logits, idx, w, dw = make(130, 24, 3, 12)
    idx[5, 0], idx[6, 2], idx[7] = -1, 24, 2 ** 30
    d = losses(1, 13)
    check(run(cuda_lib, logits, idx, w, dw, d), reference(logits, idx, w, dw, d, None, None))


def test_zero_loss_gradient_is_the_routers(cuda_lib):
    logits, idx, w, dw = make(333, 96, 6, 14)
    got = run(cuda_lib, logits, idx, w, dw, np.zeros((1, 2), np.float32))
    dl = torch.empty(333, 96, device="cuda")
    cuda_lib.moe_router_bwd(dev(idx), dev(w), dev(dw), dl)
    np.testing.assert_allclose(got[3], dl.cpu().numpy(), rtol=1e-6, atol=1e-7)


def test_gradient_against_differences(cuda_lib):
    """Central differences of the 64-bit losses (picks held fixed): h = 1e-4 leaves h^2 / 6 of the third
    derivative, under 1e-6 of the gradient's scale, and 1e-11 of the losses' rounding over h."""
    logits, idx, _, _ = make(40, 12, 3, 15)
    offsets = np.array([0, 15, 40], np.int32)
    mask = np.ones(40, bool)
    mask[[2, 20]] = False
    d = losses(2, 16)
    got = run(cuda_lib, logits, idx, None, None, d, mask, offsets)[3]
    ref = reference(logits, idx, None, None, d, mask, offsets)

    def total(x):
        return (reference(x, idx, None, None, d, mask, offsets)[2] * d).sum()
    for t, e in [(0, 0), (2, 5), (14, 11), (15, 3), (39, 7), (20, 1)]:
        up, down = logits.astype(np.float64), logits.astype(np.float64)
        up[t, e] += 1e-4
        down[t, e] -= 1e-4
        assert abs((total(up) - total(down)) / 2e-4 - got[t, e]) <= 1e-4 * ref[4][t, e] + 1e-7


def test_repeats_bit_for_bit_and_on_another_stream(cuda_lib):
    logits, idx, w, dw = make(9000, 200, 8, 17)
    offsets = np.array([0, 100, 4000, 9000], np.int32)
    d = losses(3, 18)
    one = run(cuda_lib, logits, idx, w, dw, d, None, offsets)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        two = run(cuda_lib, logits, idx, w, dw, d, None, offsets)
    for a, b in zip(one, two):
        np.testing.assert_array_equal(a, b)


def test_captured_in_a_graph(cuda_lib):
    bd = cuda_lib
    logits, idx, w, dw = make(300, 48, 4, 19)
    lg, ix, dl = dev(logits), dev(idx), torch.empty(300, 48, device="cuda")
    counts, tokens = torch.empty(1, 48, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    loss, dloss = torch.empty(1, 2, device="cuda"), dev(losses(1, 20))
    wt, dwt, ws = dev(w), dev(dw), bd.Workspace(bd.moe_balance_workspace_bytes(300, 48, 1))

    def step():
        bd.moe_balance_fwd(lg, ix, counts, tokens, loss, ws)
        bd.moe_balance_bwd(lg, ix, wt, dwt, counts, tokens, dloss, dl)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    fresh, _, _, _ = make(300, 48, 4, 21)
    lg.copy_(dev(fresh))
    g.replay()
    torch.cuda.synchronize()
    ref = reference(fresh, idx, w, dw, losses(1, 20), None, None)
    check((counts.cpu().numpy(), tokens.cpu().numpy(), loss.cpu().numpy(), dl.cpu().numpy()), ref)


def test_one_workspace_for_calls_of_all_sizes(cuda_lib):
    """A call leaves the workspace as the next one, of whatever sizes, needs it, a row of NaN included."""
    bd = cuda_lib
    ws = bd.Workspace(bd.moe_balance_workspace_bytes(20000, 1024, 40))
    for T, E, k, B, bad in [(20000, 8, 2, 1, False), (300, 1024, 4, 40, False), (9000, 130, 8, 3, True), (20000, 512, 8, 1, False)]:
        logits, idx, w, dw = make(T, E, k, seed=E)
        offsets = None if B == 1 else np.linspace(0, T, B + 1).astype(np.int32)
        d = losses(B, 22)
        if bad:
            logits[T // 2] = np.nan
            assert np.isnan(run(bd, logits, idx, w, dw, d, None, offsets, ws)[2]).any()
        else:
            check(run(bd, logits, idx, w, dw, d, None, offsets, ws), reference(logits, idx, w, dw, d, None, offsets))
