"""Cases of the operators that train the MoE layer's router and experts.

balance: the load-balance loss, the router z-loss and the per-expert counts of each segment of a batch,
and their gradient with respect to the router's logits, joined with the gradient of the top-k weights:

    c[s,e]   picks of expert e by the counted tokens of segment s (ids outside [0, E) are dropped)
    n[s]     counted tokens of segment s (mask true, offsets[s] <= t < offsets[s+1])
    p[t]     softmax of the logits of token t over all E experts,  lse[t] their log-sum-exp
    loss[s]  (E / (k n^2) sum_e c[s,e] sum_{t in s} p[t,e],  1 / n sum_{t in s} lse[t]^2), zeros where n = 0
    dlogits[t,e] = db[s] E / (k n^2) p[t,e] (c[s,e] - sum_i p[t,i] c[s,i]) + dz[s] 2 / n lse[t] p[t,e]
                   + w_j (dw_j - sum_i w_i dw_i)   where e is token t's pick j

orthogonalise: Newton-Schulz orthogonalisation of a batch of matrices (the Muon optimiser's update):

    X = G / (|G|_F + eps);  five times, with (a, b, c) = (3.4445, -4.7750, 2.0315):
    A = X X^T,  X <- a X + (b A + c A A) X      (on G^T where G has more rows than columns)

`run` computes the plain form with torch where `own` is false and calls the package where it is true.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7


def listed():
    return [
        # one step of a small model: the tiny layer's router (latency of the two calls)
        {"name": "balance_tiny", "op": "balance", "dir": "train", "T": 256, "E": 8, "k": 2, "B": 1, "mask": False},
        # statistics of a serving batch of single tokens: forward alone
        {"name": "balance_decode", "op": "balance", "dir": "fwd", "T": 64, "E": 128, "k": 8, "B": 1, "mask": False},
        # a training step of the 128-expert, top-8 layer at 16,384 tokens, one loss for the batch
        {"name": "balance_30b", "op": "balance", "dir": "train", "T": 16384, "E": 128, "k": 8, "B": 1, "mask": False},
        # the same with packed sequences of uneven length, padding and one loss for each sequence
        {"name": "balance_30b_seq", "op": "balance", "dir": "train", "T": 16384, "E": 128, "k": 8, "B": 13, "mask": True},
        # a backward alone at the router's largest expert count, with odd sizes
        {"name": "balance_max_bwd", "op": "balance", "dir": "bwd", "T": 4097, "E": 1023, "k": 32, "B": 3, "mask": True},
        # many tokens over many experts: bound by memory
        {"name": "balance_large", "op": "balance", "dir": "train", "T": 131072, "E": 512, "k": 8, "B": 16, "mask": True},
        # the router's own weight [E, H]: one small matrix, latency
        {"name": "ns_gate", "op": "ns", "N": 1, "R": 128, "C": 2048, "dtype": "f32"},
        # the tiny layer's gate and up projections, one matrix each
        {"name": "ns_tiny_w13", "op": "ns", "N": 16, "R": 128, "C": 256, "dtype": "bf16"},
        # odd sizes, a few matrices
        {"name": "ns_odd", "op": "ns", "N": 3, "R": 1001, "C": 777, "dtype": "f32"},
        # one large dense projection
        {"name": "ns_dense", "op": "ns", "N": 1, "R": 4096, "C": 4096, "dtype": "bf16"},
        # down projections of 32 experts of the 30B-shaped layer (more rows than columns)
        {"name": "ns_w2_e32", "op": "ns", "N": 32, "R": 2048, "C": 768, "dtype": "bf16"},
        # every gate and up projection of the 30B-shaped layer: 128 experts, fp32 gradients
        {"name": "ns_w13_30b", "op": "ns", "N": 256, "R": 768, "C": 2048, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        E = _log_int(rng, 2, 1024)
        T = _log_int(rng, 1, max(1, min(131072, 131072 * 512 // E)))
        return {"op": "balance", "dir": rng.choice(["train", "train", "fwd", "bwd"]), "T": T, "E": E,
                "k": _log_int(rng, 1, min(32, E)), "B": rng.choice([1, _log_int(rng, 1, 64)]), "mask": rng.random() < 0.5}
    R, C = _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)
    one = _ns_flops(1, R, C)
    most = max(1, min(256, int(_ns_flops(256, 768, 2048) // one)))
    return {"op": "ns", "N": _log_int(rng, 1, most), "R": R, "C": C, "dtype": rng.choice(["f32", "bf16"])}


def _ns_flops(N, R, C):
    """Five steps of X X^T and A A (symmetric: one triangle each) and B X."""
    m, n = min(R, C), max(R, C)
    return NS_STEPS * N * (m * (m + 1.0) * n + m * (m + 1.0) * m + 2.0 * m * m * n)


def work(case):
    if case["op"] == "ns":
        e = case["N"] * case["R"] * case["C"]
        return {"bytes": e * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": _ns_flops(case["N"], case["R"], case["C"])}
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    b = 4 * T * E + (T if case["mask"] else 0) + 4 * (B + 1)         # logits, mask, offsets
    b += 4 * T * k + 4 * B * E + 4 * B + 8 * B                       # picks; counts, tokens, losses in or out
    f = 4 * T * E
    if case["dir"] != "fwd":
        b += 4 * T * E + 8 * T * k                                   # dlogits; weights and their gradient
        f += 6 * T * E
    return {"bytes": b, "flops": f}


# ---- inputs --------------------------------------------------------------------------------------
def _prepare_ns(case, g):
    """Gradients as a layer gives them: the outer products of a few hundred tokens' activations and output
    gradients, tokens of uneven weight; one expert of a larger batch saw no token and has a zero gradient."""
    N, R, C = case["N"], case["R"], case["C"]
    K = 192
    dev = "cuda"
    left = torch.randn(N, K, R, generator=g, device=dev) * torch.rand(N, K, 1, generator=g, device=dev).square()
    right = torch.randn(N, K, C, generator=g, device=dev)
    G = torch.bmm(left.transpose(1, 2), right) * (1e-3 / K)
    if N > 8:
        G[N // 2] = 0
    G = G.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
    return {"op": "ns", "G": G, "O": torch.empty(N, R, C, dtype=torch.bfloat16, device=dev)}


def _prepare_balance(case, g):
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    dev = "cuda"
    logits = torch.randn(T, E, generator=g, device=dev) + 0.7 * torch.randn(1, E, generator=g, device=dev)
    top, idx = torch.topk(logits, k, dim=1)
    s = {"op": "balance", "dir": case["dir"], "k": k, "logits": logits, "idx": idx.to(torch.int32).contiguous(),
         "w": torch.softmax(top, 1).contiguous(), "dw": torch.randn(T, k, generator=g, device=dev),
         "mask": None, "offsets": None}
    cuts = torch.sort(torch.randint(0, T + 1, (B - 1,), generator=g, device=dev)).values
    ends = torch.cat([torch.zeros(1, device=dev, dtype=cuts.dtype), cuts, torch.full((1,), T, device=dev, dtype=cuts.dtype)])
    if B > 1:
        s["offsets"] = ends.to(torch.int32)
    if case["mask"]:  # padding at the end of each segment, a tenth on average
        t = torch.arange(T, device=dev)
        seg = torch.searchsorted(ends[1:].contiguous(), t, right=True)
        pad = 0.2 * torch.rand(B, generator=g, device=dev)
        length = (ends[1:] - ends[:-1]).float()
        s["mask"] = (t - ends[seg]).float() < (length * (1 - pad))[seg]
    s["dloss"] = torch.rand(B, 2, generator=g, device=dev) * torch.tensor([1e-2, 1e-3], device=dev) * T / B
    s["counts"] = torch.empty(B, E, dtype=torch.int32, device=dev)
    s["tokens"] = torch.empty(B, dtype=torch.int32, device=dev)
    s["loss"] = torch.empty(B, 2, device=dev)
    s["dlogits"] = torch.empty(T, E, device=dev)
    if case["dir"] == "bwd":  # the forward's counts, as the program holds them by then
        member = _members(s, torch.float32)
        s["counts"], s["tokens"] = _counts(s, member)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_ns(case, g) if case["op"] == "ns" else _prepare_balance(case, g)


# ---- plain forms ---------------------------------------------------------------------------------
def _members(s, dtype):
    """[B, T]: one where token t counts in segment s."""
    T, B = s["logits"].shape[0], s["loss"].shape[0]
    t = torch.arange(T, device=s["logits"].device)
    if s["offsets"] is None:
        m = torch.ones(B, T, dtype=torch.bool, device=t.device)
    else:
        m = (t[None] >= s["offsets"][:-1, None]) & (t[None] < s["offsets"][1:, None])
    if s["mask"] is not None:
        m = m & s["mask"][None]
    return m.to(dtype)


def _counts(s, member):
    """Counts [B, E] and counted tokens [B], int32, from the picks' one-hot sums over each segment."""
    B, E = s["loss"].shape[0], s["logits"].shape[1]
    inside = member.sum(0) > 0
    seg = member.argmax(0)
    at = seg[:, None] * E + s["idx"].long()
    ones = inside[:, None].expand_as(s["idx"]).to(torch.int32)
    counts = torch.zeros(B * E, dtype=torch.int32, device=at.device).index_add_(0, at.reshape(-1), ones.reshape(-1))
    return counts.view(B, E), (member > 0).sum(1).to(torch.int32)


def _plain_balance(s):
    logits, k = s["logits"], s["k"]
    T, E = logits.shape
    member = _members(s, torch.float32)
    counts, tokens = (s["counts"], s["tokens"]) if s["dir"] == "bwd" else _counts(s, member)
    top = logits.max(1, keepdim=True).values
    z = torch.exp(logits - top)
    total = z.sum(1, keepdim=True)
    p = z / total
    lse = (top + torch.log(total))[:, 0]
    n = tokens.to(torch.float32)
    inv = torch.where(n > 0, 1 / n, torch.zeros_like(n))
    scale = (E / k) * inv * inv
    out = {}
    if s["dir"] != "bwd":
        balance = scale * (counts * (member @ p)).sum(1)
        out.update(counts=counts, tokens=tokens, loss=torch.stack([balance, inv * (member @ lse.square())], 1))
    if s["dir"] != "fwd":
        c = member.t() @ ((s["dloss"][:, 0] * scale)[:, None] * counts)          # [T, E]: zero where a token does not count
        dz = member.t() @ (s["dloss"][:, 1] * 2 * inv)
        d = p * (c - (p * c).sum(1, keepdim=True)) + (dz * lse)[:, None] * p
        w, dw = s["w"], s["dw"]
        out["dlogits"] = d.scatter_add(1, s["idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return out


def _plain_ns(s):
    a, b, c = NS
    X = s["G"].float()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2)
    for _ in range(NS_STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.transpose(1, 2) if tall else X).to(torch.bfloat16).contiguous()


# ---- the framework's calls -----------------------------------------------------------------------
def _workspace(s, nbytes):
    """The workspace that a program makes once and keeps."""
    if "ws" not in s:
        from moe_expert_layer_permute_gb300 import binding as moe
        s["ws"] = moe.Workspace(nbytes())
    return s["ws"]


def _own_balance(s):
    from moe_expert_layer_permute_gb300 import binding as moe
    out = {}
    if s["dir"] != "bwd":
        T, E = s["logits"].shape
        ws = _workspace(s, lambda: moe.moe_balance_workspace_bytes(T, E, s["loss"].shape[0]))
        moe.moe_balance_fwd(s["logits"], s["idx"], s["counts"], s["tokens"], s["loss"], ws, mask=s["mask"],
                            seg_offsets=s["offsets"])
        out.update(counts=s["counts"], tokens=s["tokens"], loss=s["loss"])
    if s["dir"] != "fwd":
        moe.moe_balance_bwd(s["logits"], s["idx"], s["w"], s["dw"], s["counts"], s["tokens"], s["dloss"], s["dlogits"],
                            mask=s["mask"], seg_offsets=s["offsets"])
        out["dlogits"] = s["dlogits"]
    return out


def _own_ns(s):
    from moe_expert_layer_permute_gb300 import binding as moe
    G, O = s["G"], s["O"]
    ws = _workspace(s, lambda: moe.moe_orthogonalise_workspace_bytes(*G.shape))
    moe.moe_orthogonalise(G, O, ws, steps=NS_STEPS, coeffs=NS, eps=NS_EPS)
    return O


def run(state):
    if own:
        return _own_ns(state) if state["op"] == "ns" else _own_balance(state)
    return _plain_ns(state) if state["op"] == "ns" else _plain_balance(state)


# ---- 64 bits -------------------------------------------------------------------------------------
def _exact_ns(case, s):
    """In chunks of the batch; the polynomial applied as a X + b A X + c A (A X)."""
    a, b, c = NS
    out = []
    for G in s["G"].split(16):
        X = G.double()
        X = X / (torch.sqrt((X * X).sum((1, 2))) + NS_EPS)[:, None, None]
        for _ in range(NS_STEPS):
            if X.shape[1] <= X.shape[2]:
                A = torch.bmm(X, X.mT)
                Y = torch.bmm(A, X)
                X = a * X + b * Y + c * torch.bmm(A, Y)
            else:
                A = torch.bmm(X.mT, X)
                Y = torch.bmm(X, A)
                X = a * X + b * Y + c * torch.bmm(Y, A)
        out.append(X)
    return torch.cat(out)


def _exact_balance(case, s):
    E, k, B = case["E"], case["k"], case["B"]
    T = case["T"]
    x = s["logits"].double()
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    ends = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    d = torch.zeros_like(x)
    losses = []
    for i in range(B):
        rows = slice(ends[i], ends[i + 1])
        keep = torch.ones(ends[i + 1] - ends[i], dtype=torch.float64, device=x.device) if s["mask"] is None else s["mask"][rows].double()
        n = float(keep.sum())
        if n == 0:
            losses.append([0.0, 0.0])
            continue
        if case["dir"] == "bwd":
            c = s["counts"][i].double()
        else:
            c = torch.zeros(E, dtype=torch.float64, device=x.device)
            c.index_put_((s["idx"][rows].reshape(-1).long(),), keep[:, None].expand(-1, k).reshape(-1), accumulate=True)
        q = p[rows] * keep[:, None]
        f = E * c / (k * n)
        losses.append([float((f * q.sum(0)).sum()) / n, float((keep * lse[rows] ** 2).sum()) / n])
        gb, gz = (float(v) for v in s["dloss"][i].double())
        d[rows] = gb / n * (q * f - q * (q @ f)[:, None]) + 2 * gz / n * (q * lse[rows][:, None])
    out = {}
    if case["dir"] != "bwd":
        out.update(counts=None, tokens=None, loss=torch.tensor(losses, dtype=torch.float64))
    if case["dir"] != "fwd":
        w, dw = s["w"].double(), s["dw"].double()
        t = torch.arange(T, device=x.device)[:, None].expand(-1, k)
        d.index_put_((t, s["idx"].long()), w * dw - w * torch.einsum("tk,tk->t", w, dw)[:, None], accumulate=True)
        out["dlogits"] = d
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_ns(case, s) if case["op"] == "ns" else _exact_balance(case, s)
