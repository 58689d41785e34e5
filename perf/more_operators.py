"""Cases of two operators that a training step of the MoE layer needs around what is there.

select: routing by scores over all experts, with a bias that only the choice sees and with groups of experts:

    s = softmax(l) over the E experts, or sigmoid(l);   c = s + b   (b: fp32 [E], or none)
    an expert whose logit or bias is -inf is excluded
    group g (E / G consecutive experts): the sum of its `rank` largest c; the `kept` groups with the largest stay
    idx: the k largest c of the experts that stay, in descending order (-1 where there are fewer than k)
    w_j = scale s_j, divided by the sum of the k picks' s where the rule renormalises
    c is compared in 64 bits, without a bias by the logits themselves; equal ones go to the lowest index
    dlogits = sum_j dw_j dw_j/dl (the choice carries no gradient); masked tokens: idx -1, w 0, dlogits 0
    after a step the bias follows the load: b += rate sign(mean of the counts - counts[e])

adamw: one AdamW step over many tensors at once, states in 32 bits or in 8, gradients scaled by a factor (the clip
factor min(1, most / |g|) of the norm over all of them, where the case clips):

    m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2
    p' = p - lr (m' / (1 - b1^t) / (sqrt(v' / (1 - b2^t)) + eps) + decay p),  and a bf16 copy of p'
    8 bits: m and r = sqrt(v) are held as E4M3 codes times one fp32 scale for each 256 values of a tensor, x = code scale;
    scale = max|x| / 448; a value is rounded up with the probability of its distance to the code below, by 16 bits of
    a hash of (seed, number of the tensor, number of the value); codes of r are at least the smallest positive one

`run` computes the plain form with torch where `own` is false and calls the package where it is true.
"""
import math

import torch

own = False

BETAS, EPS, DECAY, LR = (0.9, 0.999), 1e-8, 0.1, 1e-3
BIAS_RATE = 1e-3
BLOCK = 256
LEAST = 1e-35   # blocks of 8-bit states with nothing larger become zeros


def _select(name, T, E, k, **kw):
    case = {"op": "select", "dir": "train", "T": T, "E": E, "k": k, "score": "softmax", "G": 1, "kept": 1, "rank": 1,
            "renorm": True, "scale": 1.0, "bias": False, "drained": 0, "mask": False, "dtype": "f32"}
    return {"name": name, **case, **kw}


def _adamw(name, tensors, elements, **kw):
    case = {"op": "adamw", "tensors": tensors, "elements": elements, "state": 32, "grad": "f32", "copy": False, "clip": False,
            "step": 100}
    return {"name": name, **case, **kw}


def listed():
    grouped = {"score": "sigmoid", "G": 8, "kept": 4, "rank": 2, "scale": 2.5, "bias": True}
    return [
        # single tokens of a serving batch through grouped, biased routing: forward alone, latency
        _select("select_decode", 64, 256, 8, dir="fwd", **grouped),
        # one step of the tiny layer's router
        _select("select_tiny", 256, 8, 2),
        # the 128-expert, top-8 layer at 16,384 tokens, softmax over all experts, renormalised, bf16 logits
        _select("select_30b", 16384, 128, 8, dtype="bf16"),
        # a step of a layer balanced by its bias alone: sigmoid scores, groups, padded tokens
        _select("select_grouped", 16384, 256, 8, mask=True, **grouped),
        # odd sizes, many picks, experts taken out of service, weights that are not renormalised (a dense gradient)
        _select("select_odd", 4097, 999, 31, G=3, kept=2, renorm=False, bias=True, drained=5),
        # many tokens over many experts: bound by memory
        _select("select_large", 131072, 512, 8, score="sigmoid", bias=True),
        # the router's own weight [E, H] and bias [E] beside orthogonalised experts: latency
        _adamw("adamw_router", 2, 128 * 2048 + 128),
        # a model's norms, biases and routers: many small tensors, clipped
        _adamw("adamw_many", 240, 1_200_000, clip=True),
        # the tiny layer's experts, bf16 gradients and bf16 weights, 8-bit states
        _adamw("adamw8_tiny", 2, 8 * 256 * 384, state=8, grad="bf16", copy=True),
        # some tens of uneven tensors in 8 bits, clipped
        _adamw("adamw8_odd", 37, 20_000_003, state=8, clip=True),
        # every expert of the 30B-shaped layer, fp32 gradients and states, bf16 weights, clipped
        _adamw("adamw_30b", 2, 128 * 3 * 768 * 2048, copy=True, clip=True),
        # the same with bf16 gradients and 8-bit states
        _adamw("adamw8_30b", 2, 128 * 3 * 768 * 2048, state=8, grad="bf16", copy=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        E = _log_int(rng, 2, 1024)
        G = rng.choice([1, rng.choice([d for d in range(1, 33) if E % d == 0])])
        kept = rng.randint(1, G)
        T = _log_int(rng, 1, max(1, min(131072, 131072 * 512 // E)))
        k = _log_int(rng, 1, min(32, kept * (E // G)))
        case = _select("", T, E, k, dir=rng.choice(["train", "train", "fwd", "bwd"]),
                       score=rng.choice(["softmax", "sigmoid"]), G=G, kept=kept, rank=rng.choice([1, 2]), renorm=k > 1 and rng.random() < 0.7,   # (one pick alone would weigh 1 whatever its logit is)
                       scale=rng.choice([1.0, 2.5]), bias=rng.random() < 0.6, mask=rng.random() < 0.4,
                       dtype=rng.choice(["f32", "f32", "bf16"]))
        if case["bias"] and rng.random() < 0.2:
            case["drained"] = rng.randint(1, max(1, E // 8))
    else:
        elements = _log_int(rng, 1000, 300_000_000)
        case = _adamw("", _log_int(rng, 1, 300), elements, state=rng.choice([32, 8]), grad=rng.choice(["f32", "bf16"]),
                      copy=rng.random() < 0.5, clip=rng.random() < 0.5, step=_log_int(rng, 1, 100_000))
    del case["name"]
    return case


def _sizes(case):
    """Elements of each tensor: uneven, from a few to some tens of times the least."""
    N, total = case["tensors"], case["elements"]
    weight = [1 + (7 * i + 3) % 11 + 29 * (i % 5 == 0) for i in range(N)]
    size = [max(1, (total - N) * w // sum(weight)) for w in weight]
    size[-1] += total - sum(size)
    return size


def work(case):
    if case["op"] == "adamw":
        n, g, state = case["elements"], 2 if case["grad"] == "bf16" else 4, 8 if case["state"] == 32 else 2
        b = n * (g + 2 * 4 + 2 * state + (2 if case["copy"] else 0))
        if state == 2:
            b += 16 * sum(-(-s // BLOCK) for s in _sizes(case))
        if case["clip"]:   # a gradient that does not fit L2 beside the rest is read for the norm and for the step
            b += n * g if n * g > 100_000_000 else 0
        return {"bytes": b, "flops": 16 * n}
    T, E, k = case["T"], case["E"], case["k"]
    e = 2 if case["dtype"] == "bf16" else 4
    dense = case["score"] == "softmax" and not case["renorm"]
    b = (T if case["mask"] else 0) + (4 * E if case["bias"] else 0) + 8 * T * k
    f = 0
    if case["dir"] != "bwd":
        b += e * T * E
        f += 6 * T * E
    if case["dir"] != "fwd":
        b += e * T * E + 4 * T * k                                   # dlogits; the weights' gradient
        f += T * E
        if dense and (case["dir"] == "bwd" or e * T * E > 100_000_000):
            b += e * T * E
    return {"bytes": b, "flops": f}


# ---- inputs --------------------------------------------------------------------------------------
def _prepare_select(case, g):
    T, E, k, dev = case["T"], case["E"], case["k"], "cuda"
    spread = 0.7 * torch.randn(1, E, generator=g, device=dev)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = {"op": "select", "case": case, "bias": None, "mask": None, "counts": None,
         "logits": (torch.randn(T, E, generator=g, device=dev) + spread).to(dtype),
         "dw": torch.randn(T, k, generator=g, device=dev)}
    if case["bias"]:   # as a bias that follows the load has become: against the spread, in steps of its rate
        unit = 0.1 if case["score"] == "sigmoid" else 0.1 / E
        b = -unit * spread[0] + 0.1 * unit * torch.randn(E, generator=g, device=dev)
        s["bias"] = torch.round(b / BIAS_RATE) * BIAS_RATE if case["score"] == "sigmoid" else b
        if case["drained"]:
            s["bias"][torch.randperm(E, generator=g, device=dev)[:case["drained"]]] = -math.inf
        s["counts"] = torch.randint(0, 2 * max(1, T * k // E) + 1, (1, E), generator=g, device=dev, dtype=torch.int32)
    if case["mask"]:
        s["mask"] = torch.rand(T, generator=g, device=dev) < 0.9
    s["idx"], s["w"] = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    s["dlogits"] = torch.empty(T, E, device=dev, dtype=dtype)
    if case["dir"] == "bwd":   # the forward's picks and weights, as the program holds them by then
        s["idx"], s["w"] = _plain_choice(s)
    return s


def _prepare_adamw(case, g):
    """Tensors at multiples of 256 elements of a few buffers, as a program that keeps its weights, gradients and states
    in one piece has them.  States are those of a run under way; some gradients are zero (experts without tokens)."""
    dev, size = "cuda", _sizes(case)
    room = [-(-n // BLOCK) * BLOCK for n in size]
    start = [0]
    for r in room:
        start.append(start[-1] + r)
    total = start[-1]
    first = torch.tensor(start, device=dev)
    length = torch.tensor(size, device=dev)

    def flat(std, dtype=torch.float32):
        return (torch.randn(total, generator=g, device=dev) * std).to(dtype)

    def views(buffer, unit=1):
        return [buffer[a // unit:a // unit + -(-n // unit)] for a, n in zip(start, size)]

    level = torch.exp(2 * torch.randn(total // BLOCK, generator=g, device=dev)) * 1e-3    # gradients of uneven size
    level[torch.rand(total // BLOCK, generator=g, device=dev) < 0.02] = 0
    level = level.repeat_interleave(BLOCK)
    s = {"op": "adamw", "case": case, "first": first, "length": length, "p": flat(0.02),
         "g": flat(1.0).mul_(level).to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32),
         "copy": None, "seed": 12345}
    m, r = flat(0.3).mul_(level), (flat(0.3) + 1).abs_().mul_(level)
    if case["state"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        for name, x in (("m", m), ("r", r)):
            x = x.view(-1, BLOCK)
            scale = x.abs().amax(1) * (1.0 / 448)
            s[name + "_scale"] = scale
            s[name] = (x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(-1)
    del m, r, level
    if case["copy"]:
        s["copy"] = s["p"].to(torch.bfloat16)
    s["norm"] = torch.zeros(2, device=dev)
    for name in ("p", "g", "m", "v", "r", "copy"):   # what lies between the tensors is nobody's
        if s.get(name) is not None:
            for a, b, n in zip(start, start[1:], size):
                s[name].view(torch.uint8 if name in ("m", "r") and case["state"] == 8 else s[name].dtype)[a + n:b] = 0
            s["list_" + name] = views(s[name])
    if case["state"] == 8:
        s["list_m_scale"], s["list_r_scale"] = views(s["m_scale"], BLOCK), views(s["r_scale"], BLOCK)
    s["most"] = 0.5 * math.sqrt(case["elements"]) * 1e-2
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_select(case, g) if case["op"] == "select" else _prepare_adamw(case, g)


# ---- plain forms ---------------------------------------------------------------------------------
def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    z = torch.exp(x - x.max(1, keepdim=True).values)
    return z / z.sum(1, keepdim=True)


def _plain_choice(s):
    """Picks int32 [T, k], -1 where there is none, and their weights: the order in 64 bits, the weights in 32."""
    case, logits, bias = s["case"], s["logits"], s["bias"]
    (T, E), k, G = logits.shape, case["k"], case["G"]
    x = logits.double()
    c = _scores(x, case["score"])
    out = torch.isinf(x) & (x < 0)
    if bias is not None:
        c = c + bias.double()
        out = out | (torch.isinf(bias) & (bias < 0))
    low = torch.full_like(c, -math.inf)
    if G > 1:
        by_group = torch.where(out, low, c).view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :case["rank"]]
        value = torch.where(by_group > low[:, :1, None], by_group, torch.zeros_like(by_group)).sum(2)
        value = torch.where(by_group[:, :, 0] > low[:, :1], value, low[:, :1])
        best = value.sort(dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        out = out | ~kept.repeat_interleave(E // G, 1)
    key = torch.where(out, low, x if bias is None else c)
    top = key.sort(dim=1, descending=True, stable=True)
    idx = torch.where(top.values[:, :k] > low[:, :1], top.indices[:, :k], torch.full_like(top.indices[:, :k], -1))
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, torch.full_like(idx, -1))
    u = torch.gather(_scores(logits.float(), case["score"]), 1, idx.clamp(min=0))
    u = torch.where(idx >= 0, u, torch.zeros_like(u))
    if case["renorm"]:
        total = u.sum(1, keepdim=True)
        u = u / torch.where(total > 0, total, torch.ones_like(total))
    return idx.to(torch.int32), u * case["scale"]


def _plain_select(s):
    case = s["case"]
    out = {}
    idx, w = s["idx"], s["w"]
    if case["dir"] != "bwd":
        idx, w = _plain_choice(s)
        out.update(idx=idx, w=w)
    if case["dir"] == "fwd":
        return out
    x, there = s["logits"].float(), idx >= 0
    at = idx.long().clamp(min=0)
    score = _scores(x, case["score"])
    dw = torch.where(there, s["dw"], torch.zeros_like(s["dw"])) * case["scale"]
    u = torch.where(there, torch.gather(score, 1, at), torch.zeros_like(dw))
    if case["renorm"]:
        total = u.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        dw = (dw - (dw * (u / total)).sum(1, keepdim=True)) / total
    if case["score"] == "sigmoid":
        d = torch.where(there, dw * u / (1 + torch.exp(torch.gather(x, 1, at))), torch.zeros_like(dw))
        d = torch.zeros_like(x).scatter_add(1, at, d)
    else:
        d = torch.zeros_like(x).scatter_add(1, at, torch.where(there, dw * u, torch.zeros_like(dw)))
        if not case["renorm"]:   # renormalised, the sum is zero
            d = d - score * (dw * u).sum(1, keepdim=True)
    out["dlogits"] = d.to(s["dlogits"].dtype)
    if s["bias"] is not None and case["dir"] == "train":
        n = s["counts"].sum(0).double()
        s["bias"].add_(torch.sign(n.mean() - n).float() * BIAS_RATE)
        out["bias"] = s["bias"]
    return out


def _noise(s, total):
    """32 random bits for every place of the buffers, as int64."""
    place = torch.arange(total, device="cuda")
    tensor = torch.bucketize(place, s["first"][1:], right=True)
    low = 0xffffffff
    h = ((place - s["first"][tensor]) * 0x9E3779B1 + s["seed"] + (tensor + 1) * 0x85EBCA77) & low
    h = ((h ^ (h >> 16)) * 0x7FEB352D) & low
    h = ((h ^ (h >> 15)) * 0x846CA68B) & low
    return h ^ (h >> 16)


def _to_codes(x, bits, least):
    """x in [0, 448] rounded to E4M3 by 16 random bits, as codes 0 to 126: times 2^-120 the codes are the leading bits
    of a number's fp32 form."""
    b = (x * 2.0 ** -120).view(torch.int32).long() + (bits << 4) + 8
    return (b >> 20).clamp(least, 126).to(torch.uint8)


def _plain_adamw(s):
    case, p, g = s["case"], s["p"], s["g"].float()
    eight, (b1, b2) = case["state"] == 8, BETAS
    out = {"p": p}
    if case["clip"]:
        norm = g.square().sum().sqrt()
        factor = (s["most"] / norm).clamp(max=1.0)
        g = g * factor
        s["norm"].copy_(torch.stack([norm, factor]))
        out["norm"] = s["norm"]
    if eight:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        r = (s["r"].float().view(-1, BLOCK) * s["r_scale"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = v.sqrt()
    fix1, fix2 = 1 - b1 ** case["step"], math.sqrt(1 - b2 ** case["step"])
    p.copy_(p - LR * (m / fix1 / (root / fix2 + EPS) + DECAY * p))
    if eight:
        h = _noise(s, p.numel())
        place = torch.arange(p.numel(), device=p.device)
        tensor = torch.bucketize(place, s["first"][1:], right=True)
        inside = place - s["first"][tensor] < s["length"][tensor]
        for name, x, bits, least in (("m", m, h & 0xffff, 0), ("r", root, h >> 16, 1)):
            x = x.view(-1, BLOCK)
            scale = x.abs().amax(1)
            scale = torch.where(scale < LEAST, torch.zeros_like(scale), scale)
            up = torch.where(scale > 0, torch.reciprocal(scale) * 448, torch.zeros_like(scale))
            code = _to_codes((x.abs() * up[:, None]).view(-1), bits, least)
            code = torch.where(inside & (up.repeat_interleave(BLOCK) > 0), code | ((x.view(-1) < 0) * 128).to(torch.uint8), torch.zeros_like(code))
            s[name].view(torch.uint8).copy_(code)
            s[name + "_scale"].copy_(scale * (1.0 / 448))
            out[name], out[name + "_scale"] = s[name], s[name + "_scale"]
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
        out["m"], out["v"] = s["m"], s["v"]
    if s["copy"] is not None:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    return out


# ---- the framework's calls -----------------------------------------------------------------------
def _own_select(s):
    from moe_expert_layer_permute_gb300 import binding as moe
    case = s["case"]
    if "rule" not in s:
        s["rule"] = moe.RouterRule(score=case["score"], groups=case["G"], topk_groups=case["kept"], group_rank=case["rank"],
                                   renormalise=case["renorm"], scale=case["scale"])
    out = {}
    if case["dir"] != "bwd":
        moe.moe_router_select_fwd(s["logits"], s["idx"], s["w"], s["rule"], bias=s["bias"], mask=s["mask"])
        out.update(idx=s["idx"], w=s["w"])
    if case["dir"] == "fwd":
        return out
    moe.moe_router_select_bwd(s["logits"], s["idx"], s["w"], s["dw"], s["dlogits"], s["rule"])
    out["dlogits"] = s["dlogits"]
    if s["bias"] is not None and case["dir"] == "train":
        moe.moe_router_bias_step(s["counts"], s["bias"], BIAS_RATE)
        out["bias"] = s["bias"]
    return out


def _own_adamw(s):
    from moe_expert_layer_permute_gb300 import binding as moe
    case = s["case"]
    eight = case["state"] == 8
    if "lists" not in s:   # made once, as a program that keeps its buffers does
        names = ["p", "g", "m", "r" if eight else "v", "copy", "m_scale", "r_scale"]
        s["lists"] = [moe.TensorList(s["list_" + n]) if s.get("list_" + n) is not None else None for n in names]
        s["ws"] = moe.Workspace(moe.moe_grad_norm_workspace_bytes(case["elements"], case["tensors"])) if case["clip"] else None
    p, g, m, v, copy, m_scale, v_scale = s["lists"]
    out = {"p": s["p"], "m": s["m"]}
    if case["clip"]:
        moe.moe_grad_norm(g, s["norm"], s["ws"], max_norm=s["most"])
        out["norm"] = s["norm"]
    moe.moe_adamw_step(p, g, m, v, case["step"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, copies=copy, m_scales=m_scale,
                       v_scales=v_scale, grad_scale=s["norm"][1:] if case["clip"] else None, seed=s["seed"])
    out.update({n: s[n] for n in (("r", "m_scale", "r_scale") if eight else ("v",))})
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


def run(state):
    if own:
        return _own_select(state) if state["op"] == "select" else _own_adamw(state)
    return _plain_select(state) if state["op"] == "select" else _plain_adamw(state)


# ---- 64 bits -------------------------------------------------------------------------------------
def _exact_select(case, s):
    """Picks by k rounds of the largest that is left; weights and gradients by each row's Jacobian at the picks."""
    x, k, E, G = s["logits"].double(), case["k"], case["E"], case["G"]
    T = x.shape[0]
    dead = x == -math.inf
    if case["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    rank_by = x.clone() if s["bias"] is None else p + s["bias"].double()
    if s["bias"] is not None:
        dead |= s["bias"] == -math.inf
    order = torch.arange(E, device=x.device)

    def largest(v, n, names):
        """Positions of each row's n largest, the first of equal ones; -1 where only -inf is left."""
        v, got = v.clone(), []
        for _ in range(n):
            top = v.amax(1, keepdim=True)
            at = torch.where(v == top, names, names.numel()).amin(1, keepdim=True)
            got.append(torch.where(top == -math.inf, -1, at))
            v.scatter_(1, at, -math.inf)
        return torch.cat(got, 1)

    if G > 1:
        c = (p if s["bias"] is None else rank_by).masked_fill(dead, -math.inf).view(T * G, E // G)
        first = c.amax(1)
        value = first
        if case["rank"] == 2 and E // G > 1:
            c = c.scatter(1, largest(c, 1, order[:E // G]).clamp(min=0), -math.inf)
            second = c.amax(1)
            value = first + torch.where(second == -math.inf, torch.zeros_like(second), second)
        groups = largest(value.view(T, G), case["kept"], order[:G])
        stays = (groups[:, :, None] == order[:G]).any(1)
        dead = dead | ~stays[:, order // (E // G)]
    idx = s["idx"].long() if case["dir"] == "bwd" else largest(rank_by.masked_fill(dead, -math.inf), k, order)
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, -1)
    live = (idx >= 0).double()
    at = idx.clamp(min=0)
    u = p.gather(1, at) * live
    a = case["scale"] / u.sum(1, keepdim=True).clamp(min=1e-300) if case["renorm"] else torch.full_like(u[:, :1], case["scale"])
    out = {}
    if case["dir"] != "bwd":
        out.update(idx=None, w=a * u)
    if case["dir"] != "fwd":
        dw = s["dw"].double() * live
        du = a * dw
        if case["renorm"]:
            du = du - a * (dw * a * u).sum(1, keepdim=True) / case["scale"]
        full = torch.zeros_like(x).scatter_add_(1, at, du * live)
        if case["score"] == "sigmoid":
            out["dlogits"] = full * p * torch.sigmoid(-x)
        else:
            out["dlogits"] = p * (full - (p * full).sum(1, keepdim=True))
        if s["bias"] is not None and case["dir"] == "train":
            n = s["counts"].double().sum(0)
            out["bias"] = s["bias"].double() + BIAS_RATE * ((n < n.mean()).double() - (n > n.mean()).double())
    return out


def _exact_adamw(case, s):
    g, p = s["g"].double(), s["p"].double()
    out = {}
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        out["norm"] = torch.stack([norm, torch.clamp(s["most"] / norm, max=1)])
        g = g * out["norm"][1]
    if case["state"] == 8:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (s["r"].double() * s["r_scale"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m, BETAS[0])
    v = torch.lerp(g * g, v, BETAS[1])
    a = m / -math.expm1(case["step"] * math.log(BETAS[0]))
    b = torch.sqrt(v / -math.expm1(case["step"] * math.log(BETAS[1]))) + EPS
    p = p * (1 - LR * DECAY) - LR * a / b
    out["p"] = p
    if s["copy"] is not None:
        out["copy"] = p
    if case["state"] == 32:
        out.update(m=m, v=v)
    else:   # (which way a code is rounded is no number of 64 bits)
        root = torch.sqrt(v)
        out.update(m=None, r=None, m_scale=m.view(-1, BLOCK).abs().amax(1) / 448, r_scale=root.view(-1, BLOCK).amax(1) / 448)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_select(case, s) if case["op"] == "select" else _exact_adamw(case, s)
