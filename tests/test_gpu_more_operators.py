"""Routing by scores, the layer, the norm and AdamW together, as a training step has them; -1 picks in the layer."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from moe_expert_layer_permute_gb300 import inputs as gen

from _layer import DeviceLayer, f64, rel_fro

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_pick_is_dropped_and_not_recorded(cuda_lib):
    """With MOE_FLAG_NO_PICK an id of -1 is no error, any other bad id still is; the result is the layer over the others."""
    moe = cuda_lib
    cfg = gen.custom_config(T=256, H=256, I=128, E=8, k=2, seed=38)
    inp = gen.make_inputs(cfg)
    idx = inp.topk_idx.copy()
    idx[5] = -1
    idx[9, 1] = -1
    inp.topk_idx = idx
    L = DeviceLayer(moe, inp)
    outs = []
    for flags in (0, moe.MOE_FLAG_NO_PICK):
        L.fwd(flags=moe.MOE_FLAG_SAVE_GU | flags)
        L.bwd(flags=moe.MOE_FLAG_REUSE_FWD | flags)
        torch.cuda.synchronize()
        assert L.status() == (0 if flags else moe.MOE_DEV_BAD_EXPERT)
        outs.append([t.clone() for t in (L.y, L.dx, L.dW13, L.dW2, L.dtw)])
        L.bwd(flags=flags)                                    # with its own routing
        torch.cuda.synchronize()
        assert L.status() == (0 if flags else moe.MOE_DEV_BAD_EXPERT)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    keep = idx >= 0
    w = np.where(keep, inp.topk_w, 0.0)
    y = oracle.forward(inp.f64("x"), np.where(keep, idx, 0), w, inp.f64("W13"), inp.f64("W2"))
    assert rel_fro(f64(L.y), y) < 1e-2 and (L.y[5] == 0).all() and (L.dx[5] == 0).all() and (L.dtw[~torch.from_numpy(keep).cuda()] == 0).all()
    idx[3, 0] = 8
    L.idx.copy_(torch.from_numpy(idx))
    L.fwd(flags=moe.MOE_FLAG_NO_PICK)
    torch.cuda.synchronize()
    assert L.status() == moe.MOE_DEV_BAD_EXPERT


def test_selection_and_layer_chain(cuda_lib):
    """logits -> selection -> layer forward and backward -> selection's gradient, against the oracle's layer and autograd."""
    moe = cuda_lib
    cfg = gen.custom_config(T=256, H=256, I=128, E=16, k=3, seed=39)
    inp = gen.make_inputs(cfg)
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(cfg.T, cfg.E, generator=g)
    mask = torch.rand(cfg.T, generator=g) < 0.85
    bias = 0.1 * torch.randn(cfg.E, generator=g)
    rule = moe.RouterRule(score="sigmoid", groups=4, topk_groups=2, group_rank=2, scale=2.0)
    L = DeviceLayer(moe, inp)
    lg = logits.cuda()
    moe.moe_router_select_fwd(lg, L.idx, L.w, rule, bias=bias.cuda(), mask=mask.cuda())
    L.fwd(flags=moe.MOE_FLAG_SAVE_GU | moe.MOE_FLAG_NO_PICK)
    L.bwd(flags=moe.MOE_FLAG_REUSE_FWD | moe.MOE_FLAG_NO_PICK)
    dl = torch.empty(cfg.T, cfg.E, device="cuda")
    moe.moe_router_select_bwd(lg, L.idx, L.w, L.dtw, dl, rule)
    counts = L.view(moe.MOE_VIEW_COUNTS, torch.int32, (1, cfg.E)).clone()
    torch.cuda.synchronize()
    assert L.status() == 0
    idx = L.idx.cpu().long()
    assert (idx[~mask] == -1).all() and (idx[mask] >= 0).all()
    assert torch.equal(counts[0].cpu(), torch.bincount(idx[mask].flatten(), minlength=cfg.E).int())
    x = logits.double().requires_grad_(True)
    live = (idx >= 0).double()
    u = torch.sigmoid(x).gather(1, idx.clamp(min=0)) * live
    w = 2.0 * u / u.sum(1, keepdim=True).clamp(min=1e-300)
    args = (inp.f64("x"), idx.clamp(min=0).numpy(), w.detach().numpy(), inp.f64("W13"), inp.f64("W2"))
    assert rel_fro(f64(L.y), oracle.forward(*args)) < 1e-2
    ref = oracle.backward(inp.f64("dy"), *args)
    (w * torch.from_numpy(ref["dtopk_w"]) * live).sum().backward()
    assert rel_fro(f64(dl), x.grad.numpy()) < 1e-2


def test_example_with_a_bias_runs(cuda_lib):
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.train(steps=25, routing="bias", log=None)
    assert len(history) == 25 and all(np.isfinite(h).all() for h in history)
