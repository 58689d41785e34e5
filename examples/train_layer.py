"""Trains one MoE layer with its router: the layer's forward and backward, the router's balance loss,
z-loss and gradient, and orthogonalised (Muon) updates of every weight.

    python examples/train_layer.py --steps 100

The data are synthetic: tokens of packed sequences of uneven length with padding, and targets from a fixed
layer of the same shape.  Each step
    logits = x Wr^T            -> moe_router_fwd -> moe_balance_fwd (a loss for each sequence) -> moe_fwd
    dy     = y - target        -> moe_bwd -> moe_balance_bwd (joins the top-k weights' gradient) -> dWr = dlogits^T x
    W     <- W - lr scale O(M)    M a momentum of the gradients, O its orthogonalised form (moe_orthogonalise),
                                  gate and up projections as matrices of their own
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Muon:
    """fp32 master and momentum of weights seen as matrices [N, R, C], and their bf16 copy in the layer."""

    def __init__(self, moe, weight, matrices, lr, momentum=0.9):
        self.moe, self.lr, self.momentum = moe, lr, momentum
        self.weight = weight.view(matrices)
        self.master = self.weight.float()
        self.state = torch.zeros_like(self.master)
        self.update = torch.empty(matrices, dtype=torch.bfloat16, device=weight.device)
        self.workspace = moe.Workspace(moe.moe_orthogonalise_workspace_bytes(*matrices))
        self.scale = max(1.0, matrices[1] / matrices[2]) ** 0.5

    def step(self, grad):
        self.state.mul_(self.momentum).add_(grad.view_as(self.state))
        self.moe.moe_orthogonalise(self.state, self.update, self.workspace)
        self.master.add_(self.update, alpha=-self.lr * self.scale)
        self.weight.copy_(self.master)


def train(steps=100, T=1024, H=256, I=128, E=8, k=2, lr=0.01, balance=0.01, z=1e-3, seed=0, log=print):
    from moe_expert_layer_permute_gb300 import binding as moe
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    bf = torch.bfloat16
    W13, W2 = normal(E, 2 * I, H, std=H ** -0.5).to(bf), normal(E, H, I, std=I ** -0.5).to(bf)
    # a router that starts out lopsided: without the balance loss it would stay so
    Wr = normal(E, H, std=0.3 * H ** -0.5)
    Wr[0] *= 8
    x = (normal(T, H) + 0.5 * normal(1, H)).to(bf)
    # the targets: a fixed layer's answers, each token through its first expert
    teacher13, teacher2 = normal(E, 2 * I, H, std=H ** -0.5).to(bf), normal(E, H, I, std=I ** -0.5).to(bf)
    scratch = moe.Scratch(T, H, I, E, k)
    idx, w = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    target, y = torch.empty(T, H, dtype=bf, device=dev), torch.empty(T, H, dtype=bf, device=dev)
    moe.moe_router_fwd(normal(T, E), idx, w)
    moe.moe_fwd(x, idx, w, teacher13, teacher2, target, scratch)

    cuts = torch.sort(torch.randperm(T - 1, generator=g, device=dev)[:5] + 1).values.int()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), cuts, torch.full((1,), T, dtype=torch.int32, device=dev)])
    B = offsets.numel() - 1
    mask = torch.rand(T, generator=g, device=dev) < 0.9            # padding
    counts, tokens = torch.empty(B, E, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    losses, dloss = torch.empty(B, 2, device=dev), torch.tensor([[balance, z]], device=dev).repeat(B, 1) / B
    workspace = moe.Workspace(moe.moe_balance_workspace_bytes(T, E, B))

    dx, dW13, dW2 = torch.empty_like(x), torch.empty_like(W13, dtype=torch.float32), torch.empty_like(W2, dtype=torch.float32)
    dw, dlogits = torch.empty(T, k, device=dev), torch.empty(T, E, device=dev)
    experts = [Muon(moe, W13, (2 * E, I, H), lr), Muon(moe, W2, (E, H, I), lr)]
    router = Muon(moe, Wr, (1, E, H), lr)
    history = []
    for step in range(steps):
        logits = x.float() @ Wr.t()
        moe.moe_router_fwd(logits, idx, w)
        moe.moe_balance_fwd(logits, idx, counts, tokens, losses, workspace, mask=mask, seg_offsets=offsets)
        moe.moe_fwd(x, idx, w, W13, W2, y, scratch, flags=moe.MOE_FLAG_SAVE_GU)
        error = (y.float() - target.float()) * mask[:, None]
        dy = (error / mask.sum()).to(bf)
        moe.moe_bwd(dy, x, idx, w, W13, W2, dx, dW13, dW2, dw, scratch, flags=moe.MOE_FLAG_REUSE_FWD)
        moe.moe_balance_bwd(logits, idx, w, dw, counts, tokens, dloss, dlogits, mask=mask, seg_offsets=offsets)
        router.step(dlogits.t() @ x.float())
        for weight, grad in zip(experts, (dW13, dW2)):
            weight.step(grad)
        scratch.epoch += 1                                          # the weights changed in place
        share = counts.sum(0).float()
        history.append((float(error.square().mean()), float(losses[:, 0].mean()), float(losses[:, 1].mean()),
                        float(share.max() / share.mean())))
        if log and (step % 10 == 0 or step + 1 == steps):
            log("step %3d  error %.4f  balance %.4f  z %.3f  busiest expert %.2f times the mean" % ((step,) + history[-1]))
    for holder in [scratch] + [m.workspace for m in experts + [router]]:
        if moe.moe_read_device_status(holder) != 0:
            raise RuntimeError("device status set")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    from moe_expert_layer_permute_gb300 import build
    build.build()
    train(steps=args.steps, seed=args.seed)
