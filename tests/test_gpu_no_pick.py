"""MOE_FLAG_NO_PICK in every precision: a layer whose padded tokens have picks of -1, and tokens with fewer picks than k."""
import dataclasses

import numpy as np
import pytest
import torch

from moe_expert_layer_permute_gb300 import inputs as gen

from _layer import DeviceLayer

pytestmark = pytest.mark.gpu


def _layers(moe, precision, share):
    """The same layer with picks of -1, and with those picks at another expert of the token's that weighs 0."""
    cfg = gen.custom_config(T=300, H=256, I=256, E=8, k=3, seed=41, precision=precision)
    inp = gen.make_inputs(cfg)
    rng = np.random.default_rng(int(10 * share))
    idx, w = inp.topk_idx.copy(), inp.topk_w.copy()
    gone = np.repeat(rng.random(cfg.T) < share, cfg.k).reshape(cfg.T, cfg.k)
    gone[:, 2] |= rng.random(cfg.T) < 0.2
    w[gone] = 0
    none = idx.copy()
    none[gone] = -1
    layers = []
    for ids in (none, idx):
        layers.append(DeviceLayer(moe, dataclasses.replace(inp, topk_idx=ids, topk_w=w)))
    return layers, torch.from_numpy(gone).cuda()


@pytest.mark.parametrize("precision,flags", [("bf16", 0), ("bf16", "fused"), ("mxfp8", 0), ("fp8_bwd", 0), ("fp8_fp4", 0)])
@pytest.mark.parametrize("share", [0.15, 0.9, 1.0])
def test_every_precision(cuda_lib, precision, flags, share):
    """Rows are quantised and multiplied one by one, so a pick that weighs 0 adds 0 to what the others give: y is equal bit for bit
    where the order of its sum is fixed; the fused combine adds in fp32 in any order, of at most k terms: 2^-8 of the largest y."""
    (a, b), gone = _layers(cuda_lib, precision, share)
    fused = cuda_lib.MOE_FLAG_FUSED_COMBINE if flags == "fused" else 0
    a.fwd(flags=cuda_lib.MOE_FLAG_NO_PICK | fused)
    b.fwd(flags=fused)
    torch.cuda.synchronize()
    assert a.status() == 0 and b.status() == 0
    none = gone.all(1)
    assert (a.y[none] == 0).all() and torch.isfinite(a.y).all()
    if fused:
        assert float((a.y.float() - b.y.float()).abs().max()) <= 2 ** -8 * float(b.y.float().abs().max())
    else:
        assert torch.equal(a.y, b.y)
    if precision == "fp8_fp4" or fused:
        return
    for L, flag in ((a, cuda_lib.MOE_FLAG_NO_PICK), (b, 0)):
        L.fwd(flags=cuda_lib.MOE_FLAG_SAVE_GU | flag)
        L.bwd(flags=cuda_lib.MOE_FLAG_REUSE_FWD | flag)
    torch.cuda.synchronize()
    assert a.status() == 0
    assert (a.dx[none] == 0).all() and (a.dtw[gone] == 0).all()
    keep = ~gone
    assert torch.equal(a.dtw[keep], b.dtw[keep])
    assert torch.equal(a.dx, b.dx)
    for x, y in ((a.dW13, b.dW13), (a.dW2, b.dW2)):
        assert torch.isfinite(x).all()
        if share == 1.0:
            assert (x == 0).all()
        if precision == "bf16":   # sums of at most 900 rows in another order, 2^-24 each, then each side's rounding, 2^-8
            assert float((x.float() - y.float()).abs().max()) <= (2 ** -7 + 2 ** -14) * float(y.float().abs().max())
