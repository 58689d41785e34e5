"""ctypes binding of the MoE layer's C ABI (`include/moe_layer.h`).

Argument marshalling only: torch tensors become `moe_tensor` views (device pointer, dtype,
shape, strides), the current torch CUDA stream becomes the `stream` argument, and every step of
the layer runs in the CUDA library.  The balance loss, the orthogonalisation, the routing by scores and AdamW marshal in C++
(`csrc/marshal.cpp`), since their smallest calls take a few microseconds.  The library is loaded on
import, the compiled marshalling by the first call that wants it; if they have not been built, that raises
(there is no fallback).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build as _build

# ---- C structures ---------------------------------------------------------------------------
MOE_BF16, MOE_MXFP8, MOE_FP8_BWD, MOE_FP8_FP4 = 0, 1, 2, 3
MOE_DT_BF16, MOE_DT_F32, MOE_DT_I32, MOE_DT_U8, MOE_DT_E4M3 = 0, 1, 2, 3, 4
MOE_FLAG_SAVE_GU, MOE_FLAG_REUSE_FWD, MOE_FLAG_REUSE_WEIGHTS, MOE_FLAG_FUSED_COMBINE = 0x1, 0x2, 0x4, 0x8
MOE_FLAG_NO_PICK = 0x10
(MOE_VIEW_COUNTS, MOE_VIEW_OFFSETS, MOE_VIEW_PERM, MOE_VIEW_INV, MOE_VIEW_PAD_OFFSETS, MOE_VIEW_XPERM,
 MOE_VIEW_HID, MOE_VIEW_GU, MOE_VIEW_YPART, MOE_VIEW_DG, MOE_VIEW_HW, MOE_VIEW_DYPERM) = range(12)
MOE_DEV_OK, MOE_DEV_BAD_EXPERT, MOE_DEV_TIMEOUT = 0, 1, 2
MOE_TEST_WITHHOLD_LOADS = 0x1
MX_VIEWS = {name: 32 + i for i, name in enumerate(
    ["x_r", "x_r_sf", "x_c", "x_c_sf", "h_r", "h_r_sf", "dy_r", "dy_r_sf", "dy_c", "dy_c_sf", "dg_r", "dg_r_sf",
     "dg_c", "dg_c_sf", "hw_c", "hw_c_sf", "w13_r", "w13_r_sf", "w13_c", "w13_c_sf", "w2_r", "w2_r_sf", "w2_c",
     "w2_c_sf"])}
ERRORS = {0: "MOE_OK", -1: "MOE_ERR_NULL", -2: "MOE_ERR_SHAPE", -3: "MOE_ERR_DTYPE", -4: "MOE_ERR_LAYOUT",
          -5: "MOE_ERR_ALIGN", -6: "MOE_ERR_SCRATCH", -7: "MOE_ERR_STATE", -8: "MOE_ERR_UNSUPPORTED",
          -9: "MOE_ERR_CUDA", -10: "MOE_ERR_DEVICE"}
ERR = {v: k for k, v in ERRORS.items()}

# every symbol the header declares
EXPORTS = ("moe_scratch_bytes", "moe_fwd", "moe_bwd", "moe_read_device_status", "moe_strerror",
           "moe_scratch_view", "moe_trace_enable", "moe_trace_reset", "moe_trace_read", "moe_route_static",
           "moe_router_fwd", "moe_router_bwd", "moe_set_wait_limit", "moe_balance_workspace_bytes", "moe_balance_fwd",
           "moe_balance_bwd", "moe_orthogonalise_workspace_bytes", "moe_orthogonalise", "moe_router_select_fwd",
           "moe_router_select_bwd", "moe_router_bias_step", "moe_adamw_step", "moe_grad_norm_workspace_bytes", "moe_grad_norm")


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 3), ("stride", ctypes.c_int64 * 3)]


class MoeDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64), ("E", ctypes.c_int64),
                ("k", ctypes.c_int64), ("precision", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class MoeScratch(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("bytes", ctypes.c_uint64), ("desc", MoeDesc),
                ("epoch", ctypes.c_uint64), ("state", ctypes.c_uint64 * 4)]


class MoeRouterRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_rank", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoeAdamwOptions(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
        [("step", ctypes.c_int64), ("seed", ctypes.c_uint64)] + \
        [(n, ctypes.POINTER(MoeTensor)) for n in ("lr_on_device", "step_on_device", "grad_scale")]


_P = ctypes.POINTER


def _load() -> ctypes.CDLL:
    path = _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built ({path}); run moe_expert_layer_permute_gb300.build.build()")
    lib = ctypes.CDLL(path)
    lib.moe_scratch_bytes.argtypes = [_P(MoeDesc)]
    lib.moe_scratch_bytes.restype = ctypes.c_size_t
    lib.moe_fwd.argtypes = [_P(MoeTensor)] * 6 + [_P(MoeScratch), ctypes.c_void_p]
    lib.moe_fwd.restype = ctypes.c_int
    lib.moe_bwd.argtypes = [_P(MoeTensor)] * 10 + [_P(MoeScratch), ctypes.c_void_p]
    lib.moe_bwd.restype = ctypes.c_int
    lib.moe_read_device_status.argtypes = [_P(MoeScratch), ctypes.c_void_p, _P(ctypes.c_int)]
    lib.moe_read_device_status.restype = ctypes.c_int
    lib.moe_strerror.argtypes = [ctypes.c_int]
    lib.moe_strerror.restype = ctypes.c_char_p
    lib.moe_scratch_view.argtypes = [_P(MoeDesc), ctypes.c_int, _P(ctypes.c_uint64), _P(ctypes.c_uint64)]
    lib.moe_scratch_view.restype = ctypes.c_int
    lib.moe_trace_enable.argtypes = [ctypes.c_int]
    lib.moe_trace_enable.restype = ctypes.c_int
    lib.moe_trace_reset.argtypes = []
    lib.moe_trace_reset.restype = ctypes.c_int
    lib.moe_trace_read.argtypes = [_P(ctypes.c_char_p), _P(ctypes.c_int64), _P(ctypes.c_double), _P(ctypes.c_int)]
    lib.moe_trace_read.restype = ctypes.c_int
    lib.moe_route_static.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64] + \
        [ctypes.c_void_p] * 5
    lib.moe_route_static.restype = ctypes.c_int
    lib.moe_router_fwd.argtypes = [_P(MoeTensor)] * 3 + [ctypes.c_void_p]
    lib.moe_router_fwd.restype = ctypes.c_int
    lib.moe_router_bwd.argtypes = [_P(MoeTensor)] * 4 + [ctypes.c_void_p]
    lib.moe_router_bwd.restype = ctypes.c_int
    lib.moe_set_wait_limit.argtypes = [_P(MoeScratch), ctypes.c_int64, ctypes.c_uint32]
    lib.moe_set_wait_limit.restype = ctypes.c_int
    lib.moe_balance_workspace_bytes.argtypes = [ctypes.c_int64] * 3
    lib.moe_balance_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_balance_fwd.argtypes = [_P(MoeTensor)] * 7 + [_P(MoeScratch), ctypes.c_void_p]
    lib.moe_balance_fwd.restype = ctypes.c_int
    lib.moe_balance_bwd.argtypes = [_P(MoeTensor)] * 10 + [ctypes.c_void_p]
    lib.moe_balance_bwd.restype = ctypes.c_int
    lib.moe_orthogonalise_workspace_bytes.argtypes = [ctypes.c_int64] * 3
    lib.moe_orthogonalise_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_orthogonalise.argtypes = [_P(MoeTensor)] * 2 + [ctypes.c_int32, _P(ctypes.c_float), ctypes.c_float,
                                                            _P(MoeScratch), ctypes.c_void_p]
    lib.moe_orthogonalise.restype = ctypes.c_int
    lib.moe_router_select_fwd.argtypes = [_P(MoeTensor)] * 5 + [_P(MoeRouterRule), ctypes.c_void_p]
    lib.moe_router_select_fwd.restype = ctypes.c_int
    lib.moe_router_select_bwd.argtypes = [_P(MoeTensor)] * 5 + [_P(MoeRouterRule), ctypes.c_int32, ctypes.c_void_p]
    lib.moe_router_select_bwd.restype = ctypes.c_int
    lib.moe_router_bias_step.argtypes = [_P(MoeTensor)] * 2 + [ctypes.c_float, ctypes.c_void_p]
    lib.moe_router_bias_step.restype = ctypes.c_int
    lib.moe_adamw_step.argtypes = [ctypes.c_int64] + [_P(MoeTensor)] * 7 + [_P(MoeAdamwOptions), ctypes.c_void_p]
    lib.moe_adamw_step.restype = ctypes.c_int
    lib.moe_grad_norm_workspace_bytes.argtypes = [ctypes.c_int64] * 2
    lib.moe_grad_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_grad_norm.argtypes = [ctypes.c_int64] + [_P(MoeTensor)] * 2 + [ctypes.c_float, _P(MoeScratch), ctypes.c_void_p]
    lib.moe_grad_norm.restype = ctypes.c_int
    return lib


LIB = _load()


_MARSHAL = None


def _marshal():
    """The compiled marshalling (`csrc/marshal.cpp`), linked against the library loaded above."""
    global _MARSHAL
    if _MARSHAL is None:
        if not os.path.exists(_build.MARSHAL):
            raise RuntimeError(f"marshalling not built ({_build.MARSHAL}); run moe_expert_layer_permute_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("_marshal", _build.MARSHAL)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _MARSHAL = module
    return _MARSHAL


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {ERRORS.get(code, code)} ({strerror(code)})")


def strerror(code: int) -> str:
    return LIB.moe_strerror(code).decode()


_DT = {torch.bfloat16: MOE_DT_BF16, torch.float32: MOE_DT_F32, torch.int32: MOE_DT_I32, torch.uint8: MOE_DT_U8,
       torch.bool: MOE_DT_U8}


def as_moe_tensor(t: torch.Tensor) -> MoeTensor:
    m = MoeTensor()
    m.data = t.data_ptr() if t.numel() else 0
    m.dtype = _DT.get(t.dtype, -1)
    m.ndim = t.dim()
    for i in range(min(t.dim(), 3)):
        m.shape[i] = t.shape[i]
        m.stride[i] = t.stride(i)
    return m


def make_desc(T, H, I, E, k, precision=MOE_BF16, flags=0) -> MoeDesc:
    return MoeDesc(T, H, I, E, k, precision, flags)


def moe_scratch_bytes(desc: MoeDesc) -> int:
    return int(LIB.moe_scratch_bytes(ctypes.byref(desc)))


def view_span(desc: MoeDesc, which: int) -> tuple:
    """(byte offset, byte count) of a named scratch region for `desc` (moe_scratch_view)."""
    off, nbytes = ctypes.c_uint64(), ctypes.c_uint64()
    rc = LIB.moe_scratch_view(ctypes.byref(desc), which, ctypes.byref(off), ctypes.byref(nbytes))
    if rc:
        raise MoeError(rc, "moe_scratch_view")
    return off.value, nbytes.value


class Scratch:
    """A caller-owned device scratch buffer (a torch uint8 tensor) and its C handle."""

    def __init__(self, T, H, I, E, k, precision=MOE_BF16, device="cuda"):
        desc = make_desc(T, H, I, E, k, precision)
        n = moe_scratch_bytes(desc)
        if n == 0:
            raise MoeError(ERR["MOE_ERR_SHAPE"], "moe_scratch_bytes")
        self.buffer = torch.zeros(n, dtype=torch.uint8, device=device)
        self.handle = MoeScratch()
        self.handle.data = self.buffer.data_ptr()
        self.handle.bytes = n
        self.handle.desc = desc

    @property
    def desc(self) -> MoeDesc:
        return self.handle.desc

    @property
    def epoch(self) -> int:
        """The caller's counter of in-place updates of x / W13 / W2 (see MOE_FLAG_REUSE_*)."""
        return int(self.handle.epoch)

    @epoch.setter
    def epoch(self, value: int) -> None:
        self.handle.epoch = value

    def set_wait_limit(self, cycles: int = 0, test_flags: int = 0) -> None:
        """Pipeline wait limit in SM cycles for later calls (0: the default) and MOE_TEST_* flags."""
        rc = LIB.moe_set_wait_limit(ctypes.byref(self.handle), cycles, test_flags)
        if rc:
            raise MoeError(rc, "moe_set_wait_limit")

    def view(self, which: int, dtype: torch.dtype, shape) -> torch.Tensor:
        off, nbytes = view_span(self.handle.desc, which)
        raw = self.buffer[off:off + nbytes]
        return raw.view(dtype).view(*shape)


class Workspace:
    """A caller-owned device buffer and its C handle for moe_balance_fwd, moe_orthogonalise and moe_grad_norm (their
    *_workspace_bytes); moe_read_device_status takes it as it takes a Scratch.  One that moe_orthogonalise
    has used is no longer zero, and moe_balance_fwd and moe_grad_norm refuse it; moe_balance_fwd refuses one of moe_grad_norm too."""

    def __init__(self, nbytes: int, device="cuda"):
        if nbytes <= 0:
            raise MoeError(ERR["MOE_ERR_UNSUPPORTED"], "Workspace")
        self.buffer = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.handle = MoeScratch()
        self.handle.data = self.buffer.data_ptr()
        self.handle.bytes = nbytes
        self.address = ctypes.addressof(self.handle)

    set_wait_limit = Scratch.set_wait_limit


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def moe_fwd(x, topk_idx, topk_w, W13, W2, y, scratch: Scratch, stream=None, flags: int = 0) -> None:
    scratch.handle.desc.flags = flags
    args = [as_moe_tensor(t) for t in (x, topk_idx, topk_w, W13, W2, y)]
    rc = LIB.moe_fwd(*[ctypes.byref(a) for a in args], ctypes.byref(scratch.handle), _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_fwd")


def moe_bwd(dy, x, topk_idx, topk_w, W13, W2, dx, dW13, dW2, dtopk_w, scratch: Scratch, stream=None,
            flags: int = 0) -> None:
    scratch.handle.desc.flags = flags
    args = [as_moe_tensor(t) for t in (dy, x, topk_idx, topk_w, W13, W2, dx, dW13, dW2, dtopk_w)]
    rc = LIB.moe_bwd(*[ctypes.byref(a) for a in args], ctypes.byref(scratch.handle), _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_bwd")


def moe_read_device_status(scratch: Scratch, stream=None) -> int:
    st = ctypes.c_int(0)
    rc = LIB.moe_read_device_status(ctypes.byref(scratch.handle), _stream_ptr(stream), ctypes.byref(st))
    if rc:
        raise MoeError(rc, "moe_read_device_status")
    return st.value


def moe_trace_enable(on: bool) -> None:
    LIB.moe_trace_enable(1 if on else 0)


def moe_trace_reset() -> None:
    LIB.moe_trace_reset()


def moe_trace_read() -> dict:
    """{kernel name: (launches, total ms)} of the launches recorded since the last reset."""
    cap = 64
    names = (ctypes.c_char_p * cap)()
    launches = (ctypes.c_int64 * cap)()
    ms = (ctypes.c_double * cap)()
    n = ctypes.c_int(cap)
    LIB.moe_trace_read(names, launches, ms, ctypes.byref(n))
    return {names[i].decode(): (int(launches[i]), float(ms[i])) for i in range(min(n.value, cap))}


def moe_route_static(topk_idx, E: int, counts, offsets, perm, inv, stream=None) -> None:
    """Routing bookkeeping into caller-owned int32 tensors, with no scratch buffer (the library's
    static device array instead): counts [E], offsets [E+1], perm [T*k], inv [T*k]."""
    T, k = topk_idx.shape
    for t in (topk_idx, counts, offsets, perm, inv):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise MoeError(ERR["MOE_ERR_DTYPE"], "moe_route_static")
    if counts.numel() != E or offsets.numel() != E + 1 or perm.numel() != T * k or inv.numel() != T * k:
        raise MoeError(ERR["MOE_ERR_SHAPE"], "moe_route_static")
    rc = LIB.moe_route_static(topk_idx.data_ptr(), T, k, E, counts.data_ptr(), offsets.data_ptr(),
                              perm.data_ptr(), inv.data_ptr(), _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_route_static")


def moe_router_fwd(logits, topk_idx, topk_w, stream=None) -> None:
    """Top-k router: logits fp32 [T, E] -> topk_idx int32 [T, k], topk_w fp32 [T, k]."""
    args = [as_moe_tensor(t) for t in (logits, topk_idx, topk_w)]
    rc = LIB.moe_router_fwd(*[ctypes.byref(a) for a in args], _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_router_fwd")


def moe_router_bwd(topk_idx, topk_w, dtopk_w, dlogits, stream=None) -> None:
    """Router backward: dlogits fp32 [T, E] from the weights' gradient dtopk_w fp32 [T, k]."""
    args = [as_moe_tensor(t) for t in (topk_idx, topk_w, dtopk_w, dlogits)]
    rc = LIB.moe_router_bwd(*[ctypes.byref(a) for a in args], _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_router_bwd")


class RouterRule:
    """How moe_router_select_fwd chooses and weighs: score "softmax" or "sigmoid", groups of consecutive experts of which
    topk_groups stay (by the sum of their group_rank largest), weights renormalised over the picks or not, their scale."""

    SCORES = {"softmax": 0, "sigmoid": 1}

    def __init__(self, score="softmax", groups=1, topk_groups=1, group_rank=1, renormalise=True, scale=1.0):
        if score not in self.SCORES:
            raise MoeError(ERR["MOE_ERR_UNSUPPORTED"], "RouterRule")
        if any(abs(n) > 2 ** 31 - 1 for n in (groups, topk_groups, group_rank)):   # (a field takes a number modulo 2^32)
            raise MoeError(ERR["MOE_ERR_UNSUPPORTED"], "RouterRule")
        self.handle = MoeRouterRule(self.SCORES[score], groups, topk_groups, group_rank, 1 if renormalise else 0, scale)
        self.address = ctypes.addressof(self.handle)


def moe_router_select_fwd(logits, topk_idx, topk_w, rule: RouterRule, bias=None, mask=None, stream=None) -> None:
    """Routing by scores: logits fp32 or bf16 [T, E], bias fp32 [E] or None, mask bool or uint8 [T] or None -> topk_idx
    int32 [T, k] (-1 where there is no pick), topk_w fp32 [T, k]."""
    rc = (_MARSHAL or _marshal()).select_fwd(logits, bias, mask, topk_idx, topk_w, rule.address,
                                             None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_router_select_fwd")


def moe_router_select_bwd(logits, topk_idx, topk_w, dtopk_w, dlogits, rule: RouterRule, accumulate: bool = False,
                          stream=None) -> None:
    """dlogits [T, E] (fp32 or bf16; fp32 with accumulate, which adds to it) from the weights' gradient dtopk_w fp32 [T, k]."""
    rc = (_MARSHAL or _marshal()).select_bwd(logits, topk_idx, topk_w, dtopk_w, dlogits, rule.address, accumulate,
                                             None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_router_select_bwd")


def moe_router_bias_step(counts, bias, rate: float, stream=None) -> None:
    """bias fp32 [E] += rate * sign(mean - n), n the sums of counts int32 [B, E] over B."""
    rc = (_MARSHAL or _marshal()).bias_step(counts, bias, rate, None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_router_bias_step")


def moe_balance_workspace_bytes(T: int, E: int, B: int = 1) -> int:
    return int(LIB.moe_balance_workspace_bytes(T, E, B))


def moe_balance_fwd(logits, topk_idx, counts, tokens, loss, workspace: Workspace, mask=None, seg_offsets=None,
                    stream=None) -> None:
    """Balance loss, z-loss and per-expert counts of each segment: logits fp32 [T, E], topk_idx int32
    [T, k], mask bool or uint8 [T] or None, seg_offsets int32 [B+1] or None (B = 1) -> counts int32
    [B, E], tokens int32 [B], loss fp32 [B, 2]."""
    rc = (_MARSHAL or _marshal()).balance_fwd(logits, topk_idx, mask, seg_offsets, counts, tokens, loss, workspace.address,
                              None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_balance_fwd")


def moe_balance_bwd(logits, topk_idx, topk_w, dtopk_w, counts, tokens, dloss, dlogits, mask=None, seg_offsets=None,
                    stream=None) -> None:
    """dlogits fp32 [T, E] of the losses (dloss fp32 [B, 2]) and, unless topk_w and dtopk_w are None,
    of the top-k weights (what moe_router_bwd gives), in one pass."""
    rc = (_MARSHAL or _marshal()).balance_bwd(logits, topk_idx, topk_w, dtopk_w, mask, seg_offsets, counts, tokens, dloss, dlogits,
                              None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_balance_bwd")


def moe_orthogonalise_workspace_bytes(N: int, R: int, C: int) -> int:
    return int(LIB.moe_orthogonalise_workspace_bytes(N, R, C))


def _triples(coeffs, steps: int) -> list:
    """The numbers of one triple for every step, or of a triple for each; a sequence, an array or a tensor."""
    def plain(v):
        return v.tolist() if hasattr(v, "tolist") else v
    rows = plain(coeffs)
    if len(rows) == 3 and isinstance(rows[0], (int, float)):
        return list(rows) * max(steps, 1)
    rows = [plain(c) for c in rows]
    if rows and not hasattr(rows[0], "__len__"):
        rows = [rows] * max(steps, 1)
    if not rows or any(len(c) != 3 for c in rows):   # (their number the call checks)
        raise MoeError(ERR["MOE_ERR_SHAPE"], "moe_orthogonalise")
    return [v for c in rows for v in c]


def moe_orthogonalise(G, O, workspace: Workspace, steps: int = 5, coeffs=None, eps: float = 1e-7, stream=None) -> None:
    """O bf16 [N, R, C] = every matrix of G (bf16 or fp32, [N, R, C]) after `steps` Newton-Schulz steps.
    coeffs: (a, b, c) for every step, a sequence of `steps` such triples (numbers, arrays or tensors), or None for the
    defaults."""
    co = () if coeffs is None else _triples(coeffs, steps)
    rc = (_MARSHAL or _marshal()).orthogonalise(G, O, workspace.address, None if stream is None else _stream_ptr(stream), steps, eps, *co)
    if rc:
        raise MoeError(rc, "moe_orthogonalise")


class TensorList:
    """Tensors for moe_adamw_step and moe_grad_norm, which take any sequence of them; of one of these the views are made once for as
    many calls as there are (a call of 240 tensors' lists takes some 20 us less).  It holds its tensors: what is done to them in
    place, `.data` set to other memory or sizes included, counts from the next call on, but a `.grad` that was set to None and made
    anew is another tensor and wants another list."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.capsule = _marshal().make_list(self.tensors)

    def __len__(self):
        return len(self.tensors)


def _list(tensors):
    if tensors is None:
        return None
    return (tensors if isinstance(tensors, TensorList) else TensorList(tensors)).capsule


def moe_adamw_step(params, grads, m, v, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, m_scales=None,
                   v_scales=None, copies=None, grad_scale=None, seed: int | None = None, stream=None) -> None:
    """One AdamW step over lists of tensors, in place: params fp32, grads fp32 or bf16, m and v fp32, or float8_e4m3fn (or
    uint8) with m_scales and v_scales fp32 [ceil(n / 256)]; copies bf16, or None.  step and lr are numbers, or tensors
    of one element on the device (int32, fp32); grad_scale fp32 [1] on the device, or None: a factor of the gradients, no
    step where it is not finite, nor at a step on the device below 1.  seed: of the 8-bit states' rounding, the step's
    number if None; it has to be another one for each step (a step on the device is added to it), since a state that meets the
    same bits each time stays where it is."""
    step_at = step if isinstance(step, torch.Tensor) else None
    lr_at = lr if isinstance(lr, torch.Tensor) else None
    if seed is None:
        seed = 0 if step_at is not None else step
    rc = (_MARSHAL or _marshal()).adamw_step(_list(params), _list(grads), _list(m), _list(v), _list(m_scales), _list(v_scales), _list(copies),
                                             0.0 if lr_at is not None else lr, betas[0], betas[1], eps, weight_decay,
                                             0 if step_at is not None else step, seed, lr_at, step_at, grad_scale,
                                             None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_adamw_step")


def moe_grad_norm_workspace_bytes(elements: int, count: int) -> int:
    return int(LIB.moe_grad_norm_workspace_bytes(elements, count))


def moe_grad_norm(grads, out, workspace: Workspace, max_norm: float = 0.0, stream=None) -> None:
    """out fp32 [2] = (norm of all gradients, the factor min(1, max_norm / norm) that brings it to max_norm; 1 with
    max_norm 0).  out[1:] is a grad_scale for moe_adamw_step."""
    room = getattr(workspace, "buffer", None)
    if room is not None and isinstance(out, torch.Tensor) and room.device != out.device:   # (out and grads are compared by the call)
        raise ValueError("tensors of several devices")
    rc = (_MARSHAL or _marshal()).grad_norm(_list(grads), out, max_norm, workspace.address, None if stream is None else _stream_ptr(stream))
    if rc:
        raise MoeError(rc, "moe_grad_norm")
