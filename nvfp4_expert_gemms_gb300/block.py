"""Binding of the operators around the experts (include/moe_gb300.h, "operators around the
experts"): the norms on the way into and out of a block, scored routing, request adapters, and
MoEBlock, which runs them with a layer of packed experts.

Tensors are checked here (shapes, types, device, contiguity of rows), since the C side sees only
pointers; every refusal is a MoEError with the status the C side would give.  Matrices are [rows,
columns] with unit column stride and any row stride.  Outputs that are not given are allocated by
torch on the tensors' device; work goes to `stream`, or torch's current one.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import MoEError, MoELayer, PackedDesc, _check, lib, moe_status_string

_DT = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}
_KIND = {"rms": 1, "layer": 2}
_GATE = {"none": 0, "linear": 0, "sigmoid": 1, "tanh": 2}
_SCORE = {"softmax": 1, "sigmoid": 2}

INVALID_ARG, UNSUPPORTED = 1, 2


class _NormDesc(C.Structure):
    _fields_ = [("kind", C.c_int32), ("dtype", C.c_int32), ("eps", C.c_float), ("weight_offset", C.c_float),
                ("weight", C.c_void_p), ("bias", C.c_void_p)]


class _RouterDesc(C.Structure):
    _fields_ = [("score", C.c_int32), ("groups", C.c_int32), ("top_groups", C.c_int32), ("group_top", C.c_int32),
                ("renormalize", C.c_int32), ("scale", C.c_float)]


def _refuse(where: str, why: str, status: int = INVALID_ARG):
    e = MoEError(status, where)
    e.args = (f"{where}: {why}: {moe_status_string(status)} (status {status})",)
    raise e


_fns = None


def _f():
    """The C functions with their argument types, resolved once."""
    global _fns
    if _fns is None:
        L = lib()
        P, I, Q, F = C.c_void_p, C.c_int, C.c_int64, C.c_float
        L.moe_block_enter.argtypes = [P, Q, I, P, P, Q, I, I, I, P]
        L.moe_block_leave.argtypes = [P, Q, I, P, Q, I, P, P, Q, I, I, I, F, F, P, P, Q, P, Q, I, I, P]
        L.moe_route_scored.argtypes = [P, P, Q, I, P, I, I, I, P, P, P]
        L.moe_layer_forward_scored.argtypes = [P, P, P, Q, I, P, I, C.POINTER(PackedDesc), P, I, P, P, C.c_size_t, P]
        L.moe_adapters_add.argtypes = [P, Q, P, Q, P, P, P, P, P, P, P, Q] + [I] * 6 + [P]
        _fns = L
    return _fns


def _stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _matrix(t, where, name, rows=None, cols=None, dtype=None, device=None):
    """Row pitch of a [rows, cols] tensor with unit column stride."""
    if t.dim() != 2 or not t.is_cuda or t.dtype not in _DT:
        _refuse(where, f"{name} is not a 2-D CUDA tensor of bf16, fp16 or fp32")
    if (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        _refuse(where, f"{name} has shape {tuple(t.shape)}, not {(rows, cols)}")
    if dtype is not None and t.dtype != dtype:
        _refuse(where, f"{name} has type {t.dtype}, not {dtype}")
    if device is not None and t.device != device:
        _refuse(where, f"{name} is on {t.device}, not {device}")
    ld, step = t.stride()
    if t.shape[0] <= 1:
        ld = max(ld, t.shape[1])
    if (step != 1 and t.shape[1] > 1) or ld < t.shape[1]:
        _refuse(where, f"{name} needs unit column stride and rows that do not overlap")
    return ld


def _vector(t, where, name, n, dtype, device):
    """Address of a contiguous [n] tensor of the given type, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or t.device != device or not t.is_contiguous():
        _refuse(where, f"{name} is not a contiguous {dtype} [{n}] on {device}")
    return t.data_ptr()


class Norm:
    """A norm's kind and parameters: v / rms(v) ("rms") or (v - mean) / std ("layer"), times
    weight + offset, plus bias (both optional, [H], one type)."""

    def __init__(self, kind="rms", weight=None, bias=None, eps=1e-6, offset=0.0):
        where = "Norm"
        if kind not in _KIND:
            _refuse(where, f"unknown kind {kind!r}")
        if not eps > 0.0:
            _refuse(where, "eps must be positive")
        given = [t for t in (weight, bias) if t is not None]
        for t in given:
            if t.dim() != 1 or not t.is_cuda or not t.is_contiguous() or t.dtype not in _DT:
                _refuse(where, "weight and bias are contiguous [H] CUDA tensors of bf16, fp16 or fp32")
            if t.dtype != given[0].dtype or t.shape != given[0].shape or t.device != given[0].device:
                _refuse(where, "weight and bias differ in type, size or device")
        self.weight, self.bias = weight, bias  # kept alive with the addresses below
        self.size = given[0].shape[0] if given else None
        self.device = given[0].device if given else None
        self.desc = _NormDesc(_KIND[kind], _DT[given[0].dtype] if given else 1, eps, offset,
                              weight.data_ptr() if weight is not None else None,
                              bias.data_ptr() if bias is not None else None)
        self._ref = C.addressof(self.desc)

    def _at(self, where, H, device):
        if self.size is not None and (self.size != H or self.device != device):
            _refuse(where, f"the norm's parameters are [{self.size}] on {self.device}, the rows [{H}] on {device}")
        return self._ref


class Router:
    """How logits become experts and weights (moe_router_t): score "softmax" or "sigmoid", experts in
    `groups` equal runs of which the top_groups best (by the sum of their group_top best) are
    candidates, weights renormalised over the chosen and scaled."""

    def __init__(self, score="softmax", groups=1, top_groups=None, group_top=1, renormalize=True, scale=1.0):
        if score not in _SCORE:
            _refuse("Router", f"unknown score {score!r}")
        top_groups = groups if top_groups is None else top_groups
        self.desc = _RouterDesc(_SCORE[score], groups, top_groups, group_top, int(bool(renormalize)), scale)
        self._ref = C.addressof(self.desc)


def moe_block_enter(x, norm: Norm, dtype=None, out=None, stream=None):
    """y = norm(x) for x [T, H]; y in `dtype` (default x's; x may be fp32 and y narrower)."""
    where = "moe_block_enter"
    ldx = _matrix(x, where, "x")
    T, H = x.shape
    device = x.device
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype if dtype is None else dtype, device=device)
        ldy = H
    else:
        ldy = _matrix(out, where, "out", T, H, dtype, device)
    if out.dtype not in _DT:
        _refuse(where, f"type {out.dtype} is not bf16, fp16 or fp32")
    _check(_f().moe_block_enter(x.data_ptr(), ldx, _DT[x.dtype], norm._at(where, H, device), out.data_ptr(), ldy,
                                _DT[out.dtype], T, H, _stream(stream, device)), where)
    return out


def moe_block_leave(x, block, post: Norm = None, gate=None, gate_act="none", alpha=1.0, beta=1.0, next: Norm = None,
                    out=None, y=None, stream=None):
    """out = alpha x + beta g(gate) post(block), and with `next` also y = next(out) in block's type.

    x [T, H] is the residual stream, block [T, H] the block's output (x's type, or any where x is
    fp32).  gate: None, [H] (per channel), [T, 1] (per token) or [T, H]; g = gate_act "none",
    "sigmoid" or "tanh".  out may be x and y may be block (updated in place).  Returns out, or
    (out, y)."""
    where = "moe_block_leave"
    ldx = _matrix(x, where, "x")
    T, H = x.shape
    device = x.device
    ldb = _matrix(block, where, "block", T, H, None, device)
    if gate_act not in _GATE:
        _refuse(where, f"unknown gate_act {gate_act!r}")
    gp, gld, gstep, gdt = None, 0, 0, 1
    if gate is not None:
        if gate.dtype not in _DT or gate.device != device:
            _refuse(where, "gate is not bf16, fp16 or fp32 on x's device")
        shape = tuple(gate.shape)
        if shape == (H,):
            gstep = 1
            if H > 1 and gate.stride(0) != 1:
                _refuse(where, "gate needs unit column stride")
        elif shape == (T, 1) and H > 1:
            gld = gate.stride(0)
        elif shape == (T, H):
            gstep, gld = 1, gate.stride(0)
            if H > 1 and gate.stride(1) != 1:
                _refuse(where, "gate needs unit column stride")
        else:
            _refuse(where, f"gate has shape {shape}, not {(H,)}, {(T, 1)} or {(T, H)}")
        gp, gdt = gate.data_ptr(), _DT[gate.dtype]
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=device)
        ldo = H
    else:
        ldo = _matrix(out, where, "out", T, H, x.dtype, device)
    yp, ldy = None, 0
    if next is not None:
        if y is None:
            y = torch.empty((T, H), dtype=block.dtype, device=device)
            ldy = H
        else:
            ldy = _matrix(y, where, "y", T, H, block.dtype, device)
        yp = y.data_ptr()
    _check(_f().moe_block_leave(x.data_ptr(), ldx, _DT[x.dtype], block.data_ptr(), ldb, _DT[block.dtype],
                                post._at(where, H, device) if post is not None else None, gp, gld, gstep, gdt,
                                _GATE[gate_act], alpha, beta, next._at(where, H, device) if next is not None else None,
                                out.data_ptr(), ldo, yp, ldy, T, H, _stream(stream, device)), where)
    return out if next is None else (out, y)


def moe_route_scored(logits, router: Router, top_k: int, bias=None, topk_idx=None, topk_w=None, stream=None):
    """(topk_idx int32 [T, top_k], topk_w fp32 [T, top_k]) of logits [T, E] (bf16, fp16 or fp32) and the
    choice bias (fp32 [E]) or None."""
    where = "moe_route_scored"
    ld = _matrix(logits, where, "logits")
    T, E = logits.shape
    device = logits.device
    bp = _vector(bias, where, "bias", E, torch.float32, device)
    if not 1 <= top_k <= 8:
        _refuse(where, f"top_k = {top_k} is not in 1 .. 8")
    if topk_idx is None:
        topk_idx = torch.empty((T, top_k), dtype=torch.int32, device=device)
    if topk_w is None:
        topk_w = torch.empty((T, top_k), dtype=torch.float32, device=device)
    for t, dt, name in ((topk_idx, torch.int32, "topk_idx"), (topk_w, torch.float32, "topk_w")):
        if t.dtype != dt or t.shape != (T, top_k) or not t.is_contiguous() or t.device != device:
            _refuse(where, f"{name} is not a contiguous {dt} {(T, top_k)} on {device}")
    _check(_f().moe_route_scored(router._ref, logits.data_ptr(), ld, _DT[logits.dtype], bp, T, E, top_k,
                                 topk_idx.data_ptr(), topk_w.data_ptr(), _stream(stream, device)), where)
    return topk_idx, topk_w


def moe_layer_forward_scored(x, logits, router: Router, desc, packed, top_k: int, out, workspace, bias=None, stream=None):
    """moe_layer_forward with the experts chosen and weighted by `router`."""
    where = "moe_layer_forward_scored"
    T, E, H = x.shape[0], desc.E, desc.H
    device = x.device
    ld = _matrix(logits, where, "logits", T, E, None, device)
    for t, name in ((x, "x"), (out, "out")):
        _matrix(t, where, name, T, H, torch.bfloat16, device)
        if not t.is_contiguous():
            _refuse(where, f"{name} is not contiguous")
    bp = _vector(bias, where, "bias", E, torch.float32, device)
    _check(_f().moe_layer_forward_scored(x.data_ptr(), router._ref, logits.data_ptr(), ld, _DT[logits.dtype], bp, T,
                                         C.byref(desc), packed.data_ptr(), top_k, out.data_ptr(), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), _stream(stream, device)), where)


def moe_adapters_add(x, base, a, b, starts, slot, scale=None, rank=None, out=None, stream=None):
    """out[t] = base[t] + scale[s] b[s] (a[s] x[t]) with s = slot[q] of the request q that holds t.

    x bf16 [T, H], base bf16 [T, N]; a bf16 [n, r, H], b bf16 [n, N, r] contiguous; starts int32
    [R + 1] (request q has tokens starts[q] .. starts[q+1]-1), slot int32 [R] (outside 0 .. n-1: no
    adapter); scale fp32 [n] or None; rank int32 [n] (each adapter's own, at most r) or None.  out
    may be base (added in place)."""
    where = "moe_adapters_add"
    bf16 = torch.bfloat16
    ldx = _matrix(x, where, "x", None, None, bf16)
    T, H = x.shape
    device = x.device
    if a.dim() != 3 or b.dim() != 3:
        _refuse(where, "a and b are [n, r, H] and [n, N, r]")
    n, r, N = a.shape[0], a.shape[1], b.shape[1]
    for t, shape, name in ((a, (n, r, H), "a"), (b, (n, N, r), "b")):
        if t.dtype != bf16 or t.shape != shape or not t.is_contiguous() or t.device != device:
            _refuse(where, f"{name} is not a contiguous bf16 {shape} on {device}")
    ldb = _matrix(base, where, "base", T, N, bf16, device)
    i32 = torch.int32
    R = slot.shape[0] if slot.dim() == 1 else -1
    sp = _vector(starts, where, "starts", R + 1, i32, device)
    qp = _vector(slot, where, "slot", R, i32, device)
    fp = _vector(scale, where, "scale", n, torch.float32, device)
    rp = _vector(rank, where, "rank", n, i32, device)
    if out is None:
        out = torch.empty((T, N), dtype=bf16, device=device)
        ldo = N
    else:
        ldo = _matrix(out, where, "out", T, N, bf16, device)
    _check(_f().moe_adapters_add(x.data_ptr(), ldx, base.data_ptr(), ldb, a.data_ptr(), b.data_ptr(), fp, rp, sp, qp,
                                 out.data_ptr(), ldo, T, R, n, r, H, N, _stream(stream, device)), where)
    return out


class MoEBlock:
    """A mixture-of-experts block of a serving loop: norm, router, packed experts with the requests'
    adapters, and the way back into the residual stream.

        h   = pre(x);  logits = h @ w_router.T
        m   = experts(h, router(logits))  [+ adapters(h)]
        out = alpha x + beta g(gate) post(m);  y = next(out)   (the following block's h)
    """

    def __init__(self, layer: MoELayer, w_router, router: Router, top_k: int, pre: Norm, post: Norm = None,
                 router_bias=None, alpha=1.0, beta=1.0):
        self.layer, self.w_router, self.router, self.top_k = layer, w_router, router, top_k
        self.pre, self.post, self.router_bias, self.alpha, self.beta = pre, post, router_bias, alpha, beta

    def forward(self, x, h=None, adapters=None, gate=None, gate_act="none", next: Norm = None, stream=None):
        """x [T, H] (bf16, or an fp32 stream).  h: the block's input where the previous block's
        `next` has already made it.  adapters: None or a dict of moe_adapters_add's a, b, starts, slot,
        scale, rank.  Returns out, or (out, y) with `next`.  `stream`, if given, must be torch's
        current one: the router's product is torch's."""
        if h is None:
            h = moe_block_enter(x, self.pre, dtype=torch.bfloat16, stream=stream)
        logits = h @ self.w_router.t()
        m = torch.empty_like(h)
        ws = self.layer.ensure_workspace(int(h.shape[0]), self.top_k)
        moe_layer_forward_scored(h, logits, self.router, self.layer.desc, self.layer.packed, self.top_k, m, ws,
                                 bias=self.router_bias, stream=stream)
        if adapters is not None:
            moe_adapters_add(h, m, out=m, stream=stream, **adapters)
        return moe_block_leave(x, m, post=self.post, gate=gate, gate_act=gate_act, alpha=self.alpha, beta=self.beta,
                               next=next, out=None, stream=stream)
