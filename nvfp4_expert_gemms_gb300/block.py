"""Binding of the operators around the experts (include/moe_gb300.h, "operators around the
experts"): the norms on the way into and out of a block, scored routing, request adapters, and
MoEBlock, which runs them with a layer of packed experts.

Tensors are checked here (shapes, types, device, strides), since the C side sees only pointers; every
refusal is a MoEError with the status the C side would give.  Matrices are [rows, columns] with unit
column stride and any row stride.  Outputs that are not given are allocated by torch.  Work goes to
torch's current stream on the tensors' device, or to `stream` (a torch stream or a raw handle), for
which outputs are then allocated; as with torch's own operators the caller orders that stream after
the ones that made the inputs.  The checks and the calls are native (csrc/binding/block_binding.cpp).
"""
from __future__ import annotations

import ctypes as C
import importlib.util

import torch

from . import MoEError, MoELayer, PackedDesc, _build, _check, lib, moe_status_string

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


class _NormKey(C.Structure):
    """What the native side reads of a Norm: the C descriptor's kind, eps and offset, and the tensors themselves."""
    _fields_ = [("desc", _NormDesc), ("weight", C.c_void_p), ("bias", C.c_void_p)]


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
        L.moe_get_adapter_error.argtypes = [P, C.POINTER(C.c_int32)]
        L.moe_adapters_add.argtypes = [P, Q, P, Q, P, P, P, P, P, P, P, Q] + [I] * 6 + [P]
        _fns = L
    return _fns


_ext = None


def _native():
    """The binding extension, loaded (built first when its sources are newer) and given the C functions."""
    global _ext
    if _ext is None:
        L = _f()
        spec = importlib.util.spec_from_file_location("_block_ext", _build.build_binding())
        ext = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(ext)
        addr = lambda f: C.cast(f, C.c_void_p).value  # noqa: E731
        ext.init(_refuse, addr(L.moe_block_enter), addr(L.moe_block_leave), addr(L.moe_route_scored),
                 addr(L.moe_adapters_add))
        _ext = ext
    return _ext


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


class Norm:
    """A norm's kind and parameters: v / rms(v) ("rms") or (v - mean) / std ("layer"), times
    weight + offset, plus bias (both optional, [H], one type).  weight and bias may be replaced, or given other
    storage: a call uses what they are by then (a captured graph what they were)."""

    def __init__(self, kind="rms", weight=None, bias=None, eps=1e-6, offset=0.0):
        where = "Norm"
        if kind not in _KIND:
            _refuse(where, f"unknown kind {kind!r}")
        if not eps > 0.0:
            _refuse(where, "eps must be positive")
        self._desc = _NormKey(_NormDesc(_KIND[kind], 1, eps, offset, None, None), None, None)
        self._key = C.addressof(self._desc)
        self._made = kind, eps, offset
        self._set(weight, bias)
        if weight is not None and bias is not None and (weight.dtype, weight.shape, weight.device) != (bias.dtype, bias.shape, bias.device):
            _refuse(where, "weight and bias differ in type, size or device")

    def _set(self, weight, bias):
        given = [t for t in (weight, bias) if t is not None]
        for t in given:
            if not isinstance(t, torch.Tensor) or t.dim() != 1 or not t.is_cuda or not t.is_contiguous() or t.dtype not in _DT:
                _refuse("Norm", "weight and bias are contiguous [H] CUDA tensors of bf16, fp16 or fp32")
        # the native side reads the tensors at each call, so what they hold by then is what counts
        self._weight, self._bias = weight, bias
        self._desc.weight, self._desc.bias = (None if t is None else id(t) for t in (weight, bias))

    weight = property(lambda self: self._weight, lambda self, t: self._set(t, self._bias))
    bias = property(lambda self: self._bias, lambda self, t: self._set(self._weight, t))

    def __reduce__(self):  # a copy has a descriptor of its own
        kind, eps, offset = self._made
        return Norm, (kind, self._weight, self._bias, eps, offset)


class Router:
    """How logits become experts and weights (moe_router_t): score "softmax" or "sigmoid", experts in
    `groups` equal runs of which the top_groups best (by the sum of their group_top best) are
    candidates, weights renormalised over the chosen and scaled."""

    def __init__(self, score="softmax", groups=1, top_groups=None, group_top=1, renormalize=True, scale=1.0):
        if score not in _SCORE:
            _refuse("Router", f"unknown score {score!r}")
        top_groups = groups if top_groups is None else top_groups
        self._desc = _RouterDesc(_SCORE[score], groups, top_groups, group_top, int(bool(renormalize)), scale)
        self._ref = C.addressof(self._desc)
        self._made = score, groups, top_groups, group_top, renormalize, scale

    desc = property(lambda self: self._desc)  # never another one than _ref's

    def __reduce__(self):  # a copy has a descriptor of its own
        return Router, self._made


def moe_block_enter(x, norm: Norm, dtype=None, out=None, stream=None):
    """y = norm(x) for x [T, H]; y in `dtype` (default x's; x may be fp32 and y narrower).  out may be x."""
    return (_ext or _native()).enter(x, norm, dtype, out, None if stream is None else _handle(stream))


def moe_block_leave(x, block, post: Norm = None, gate=None, gate_act="none", alpha=1.0, beta=1.0, next: Norm = None,
                    out=None, y=None, stream=None):
    """out = alpha x + beta g(gate) post(block), and with `next` also y = next(out) in block's type.

    x [T, H] is the residual stream, block [T, H] the block's output (x's type, or any where x is
    fp32).  gate: None, [H] (per channel), [T, 1] (per token) or [T, H]; g = gate_act "none",
    "sigmoid" or "tanh".  out may be x and y may be block (updated in place).  Returns out, or
    (out, y)."""
    act = _GATE.get(gate_act)
    if act is None:
        _refuse("moe_block_leave", f"unknown gate_act {gate_act!r}")
    return (_ext or _native()).leave(x, block, post, gate, act, alpha, beta, next, out, y,
                                     None if stream is None else _handle(stream))


def moe_route_scored(logits, router: Router, top_k: int, bias=None, topk_idx=None, topk_w=None, stream=None):
    """(topk_idx int32 [T, top_k], topk_w fp32 [T, top_k]) of logits [T, E] (bf16, fp16 or fp32) and the
    choice bias (fp32 [E]) or None."""
    return (_ext or _native()).route(logits, router._ref, top_k, bias, topk_idx, topk_w,
                                     None if stream is None else _handle(stream))


def moe_adapters_add(x, base, a, b, starts, slot, scale=None, rank=None, out=None, stream=None):
    """out[t] = base[t] + scale[s] b[s] (a[s] x[t]) with s = slot[q] of the request q that holds t.

    x bf16 [T, H], base bf16 [T, N]; a bf16 [n, r, H], b bf16 [n, N, r] contiguous; starts int32
    [R + 1] (request q has tokens starts[q] .. starts[q+1]-1), slot int32 [R] (outside 0 .. n-1: no
    adapter); scale fp32 [n] or None; rank int32 [n] (each adapter's own, at most r) or None.  out
    may be base (added in place)."""
    return (_ext or _native()).adapters(x, base, a, b, starts, slot, scale, rank, out,
                                        None if stream is None else _handle(stream))


def moe_layer_forward_scored(x, logits, router: Router, desc, packed, top_k: int, out, workspace, bias=None, stream=None):
    """moe_layer_forward with the experts chosen and weighted by `router`: x and out bf16 [T, H] contiguous,
    logits [T, E] of any of the three types, bias fp32 [E] or None."""
    where = "moe_layer_forward_scored"
    T, E, H = int(x.shape[0]), desc.E, desc.H
    for t, name in ((x, "x"), (out, "out")):
        if t.shape != (T, H) or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != logits.device:
            _refuse(where, f"{name} is not a contiguous bf16 {(T, H)} on the logits' device")
    if logits.shape != (T, E) or logits.dtype not in _DT or not logits.is_cuda or (E > 1 and logits.stride(1) != 1):
        _refuse(where, f"logits are not a CUDA [{T}, {E}] of bf16, fp16 or fp32 with unit column stride")
    if bias is not None and (bias.shape != (E,) or bias.dtype != torch.float32 or not bias.is_contiguous() or bias.device != x.device):
        _refuse(where, f"bias is not a contiguous fp32 [{E}] on the logits' device")
    ld = max(logits.stride(0), E) if T <= 1 else logits.stride(0)
    with torch.cuda.device(x.device):
        _check(_f().moe_layer_forward_scored(x.data_ptr(), router._ref, logits.data_ptr(), ld, _DT[logits.dtype],
                                             None if bias is None else bias.data_ptr(), T, C.byref(desc), packed.data_ptr(), top_k,
                                             out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             torch.cuda.current_stream(x.device).cuda_stream if stream is None else _handle(stream)), where)


def moe_get_adapter_error(stream=None) -> int:
    """Synchronise the stream, then read and clear the current device's error word of moe_adapters_add (0: none)."""
    code = C.c_int32()
    _check(_f().moe_get_adapter_error(torch.cuda.current_stream().cuda_stream if stream is None else _handle(stream),
                                      C.byref(code)), "moe_get_adapter_error")
    return code.value


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

    def forward(self, x, h=None, adapters=None, gate=None, gate_act="none", next: Norm = None):
        """x [T, H] (bf16, or an fp32 stream).  h: the block's input where the previous block's
        `next` has already made it.  adapters: None or a dict of moe_adapters_add's a, b, starts, slot,
        scale, rank.  Returns out, or (out, y) with `next`.  Runs on torch's current stream (the
        layer's workspace serves one stream at a time)."""
        if h is None:
            h = moe_block_enter(x, self.pre, dtype=torch.bfloat16)
        logits = h @ self.w_router.t()
        m = torch.empty_like(h)
        ws = self.layer.ensure_workspace(int(h.shape[0]), self.top_k)
        moe_layer_forward_scored(h, logits, self.router, self.layer.desc, self.layer.packed, self.top_k, m, ws,
                                 bias=self.router_bias)
        if adapters is not None:
            moe_adapters_add(h, m, out=m, **adapters)
        return moe_block_leave(x, m, post=self.post, gate=gate, gate_act=gate_act, alpha=self.alpha, beta=self.beta,
                               next=next)
