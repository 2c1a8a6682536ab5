"""Argument checks of the operators around the experts that need no GPU: the C entry points refuse
bad arguments before any CUDA call, and the binding refuses tensors that are not on a CUDA device."""
import ctypes as C

import pytest
import torch

import nvfp4_expert_gemms_gb300 as M
from nvfp4_expert_gemms_gb300 import block

P = 4096  # an aligned address that nothing reads: every call below is refused first


def test_norm_entry_points_refuse():
    f = block._f()
    n = block._NormDesc(1, 1, 1e-6, 0.0, P, None)
    at = C.addressof(n)
    enter = lambda **k: f.moe_block_enter(*{**dict(x=P, ldx=64, xd=1, n=at, y=2 * P, ldy=64, yd=1, T=4, H=64, s=None), **k}.values())  # noqa: E731
    assert enter(T=-1) == enter(H=0) == enter(n=None) == enter(xd=0) == enter(yd=4) == 1
    assert enter(x=None) == enter(y=None) == enter(ldx=63) == enter(ldy=63) == enter(x=P + 1) == 1
    assert enter(yd=2) == enter(yd=3) == 2  # a bf16 stream gives bf16
    for field, bad in (("kind", 0), ("kind", 3), ("eps", 0.0), ("eps", float("nan")), ("dtype", 7), ("weight", P + 1), ("bias", P + 1)):
        keep = getattr(n, field)
        setattr(n, field, bad)
        assert enter() == 1, field
        setattr(n, field, keep)
    leave = lambda **k: f.moe_block_leave(*{**dict(x=P, ldx=64, xd=3, b=2 * P, ldb=64, bd=1, post=at, g=3 * P, gl=64, gs=1, gd=1, ga=0,  # noqa: E731
                                                  al=1.0, be=1.0, nx=at, o=4 * P, lo=64, y=5 * P, ly=64, T=4, H=64, s=None), **k}.values())
    assert leave(T=-1) == leave(H=0) == leave(b=None) == leave(o=None) == leave(y=None) == leave(ldb=8) == leave(lo=8) == leave(ly=8) == 1
    assert leave(gd=9) == leave(ga=3) == leave(gs=2) == leave(gl=-1) == leave(g=P + 1) == 1
    assert leave(xd=1, bd=2) == leave(xd=2, bd=3) == 2


def test_router_entry_points_refuse():
    f = block._f()
    good = dict(score=2, groups=8, top_groups=4, group_top=2, renormalize=1, scale=1.0)

    def route(k=8, E=64, T=4, **over):
        args = dict(l=P, ld=64, dt=3, b=None, i=P, w=P)
        args.update({n: v for n, v in over.items() if n in args})
        r = block._RouterDesc(*{**good, **{n: v for n, v in over.items() if n in good}}.values())
        return f.moe_route_scored(C.addressof(r), args["l"], args["ld"], args["dt"], args["b"], T, E, k, args["i"], args["w"], None)

    for bad in (dict(score=0), dict(score=3), dict(groups=0), dict(groups=7), dict(groups=64), dict(top_groups=0), dict(top_groups=9),
                dict(group_top=0), dict(group_top=3), dict(renormalize=2), dict(scale=float("nan")), dict(k=0), dict(k=9),
                dict(E=0), dict(E=264), dict(T=-1), dict(l=None), dict(i=None), dict(w=None), dict(ld=63), dict(dt=0), dict(l=P + 2),
                dict(b=P + 1), dict(top_groups=1, groups=32, k=3)):
        assert route(**bad) == 1, bad
    assert f.moe_route_scored(None, P, 64, 3, None, 4, 64, 8, P, P, None) == 1
    # the layer with a scored router: the router's refusals, then the layer's own
    d = M.moe_packed_size("fp8", 64, 256, 128)
    r = block._RouterDesc(*good.values())
    layer = lambda **k: f.moe_layer_forward_scored(*{**dict(x=P, r=C.addressof(r), l=P, ld=64, dt=3, b=None, T=4, d=C.byref(d), p=P, k=8,  # noqa: E731
                                                            o=2 * P, w=P, n=16, s=None), **k}.values())
    assert layer() == 3  # a workspace of 16 bytes
    assert layer(r=None) == layer(ld=63) == layer(dt=0) == layer(k=9) == layer(l=P + 2) == layer(b=P + 1) == layer(o=P) == 1


def test_adapter_entry_point_refuses():
    f = block._f()
    call = lambda **k: f.moe_adapters_add(*{**dict(x=P, lx=64, b=P, lb=64, A=P, B=P, sc=None, rk=None, st=P, sl=P, o=P, lo=64, T=4, R=1,  # noqa: E731
                                                   n=1, r=8, H=64, N=64, s=None), **k}.values())
    for bad in (dict(T=-1), dict(R=-1), dict(n=-1), dict(H=60), dict(H=0), dict(N=4), dict(N=0), dict(r=0), dict(r=4), dict(r=136), dict(r=12),
                dict(x=None), dict(b=None), dict(o=None), dict(A=None), dict(B=None), dict(st=None), dict(sl=None), dict(x=P + 8),
                dict(A=P + 2), dict(lx=56), dict(lb=60), dict(lo=68), dict(sc=P + 1), dict(rk=P + 2), dict(st=P + 1), dict(sl=P + 1)):
        assert call(**bad) == 1, bad


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 8), dtype=torch.bfloat16)
    for call in (lambda: M.moe_block_enter(x, M.Norm("rms")), lambda: M.moe_block_leave(x, x),
                 lambda: M.moe_route_scored(x, M.Router(), 2), lambda: M.Norm("rms", torch.ones(8))):
        with pytest.raises(M.MoEError) as e:
            call()
        assert e.value.status == 1 and "invalid argument" in str(e.value)


def test_adapter_entry_point_refuses_tokens_of_no_request():
    f = block._f()
    call = lambda T, R: f.moe_adapters_add(P, 64, P, 64, P, P, None, None, P, P, P, 64, T, R, 1, 8, 64, 64, None)  # noqa: E731
    assert call(4, 0) == call(1, 0) == 1  # nothing would write them
