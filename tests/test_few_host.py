"""Argument checks of the layer for a few tokens and of the FP8 block products that need no GPU: the C entry points
refuse before any CUDA call, and the binding refuses tensors that are not on a CUDA device."""
import ctypes as C
import gc
import weakref

import pytest
import torch

import nvfp4_expert_gemms_gb300 as M
from nvfp4_expert_gemms_gb300 import block

P = 4096  # an aligned address that nothing reads: every call below is refused first


def test_few_refuses():
    f = block._f()
    d = M.moe_packed_size("fp8", 64, 256, 128)
    r = block._RouterDesc(2, 8, 4, 2, 1, 1.0)
    n = C.c_size_t()
    size = lambda T, k, desc=d: f.moe_layer_few_workspace_size(C.byref(desc), T, k, C.byref(n))  # noqa: E731
    assert size(32, 8) == 0 and n.value > 0
    assert size(33, 8) == size(-1, 8) == size(4, 0) == size(4, 9) == 1
    assert f.moe_layer_few_workspace_size(None, 4, 2, C.byref(n)) == f.moe_layer_few_workspace_size(C.byref(d), 4, 2, None) == 1
    sizes = [(size(T, 8), n.value)[1] for T in range(33)]
    assert sizes == sorted(sizes)  # a workspace of more tokens serves fewer

    def few(**over):
        a = dict(x=P, lx=256, w=P, lw=256, wd=1, r=C.addressof(r), b=None, T=4, d=C.byref(d), p=P, k=8, o=2 * P, lo=256, ti=None, tw=None,
                 ws=P, n=1 << 40, s=None)
        return f.moe_layer_few(*{**a, **over}.values())

    for bad in (dict(T=-1), dict(T=33), dict(x=None), dict(w=None), dict(p=None), dict(o=None), dict(ws=None), dict(x=P + 2), dict(w=P + 2),
                dict(o=P + 2), dict(p=P + 16), dict(ws=P + 16), dict(b=P + 1), dict(ti=P + 2), dict(tw=P + 1), dict(lx=248), dict(lx=260),
                dict(lw=255), dict(lw=257), dict(lo=128), dict(lo=257), dict(wd=0), dict(wd=4), dict(k=0), dict(k=9), dict(r=None), dict(d=None)):
        assert few(**bad) == 1, bad
    assert few(n=size(4, 8) or n.value - 1) == 3
    for field, bad in (("score", 3), ("groups", 7), ("top_groups", 9), ("group_top", 0), ("renormalize", 2), ("scale", float("nan"))):
        keep = getattr(r, field)
        setattr(r, field, bad)
        assert few() == 1, field
        setattr(r, field, keep)
    for field, bad in (("fmt", 9), ("E", 0), ("H", 200), ("I", 64)):
        keep = getattr(d, field)
        setattr(d, field, bad)
        assert few() == 1, field
        setattr(d, field, keep)


def test_quantize_refuses():
    f = block._f()
    call = lambda **k: f.moe_fp8_quantize(*{**dict(x=P, lx=64, dt=1, q=P, lq=64, s=P, T=4, K=64, st=None), **k}.values())  # noqa: E731
    for bad in (dict(T=-1), dict(K=0), dict(K=2 ** 31 - 512, lx=1 << 31, lq=1 << 31), dict(dt=0), dict(dt=4), dict(lx=63), dict(lq=63), dict(x=None), dict(q=None), dict(s=None), dict(x=P + 1),
                dict(s=P + 2)):
        assert call(**bad) == 1, bad


def test_linear_refuses():
    f = block._f()
    n = C.c_size_t()
    size = lambda *a: f.moe_fp8_linear_workspace_size(*a, C.byref(n))  # noqa: E731
    assert size(1, 4, 64, 32, 0) == size(4, 4, 64, 32, 1) == 0
    for bad in ((0, 4, 64, 32, 0), (5, 4, 64, 32, 0), (1, -1, 64, 32, 0), (1, 4, 0, 32, 0), (1, 4, 24, 32, 0), (1, 4, 64, 0, 0), (1, 4, 64, 33, 1),
                (1, 2 ** 31 - 512, 64, 32, 0), (1, 4, 2 ** 31 - 16, 32, 0), (1, 4, 64, 2 ** 31 - 512, 0),
                (1, 4, 64, 32, 2)):
        assert size(*bad) == 1, bad
    assert f.moe_fp8_linear_workspace_size(1, 4, 64, 32, 0, None) == 1

    def call(**over):
        a = dict(x=P, lx=64, xd=1, xs=None, w=P, wsc=P, act=0, b=None, lb=0, o=2 * P, lo=32, od=1, T=4, K=64, N=32, ws=P, n=1 << 40, s=None)
        return f.moe_fp8_linear(*{**a, **over}.values())

    for bad in (dict(T=-1), dict(K=0), dict(K=24), dict(N=0), dict(act=2), dict(act=1, N=31), dict(xd=0), dict(xd=5), dict(od=0), dict(od=4),
                dict(lx=63), dict(lo=31), dict(b=P, lb=31), dict(x=None), dict(w=None), dict(wsc=None), dict(o=None), dict(x=P + 1), dict(w=P + 8),
                dict(wsc=P + 2), dict(o=P + 1), dict(b=P + 1, lb=32), dict(ws=None), dict(ws=P + 16), dict(xd=4), dict(xd=4, xs=P, x=P + 8),
                dict(xd=4, xs=P, lx=72), dict(xd=4, xs=P + 1)):
        assert call(**bad) == 1, bad
    assert call(n=16) == 3
    assert f.moe_get_fp8_linear_error(None, None) == 1


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    d = M.moe_packed_size("fp8", 8, 256, 128)
    ws = torch.zeros(16, dtype=torch.uint8)
    w8 = torch.zeros((64, 256), dtype=torch.uint8)
    for call in (lambda: M.moe_layer_few(x, x, M.Router(), d, ws, 2, ws), lambda: M.moe_fp8_quantize(x),
                 lambda: M.Fp8Weight(w8, torch.ones((1, 2)))):
        with pytest.raises(M.MoEError) as e:
            call()
        assert e.value.status == 1 and "invalid argument" in str(e.value)


@pytest.fixture
def host_layer(monkeypatch):
    """A layer whose buffers stand on the host and hold nothing: for what MoELayer and MoEBlock keep and choose."""
    monkeypatch.setattr(M, "moe_pack_experts", lambda *a: None)
    return M.MoELayer("fp8", torch.zeros((4, 256, 256), dtype=torch.bfloat16), torch.zeros((4, 256, 128), dtype=torch.bfloat16))


def block_of(layer, **kw):
    return M.MoEBlock(layer, torch.zeros((4, 256), dtype=torch.bfloat16), M.Router(), 2, M.Norm("rms"), **kw)


def test_few_workspaces_outlive_their_replacement(host_layer):
    a = block_of(host_layer, few_tokens=2)
    first = a.few_workspace.data_ptr()
    held = weakref.ref(host_layer.ensure_few_workspace(2, 2))
    assert held().data_ptr() == first  # no other for no more tokens
    b = block_of(host_layer, few_tokens=32)
    assert b.few_workspace.numel() > a.few_workspace.numel() and a.few_workspace.data_ptr() == first
    del a
    gc.collect()
    assert held() is not None  # a graph that block a captured may still write there
    assert block_of(host_layer).few_workspace is None


def test_captured_workspaces_outlive_their_replacement(host_layer, monkeypatch):
    eager = weakref.ref(host_layer.ensure_workspace(4, 2))
    monkeypatch.setattr(M, "_capturing", lambda: True, raising=False)
    captured = weakref.ref(host_layer.ensure_workspace(64, 2))
    assert host_layer.ensure_workspace(64, 2) is captured() and len(host_layer._captured_workspaces) == 1
    monkeypatch.setattr(M, "_capturing", lambda: False, raising=False)
    host_layer.ensure_workspace(512, 2)
    gc.collect()
    assert eager() is None and captured() is not None and captured() is not host_layer.workspace


def test_few_workspace_reports_no_error_before_its_first_call(host_layer):
    torch.use_deterministic_algorithms(True)  # fills what torch.empty gives
    try:
        ws = host_layer.ensure_few_workspace(4, 2)
    finally:
        torch.use_deterministic_algorithms(False)
    assert ws[:256].view(torch.int32).eq(0).all()


@pytest.mark.parametrize("few_tokens", [0, 8])
def test_block_sends_no_tokens_the_way_of_many(host_layer, monkeypatch, few_tokens):
    # w_router may be any view there, of which the operator for few tokens takes whole aligned rows alone
    blk = block_of(host_layer, few_tokens=few_tokens)
    blk.w_router = torch.zeros((256, 4), dtype=torch.bfloat16).t()
    went = []
    monkeypatch.setattr(block, "moe_layer_few", lambda *a, **k: went.append("few"))
    monkeypatch.setattr(block, "moe_layer_forward_scored", lambda *a, **k: went.append("many"))
    monkeypatch.setattr(block, "moe_block_leave", lambda x, m, **k: m)
    assert blk.forward(torch.zeros((0, 256)), h=torch.zeros((0, 256), dtype=torch.bfloat16)).shape == (0, 256)
    assert went == ["many"]


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_block_multiplies_routers_of_any_type(host_layer, monkeypatch, w_dtype):
    g = torch.Generator().manual_seed(3)
    h = torch.randn((3, 256), generator=g).bfloat16()
    blk = block_of(host_layer)
    blk.w_router = torch.randn((4, 256), generator=g).to(w_dtype)
    seen = []
    monkeypatch.setattr(block, "moe_layer_forward_scored", lambda x, logits, *a, **k: seen.append(logits))
    monkeypatch.setattr(block, "moe_block_leave", lambda x, m, **k: m)
    blk.forward(torch.zeros((3, 256)), h=h)
    want = h @ blk.w_router.t() if w_dtype == torch.bfloat16 else h.float() @ blk.w_router.float().t()
    assert seen[0].dtype == want.dtype and torch.equal(seen[0], want)


def host_weight(N, K, device="cpu"):
    w = object.__new__(M.Fp8Weight)  # (the class takes CUDA tensors alone)
    w.codes, w.scale_inv = torch.zeros((N, K), dtype=torch.uint8, device=device), torch.ones(((N + 127) // 128, (K + 127) // 128), device=device)
    return w


def test_block_refuses_a_shared_pair_when_it_is_made(host_layer):  # H = 256
    for pair in ((host_weight(192, 256), host_weight(256, 96)), [host_weight(32, 256), host_weight(256, 16)]):
        assert block_of(host_layer, shared=pair).shared is pair
    up, down = host_weight(192, 256), host_weight(256, 96)
    for bad in (up, (up,), (up, down, down), (up, None), (up.codes, down.codes), (down, up), (up, host_weight(256, 192)), (up, host_weight(128, 96)),
                (host_weight(192, 128), down), (host_weight(190, 256), down), (up, host_weight(256, 96, "meta"))):
        with pytest.raises(M.MoEError) as e:
            block_of(host_layer, shared=bad)
        assert e.value.status == 1
