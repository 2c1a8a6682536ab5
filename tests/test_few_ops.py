"""The layer for a few tokens and the FP8 block products against plain 64-bit implementations (GPU).

Tolerances, elementwise, with u = 2^-24 and h = finfo(out).eps / 2 (bf16 2^-8, fp16 2^-11, fp32 2^-24):
  products   an inner product of n terms in fp32, in whatever order and with tensor cores that may truncate, is off by
             at most (n + 16) 2^-23 * sum |a||b|; 16 covers the scales' own roundings
  few        gate and up are off by eg, eu so bounded; |silu'| < 1.1, so silu(g) u is off by at most
             1.1 eg (|u| + eu) + |silu(g)| eu + 16 u |h|; as an operand h may be held in two terms of 8 or 11 bits:
             2^-16 |h| (two bf16 terms) + 2^-22 of the row's largest (what two fp16 terms with one exponent per row lose);
             the down products and their weighted sum as above, and out is rounded once
  linear     the products' error, the same silu, a few u of the result and base, and the rounding
The quantizer, the choice of experts and their weights are compared bit for bit.
"""
import os
import sys

import pytest
import torch

import nvfp4_expert_gemms_gb300 as M

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------------------------------ the layer for a few tokens
def weights(desc, packed, which, e):
    """Expert e's dequantized gate/up (0) or down (1) matrix in fp64, from the canonical tensors."""
    a, b, gs = ((M.MOE_T_GU_A, M.MOE_T_GU_B, M.MOE_T_GU_GS), (M.MOE_T_D_A, M.MOE_T_D_B, M.MOE_T_D_GS))[which]
    c = M.packed_view(desc, packed, a)[e]
    if desc.fmt == M.FMT_BF16:
        return c.double()
    s = M.packed_view(desc, packed, b)[e]
    if desc.fmt in (M.FMT_FP8, M.FMT_FP8_W8A8):
        return c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    if desc.fmt == M.FMT_INT4:
        q = torch.stack([(c >> (4 * j)) & 15 for j in range(8)], 1).flatten(0, 1)  # [K, N]
        return ((q - 8).double() * s.double().repeat_interleave(128, 0)).t()
    q = torch.stack((c & 15, c >> 4), -1).flatten(1).long()
    v = E2M1.cuda()[q] * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return v / M.packed_view(desc, packed, gs)[e].double()


def reference(x, idx, wt, desc, packed):
    """out and its bound, both fp64, for the given choice."""
    T, H, I = x.shape[0], desc.H, desc.I
    out, err = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
    xd = x.double()
    for e in sorted(set(idx.flatten().tolist())):
        rows, slots = (idx == e).nonzero(as_tuple=True)
        xe = xd[rows]
        w = weights(desc, packed, 0, e)
        v, b = xe @ w.t(), (xe.abs() @ w.abs().t()) * (H + 16) * 2.0 ** -23
        g, u, eg, eu = v[:, :I], v[:, I:], b[:, :I], b[:, I:]
        sg = g * torch.sigmoid(g)
        h = sg * u
        eh = 1.1 * eg * (u.abs() + eu) + sg.abs() * eu + 16 * U * h.abs()
        eh = eh + 2.0 ** -16 * h.abs() + 2.0 ** -22 * h.abs().amax(1, keepdim=True)
        w = weights(desc, packed, 1, e)
        p = wt[rows, slots].double()[:, None]
        out.index_add_(0, rows, p * (h @ w.t()))
        err.index_add_(0, rows, p.abs() * (eh @ w.abs().t() + (I + 16) * 2.0 ** -23 * (h.abs() @ w.abs().t())))
    return out, err + half(torch.bfloat16) * (out.abs() + err)


def logits_of(x, w_router):
    return (x.double() @ w_router.double().t()).float()


class Layer:
    def __init__(self, fmt, T, E, k, H, I, seed=0, router=None, bias=False, w_dtype=torch.bfloat16):
        g = gen(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.k, self.T = k, T
        self.desc = M.moe_packed_size(fmt, E, H, I)
        self.packed = torch.empty(self.desc.bytes, dtype=torch.uint8, device="cuda")
        M.moe_pack_experts(self.desc, (rnd(E, 2 * I, H) / H ** 0.5).bfloat16(), (rnd(E, H, I) / I ** 0.5).bfloat16(), self.packed)
        self.x = (rnd(T, H) * torch.exp(rnd(H))).bfloat16()
        self.w_router = (rnd(E, H) / H ** 0.5).to(w_dtype)
        self.bias = 0.05 * rnd(E) if bias else None
        self.router = router or M.Router()
        self.ws = torch.full((M.moe_layer_few_workspace_size(self.desc, T, k),), 255, dtype=torch.uint8, device="cuda")
        self.idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        self.wt = torch.full((T, k), -1.0, device="cuda")

    def run(self, x=None, **kw):
        kw = {**dict(bias=self.bias, topk_idx=self.idx, topk_w=self.wt), **kw}
        return M.moe_layer_few(self.x if x is None else x, self.w_router, self.router, self.desc, self.packed, self.k, self.ws, **kw)

    def choice(self, x=None):
        return M.moe_route_scored(logits_of(self.x if x is None else x, self.w_router), self.router, self.k, bias=self.bias)

    def check(self, out, x=None, rows=slice(None)):
        idx, wt = self.choice(x)
        assert torch.equal(idx, self.idx) and torch.equal(wt, self.wt)
        ref, tol = reference(self.x if x is None else x, idx, wt, self.desc, self.packed)
        ref, tol, out = ref[rows], tol[rows], out[rows]
        d = (out.double() - ref).abs()
        assert torch.isfinite(out).all() and (d <= tol).all(), f"{(d / tol).max().item():.3f} of the bound"
        # the bound above allows every rounding to go the same way; one rounding to bf16 is 2^-8 of each element
        assert d.norm() <= (2.0 ** -8 + 1e-4) * ref.norm()
        assert M.moe_get_device_error(self.ws) == 0


MANY = [(32, 256, 8, 384, 128), (31, 100, 7, 640, 896), (8, 6, 6, 9216, 256), (2, 4, 2, 256, 5120)]
SIZES = [(1, 8, 2, 256, 128), (3, 16, 4, 384, 256), (32, 8, 8, 128, 128), (5, 60, 4, 1408, 640), (2, 256, 8, 512, 384), (1, 1, 1, 128, 128),
         (9, 12, 3, 2304, 1152), (4, 5, 5, 4352, 128), (17, 9, 1, 128, 2176)]


@pytest.mark.parametrize("fmt", sorted(M.FORMATS))
@pytest.mark.parametrize("T,E,k,H,I", SIZES)
def test_few(fmt, T, E, k, H, I):
    layer = Layer(fmt, T, E, k, H, I, seed=T + H)
    layer.check(layer.run())


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 128, 128), (1, 3, 3, 640, 128), (3, 7, 5, 1152, 128), (5, 256, 1, 4224, 128)])
def test_few_rows_and_marks_that_end_inside_a_warp(T, E, k, H, I):
    # H / 8 pieces of a row, and a sixteenth of h's and y's bytes, that are no multiples of 32: lanes of one warp take
    # different numbers of turns before the router's blocks meet
    layer = Layer("fp8", T, E, k, H, I, seed=H)
    want = layer.run()
    layer.check(want)
    assert all(torch.equal(layer.run(), want) for _ in range(20))


@pytest.mark.parametrize("fmt", sorted(M.FORMATS))
@pytest.mark.parametrize("T,E,k,H,I", MANY)
def test_few_of_many_slots_and_long_rows(fmt, T, E, k, H, I):
    # every slot there can be; matrices of more stages than the warps keep activations of
    layer = Layer(fmt, T, E, k, H, I, seed=T + I, router=M.Router("sigmoid"), bias=True)
    want = layer.run()
    layer.check(want)
    assert torch.equal(layer.run(), want)
    x = layer.x.clone()
    layer.run(x, out=x)  # in place
    assert torch.equal(x, want)


@pytest.mark.parametrize("fmt,T", [("fp8", 1), ("fp8", 16), ("int4", 4), ("nvfp4_w4a16", 1), ("nvfp4_w4a16", 32), ("bf16", 2)])
def test_few_at_full_size(fmt, T):
    layer = Layer(fmt, T, 128, 8, 2048, 768, seed=T)
    layer.check(layer.run())


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("score,bias,groups,top_groups,renorm", [("softmax", False, 1, 1, False), ("sigmoid", True, 8, 3, True),
                                                                   ("softmax", True, 4, 2, True), ("sigmoid", False, 16, 9, False)])
def test_few_routers(w_dtype, score, bias, groups, top_groups, renorm):
    router = M.Router(score, groups=groups, top_groups=top_groups, group_top=2, renormalize=renorm, scale=2.5)
    layer = Layer("fp8", 6, 64, 6, 512, 256, seed=3, router=router, bias=bias, w_dtype=w_dtype)
    layer.check(layer.run())


def test_few_chooses_by_the_exact_sum():
    # rows of the router whose logits are large sums that cancel to a few units: any order of fp32 sums would mix them up
    layer = Layer("fp8", 4, 32, 4, 1024, 128, seed=5, w_dtype=torch.float32)
    g = gen(6)
    x = torch.randn((4, 1024), generator=g, device="cuda").bfloat16()
    x[:, 512:] = -x[:, :512]
    base = torch.randn(512, generator=g, device="cuda") * 4096.0
    layer.w_router[:, :512] = base
    layer.w_router[:, 512:] = base + torch.randn((32, 512), generator=g, device="cuda") * 1e-2
    layer.x = x
    layer.check(layer.run())
    layer.w_router.copy_(layer.w_router[:1].expand(32, -1).clone())  # all equal: the lowest indices
    layer.check(layer.run())
    assert torch.equal(layer.idx, torch.arange(4, device="cuda", dtype=torch.int32).expand(4, 4))


@pytest.mark.parametrize("fmt", ["fp8", "int4", "nvfp4_w4a16", "bf16"])
def test_few_all_tokens_on_the_same_experts(fmt):
    layer = Layer(fmt, 32, 16, 2, 640, 384, seed=7, bias=True, router=M.Router("sigmoid"))
    layer.bias[3] += 50.0
    layer.bias[9] += 40.0
    layer.check(layer.run())
    assert torch.equal(layer.idx, torch.tensor([[3, 9]] * 32, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("fmt", ["fp8", "int4", "nvfp4_w4a16", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 3e4, 1e12])
def test_few_of_any_magnitude(fmt, scale):
    # in each row a wide range of sizes, a row of zeros, and one value that is far above the others
    layer = Layer(fmt, 4, 16, 4, 512, 256, seed=11)
    x = layer.x.float() * scale
    x[1] = 0.0
    x[2, 7] *= 2.0 ** 30
    x = x.bfloat16()
    if scale <= 1e-12:  # gate * up is below fp32's range or near it: the 64-bit value's own rounding to out is all there is
        out = layer.run(x)
        idx, wt = layer.choice(x)
        assert torch.equal(idx, layer.idx) and torch.equal(wt, layer.wt)
        ref, tol = reference(x, idx, wt, layer.desc, layer.packed)
        # products below 2^-126 may be lost: 2^-126 for each of the terms of a sum, times the weights of the next (below 8)
        assert ((out.double() - ref).abs() <= tol + 2.0 ** -126 * (512 + 256) * 64).all()
    else:
        # 1e12 2^30 = 1.1e21: silu(gate) * up of row 2 is of the order of its square, 1e42, which fp32 (3.4e38) does not hold
        layer.check(layer.run(x), x, [0, 1, 3] if scale == 1e12 else slice(None))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 512, 256), (16, 16, 4, 2304, 1152)])
@pytest.mark.parametrize("above", [2.0 ** 10, 2.0 ** 14, 2.0 ** 18])
def test_few_int4_weights_of_zero_take_large_activations_out(T, E, k, H, I, above):
    # channels far above the others that every gate and up gives a weight of zero (code 8): what they leave is an error by
    # the weights' sizes, sum |w| |x|, to which they add nothing
    layer = Layer("int4", T, E, k, H, I, seed=T)
    gu = M.packed_view(layer.desc, layer.packed, M.MOE_T_GU_A)  # words [E, H / 8, 2 I] of eight channels, lowest nibble first
    layer.x = torch.randn((T, H), generator=gen(H), device="cuda").bfloat16()
    for c in (5, 130, H - 2):
        gu[:, c // 8] = gu[:, c // 8] & ~(15 << 4 * (c % 8)) | 8 << 4 * (c % 8)
        layer.x[:, c] *= above
    layer.check(layer.run())
    gu.fill_(-0x77777778)  # 0x88888888: weights of zero alone
    assert (layer.run() == 0).all()


def test_few_keeps_nan_and_infinity_in_their_rows():
    for fmt in ("fp8", "int4", "nvfp4_w4a16", "bf16"):
        layer = Layer(fmt, 5, 8, 4, 256, 256, seed=13)
        clean = layer.run()
        x = layer.x.clone()
        x[1, 17], x[3, 200] = float("nan"), float("inf")
        out = layer.run(x)
        for t in (0, 2, 4):
            assert torch.equal(out[t], clean[t])
        assert not torch.isfinite(out[1]).any() and not torch.isfinite(out[3]).any()
        assert M.moe_get_device_error(layer.ws) == 0


def large_h(fmt, gate, up, down, x):
    """A layer of one expert, 128 x 128, of which the seventh feature alone has ups, and its output."""
    layer = Layer(fmt, x.shape[0], 1, 1, 128, 128)
    wgu, g = torch.zeros((1, 256, 128), device="cuda"), gen(67)
    wgu[0, :128] = torch.randn((128, 128), generator=g, device="cuda")
    wgu[0, 7], wgu[0, 128 + 7] = gate, up
    M.moe_pack_experts(layer.desc, wgu.bfloat16(), down[None].bfloat16(), layer.packed)
    layer.x = x
    return layer, layer.run()


@pytest.mark.parametrize("fmt", ["fp8", "int4", "nvfp4_w4a16", "bf16"])
def test_few_h_past_fp32_gives_infinities(fmt):
    # silu(gate) up of row 0 is of the order of 1e50: an infinity times the down weight, with its sign, NaN where that is zero
    x = torch.randn((2, 128), generator=gen(71), device="cuda").bfloat16()
    ones, down = torch.ones(128, device="cuda"), torch.randn((128, 128), generator=gen(73), device="cuda")
    down[5, 7] = 0.0
    _, clean = large_h(fmt, ones, ones, down, x)
    x[0] = 1e25
    layer, out = large_h(fmt, ones, ones, down, x)
    w = weights(layer.desc, layer.packed, 1, 0)[:, 7]
    assert w[5] == 0.0 and torch.equal(out[0].isnan(), w == 0.0)
    assert torch.equal(out[0].float()[w != 0.0], torch.full_like(w, float("inf"), dtype=torch.float32)[w != 0.0] * w.float().sign()[w != 0.0])
    assert torch.equal(out[1], clean[1])


def test_few_h_that_bf16_would_round_to_infinity():
    # gate = x_0, up = x_1, and (1 + 2^-7) (1 - 2^-7) 2^128 is a number of fp32 above the largest of bf16
    e0, e1 = torch.eye(128, device="cuda")[:2]
    down = torch.full((128, 128), 2.0 ** -20, device="cuda")
    x = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 1] = (1 + 2.0 ** -7) * 2.0 ** 63, (1 - 2.0 ** -7) * 2.0 ** 65
    _, out = large_h("bf16", e0, e1, down, x)
    assert (out == 2.0 ** 108).all()  # (1 - 2^-14) 2^108, rounded


def test_few_pitches_aliases_streams_and_repeats():
    layer = Layer("fp8", 7, 16, 4, 512, 256, seed=17)
    want = layer.run()
    layer.check(want)
    wide = torch.full((7, 512 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = wide[:, :512]
    x.copy_(layer.x)
    wr = torch.full((16, 512 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :512]
    wr.copy_(layer.w_router)
    layer.w_router = wr
    out = torch.full((7, 512 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    assert layer.run(x, out=out[:, :512]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:, :512], want) and (out[:, 512:] == 3.0).all()
    for _ in range(5):
        assert torch.equal(layer.run(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    assert torch.equal(layer.run(topk_idx=None, topk_w=None), want)
    layer.run(x, out=x)  # in place
    assert torch.equal(x, want) and wide[:, 512:].isnan().all()
    big = torch.full((M.moe_layer_few_workspace_size(layer.desc, 32, 8),), 77, dtype=torch.uint8, device="cuda")
    layer.ws = big  # any workspace that is large enough, whatever it holds
    assert torch.equal(layer.run(), want)
    layer.x = layer.x[:3].contiguous()  # fewer tokens on the same workspace
    layer.idx, layer.wt = layer.idx[:3].contiguous(), layer.wt[:3].contiguous()
    assert torch.equal(layer.run(), want[:3])
    one = layer.x[1:2]
    assert torch.equal(layer.run(one, topk_idx=None, topk_w=None), want[1:2])  # a row does not depend on the others
    empty = layer.run(layer.x[:0], topk_idx=None, topk_w=None)
    assert empty.shape == (0, 512)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4_w4a16"])
def test_few_two_calls_at_once_and_in_graphs(fmt):
    a, b = Layer(fmt, 8, 32, 4, 1024, 512, seed=19), Layer(fmt, 3, 32, 4, 1024, 512, seed=23)
    wa, wb = a.run(), b.run()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    outs = [(a.run(stream=sa), b.run(stream=sb)) for _ in range(20)]  # each on its own workspace
    torch.cuda.synchronize()
    assert all(torch.equal(p, wa) and torch.equal(q, wb) for p, q in outs)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    x2 = a.x.clone()
    with torch.cuda.graph(ga):
        for _ in range(3):
            y = a.run(x2)
    with torch.cuda.graph(gb):  # another graph on the same workspace, replayed after the first
        z = a.run(a.x)
    ga.replay()
    gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, wa) and torch.equal(z, wa)
    x2.copy_(torch.roll(a.x, 1, 0))
    ga.replay()
    assert torch.equal(y, torch.roll(wa, 1, 0))
    for w in (a.ws, b.ws):
        assert M.moe_get_device_error(w) == 0


def test_few_reads_canonical_tensors_only():
    for fmt in ("nvfp4_w4a4", "nvfp4_w4a16"):
        layer = Layer(fmt, 4, 8, 2, 256, 256, seed=29)
        want = layer.run()
        for which in (M.MOE_T_GU_IMG, M.MOE_T_D_IMG):
            M.packed_view(layer.desc, layer.packed, which).fill_(255)
        assert torch.equal(layer.run(), want)


def test_few_refusals():
    layer = Layer("fp8", 4, 16, 4, 256, 128, seed=31)
    ok = dict(x=layer.x, w_router=layer.w_router, router=layer.router, desc=layer.desc, packed=layer.packed, top_k=4, workspace=layer.ws)

    def refused(status=1, **over):
        with pytest.raises(M.MoEError) as e:
            M.moe_layer_few(**{**ok, **over})
        assert e.value.status == status

    refused(x=layer.x.float())
    refused(x=layer.x[:, :128])
    refused(x=layer.x.t())
    refused(x=torch.zeros((33, 256), dtype=torch.bfloat16, device="cuda"))
    refused(x=torch.zeros((4, 260), dtype=torch.bfloat16, device="cuda")[:, :256])  # a pitch of 260
    refused(x=torch.zeros((4, 257), dtype=torch.bfloat16, device="cuda")[:, 1:])
    refused(x=layer.x.cpu())
    refused(w_router=layer.w_router[:8])
    refused(w_router=layer.w_router.double())
    refused(packed=layer.packed[:-1])
    refused(top_k=0)
    refused(top_k=9)
    refused(3, workspace=layer.ws[:256])
    refused(bias=torch.zeros(15, device="cuda"))
    refused(bias=torch.zeros(16, dtype=torch.bfloat16, device="cuda"))
    refused(out=torch.zeros((4, 256), device="cuda"))
    refused(out=torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda"))
    refused(topk_idx=torch.zeros((4, 4), dtype=torch.int64, device="cuda"))
    refused(topk_w=torch.zeros((4, 3), device="cuda"))
    refused(router=M.Router(groups=5))


# ------------------------------------------------------------------------------------------ the quantizer
def plain_quantize(x):
    """The definition on the host, one IEEE fp32 operation at a time."""
    v = x.cpu().float()
    T, K = v.shape
    p = torch.nn.functional.pad(v, (0, -K % 128)).view(T, (K + 127) // 128, 128)
    amax = torch.where(p.isnan(), torch.zeros_like(p), p.abs()).amax(-1).clamp_min(1e-12)
    s = torch.full_like(amax, 448.0) / amax
    u = p * s[..., None]
    q = u.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(T, -1)[:, :K], torch.ones_like(s) / s


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("T,K,pad,off", [(1, 1, 0, 0), (1, 128, 0, 0), (3, 127, 0, 0), (5, 129, 3, 1), (2, 2048, 0, 0), (300, 1999, 5, 0),
                                         (257, 256, 8, 8), (4096, 384, 0, 0), (7, 16384, 0, 0)])
def test_quantize(dtype, T, K, pad, off):
    g = gen(T + K)
    buf = torch.full((T, K + pad + off), float("nan"), dtype=DT[dtype], device="cuda")
    x = buf[:, off:off + K]
    x.copy_(torch.randn((T, K), generator=g, device="cuda") * torch.exp(2.0 * torch.randn((T, 1), generator=g, device="cuda")))
    q, s = M.moe_fp8_quantize(x)
    wq, ws = plain_quantize(x)
    assert q.dtype == torch.float8_e4m3fn and q.shape == (T, K)
    assert torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s.cpu(), ws)


def test_quantize_edges():
    x = torch.zeros((6, 300), device="cuda")
    x[1] = 1e-20  # below the smallest maximum
    x[2, :] = torch.linspace(-3e38, 3e38, 300)
    x[3, 5] = float("nan")
    x[3, 6:] = 2.0
    x[4, 200] = float("-inf")
    x[5] = torch.arange(300) - 150.0
    q, s = M.moe_fp8_quantize(x)
    wq, ws = plain_quantize(x)
    for t in (0, 1, 2, 5):
        assert torch.equal(q[t].cpu().view(torch.uint8), wq[t].view(torch.uint8)) and torch.equal(s[t].cpu(), ws[t])
    v = q.float() * s.repeat_interleave(128, 1)[:, :300]
    assert v[3, 5].isnan() and torch.equal(v[3, 6:], x[3, 6:]) and (v[3, :5] == 0).all()
    assert v[4, 128:256].isnan().all() and (v[4, :128] == 0).all() and (v[4, 256:] == 0).all()
    # into the caller's tensors, with a pitch, on another stream
    codes = torch.full((6, 320), 9, dtype=torch.uint8, device="cuda")
    scale = torch.empty((6, 3), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.moe_fp8_quantize(x, codes=codes[:, :300], scale_inv=scale, stream=side)
    side.synchronize()
    assert torch.equal(codes[:, :300], q.view(torch.uint8)) and (codes[:, 300:] == 9).all() and torch.equal(scale.nan_to_num(), s.nan_to_num())
    q0, s0 = M.moe_fp8_quantize(x[:0])
    assert q0.shape == (0, 300) and s0.shape == (0, 3)
    for bad in (dict(x=x.double()), dict(x=x.t()), dict(x=x, codes=torch.empty((6, 299), dtype=torch.uint8, device="cuda")),
                dict(x=x, scale_inv=torch.empty((6, 2), device="cuda")), dict(x=x[:, :0])):
        with pytest.raises(M.MoEError):
            M.moe_fp8_quantize(**bad)


def test_quantize_agrees_with_the_experts_quantizer():
    x = (torch.randn((33, 512), generator=gen(1), device="cuda") * 3).bfloat16()
    q, s = M.moe_fp8_quantize(x)
    wq, ws = M.moe_debug_quant_act_fp8(x)
    assert torch.equal(q.view(torch.uint8), wq) and torch.equal(s, ws)


# ------------------------------------------------------------------------------------------ products
def make_weight(N, K, g, amp=1.0):
    w = (torch.randn((N, K), generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = amp * (0.2 + torch.rand(((N + 127) // 128, (K + 127) // 128), generator=g, device="cuda")) / (100 * K ** 0.5)
    return M.Fp8Weight(w, s)


def linear_reference(q, qs, weight, act, base, dtype):
    K, N = q.shape[1], weight.codes.shape[0]
    a = q.double() * qs.double().repeat_interleave(128, 1)[:, :K]
    w = weight.codes.view(torch.float8_e4m3fn).double()
    w = w * weight.scale_inv.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y, e = a @ w.t(), (a.abs() @ w.abs().t()) * (K + 16) * 2.0 ** -23
    if act == "silu_mul":
        g, u, eg, eu = y[:, :N // 2], y[:, N // 2:], e[:, :N // 2], e[:, N // 2:]
        sg = g * torch.sigmoid(g)
        y, e = sg * u, 1.1 * eg * (u.abs() + eu) + sg.abs() * eu + 16 * U * (sg * u).abs()
    if base is not None:
        y = y + base.double()
        e = e + U * y.abs()
    return y, e + half(dtype) * (y.abs() + e) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def check_linear(out, x, weight, act="none", base=None, x_scale=None):
    q, qs = (x, x_scale) if x_scale is not None else plain_quantize(x)
    ref, tol = linear_reference(q.cuda(), qs.cuda(), weight, act, base, out.dtype)
    d = (out.double() - ref).abs()
    assert torch.isfinite(out).all() and (d <= tol).all(), f"{(d / tol).max().item():.3f} of the bound"
    assert d.norm() <= (half(out.dtype) + 2e-5) * ref.norm() + 1e-6 * ref.numel() ** 0.5 * (out.dtype == torch.float16)


ROWS = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 257, 513]


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("K,N", [(128, 128), (512, 200), (1504, 64)])
def test_linear_rows(T, K, N):
    g = gen(T)
    x = (torch.randn((T, K), generator=g, device="cuda") * torch.exp(torch.randn((T, 1), generator=g, device="cuda"))).bfloat16()
    w = make_weight(N, K, g)
    check_linear(M.moe_fp8_linear(x, w), x, w)
    check_linear(M.moe_fp8_linear(x, w, act="silu_mul"), x, w, "silu_mul")


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("K", [16, 112, 144, 272, 2048, 4112])
@pytest.mark.parametrize("N", [1, 2, 8, 63, 130, 1111])
def test_linear_sizes(T, K, N):
    g = gen(K + N)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = make_weight(N, K, g)
    check_linear(M.moe_fp8_linear(x, w, dtype=torch.float32), x, w)


@pytest.mark.parametrize("T", [3, 48, 260])
@pytest.mark.parametrize("x_type", ["bf16", "f16", "f32", "codes"])
@pytest.mark.parametrize("out_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("with_base", [False, True])
def test_linear_types(T, x_type, out_type, act, with_base):
    g = gen(T)
    K, N = 400, 328
    n = N // 2 if act == "silu_mul" else N
    w = make_weight(N, K, g)
    v = torch.randn((T, K + 16), generator=g, device="cuda")
    base = torch.randn((T, n + 3), generator=g, device="cuda").to(DT[out_type])[:, 1:1 + n] if with_base else None
    out = torch.full((T, n + 5), 7.0, dtype=DT[out_type], device="cuda")
    if x_type == "codes":
        q, s = M.moe_fp8_quantize(v[:, :K])
        wide = torch.zeros((T, K + 16), dtype=torch.uint8, device="cuda")
        wide[:, :K] = q.view(torch.uint8)
        x, xs = wide[:, :K].view(torch.float8_e4m3fn) if T == 3 else wide[:, :K], s
    else:
        x, xs = v.to(DT[x_type])[:, 3:3 + K], None
    got = M.moe_fp8_linear(x, w, x_scale=xs, act=act, base=base, out=out[:, 2:2 + n])
    assert got.data_ptr() == out[:, 2:].data_ptr() and (out[:, :2] == 7.0).all() and (out[:, 2 + n:] == 7.0).all()
    check_linear(got, x if xs is None else x.view(torch.float8_e4m3fn), w, act, base, xs)
    fresh = M.moe_fp8_linear(x, w, x_scale=xs, act=act, base=base, dtype=DT[out_type])
    assert torch.equal(fresh, got)
    if with_base:  # added in place
        b = base.clone()
        assert torch.equal(M.moe_fp8_linear(x, w, x_scale=xs, act=act, base=b, out=b), got)


@pytest.mark.parametrize("T", [8, 9, 16, 17])
@pytest.mark.parametrize("K,N,act", [(4096, 4096, "none"), (4096, 4097, "none"), (4096, 14336, "none"), (4096, 14336, "silu_mul")])
def test_linear_rows_of_large_matrices(T, K, N, act):
    # both sides of 8 and 16 rows and of 2^24 weights, where one kernel takes over from another
    g = gen(T + N)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = make_weight(N, K, g)
    out = M.moe_fp8_linear(x, w, act=act)
    check_linear(out, x, w, act)
    for t in (0, T - 1):  # and a row comes out of them alike, but for the order of its sums
        check_linear(M.moe_fp8_linear(x[t:t + 1], w, act=act), x[t:t + 1], w, act)


@pytest.mark.parametrize("T", [24, 100])
@pytest.mark.parametrize("K,N,act", [(2048, 200, "silu_mul"), (2048, 2742, "silu_mul"), (1040, 256, "silu_mul"), (2048, 2752, "silu_mul"), (2048, 1111, "none"),
                                     (4112, 64, "none")])
@pytest.mark.parametrize("out_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_base", [False, True])
def test_linear_of_long_rows_in_clusters(T, K, N, act, out_type, with_base):
    # eight groups of columns and more, in few tiles: a cluster's blocks share the groups, two or four to a tile; ups that cross a
    # block of 128 rows among them (100 and 1371 gates)
    g = gen(T + K + N)
    n = N // 2 if act == "silu_mul" else N
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = make_weight(N, K, g)
    base = torch.randn((T, n + 3), generator=g, device="cuda").to(DT[out_type])[:, 2:2 + n] if with_base else None
    out = torch.full((T + 1, n + 5), 7.0, dtype=DT[out_type], device="cuda")
    M.moe_fp8_linear(x, w, act=act, base=base, out=out[:T, 1:1 + n])
    assert (out[:, :1] == 7.0).all() and (out[:, 1 + n:] == 7.0).all() and (out[T:] == 7.0).all()
    check_linear(out[:T, 1:1 + n], x, w, act, base)
    assert torch.equal(M.moe_fp8_linear(x, w, act=act, base=base, dtype=DT[out_type]), out[:T, 1:1 + n])
    if with_base:
        b = base.clone()
        assert torch.equal(M.moe_fp8_linear(x, w, act=act, base=b, out=b), out[:T, 1:1 + n])
    assert M.moe_get_fp8_linear_error() == 0


@pytest.mark.parametrize("T,K,N,act", [(1, 2048, 4096, "none"), (96, 2048, 3200, "silu_mul"), (1237, 1504, 1111, "none"), (2500, 1536, 2048, "none"),
                                       (4000, 1024, 2304, "silu_mul")])
def test_linear_at_full_size(T, K, N, act):
    g = gen(T)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = make_weight(N, K, g)
    out = M.moe_fp8_linear(x, w, act=act)
    check_linear(out, x, w, act)
    assert torch.equal(M.moe_fp8_linear(x, w, act=act), out)


@pytest.mark.parametrize("T,K,N,act", [(2000, 400, 2742, "silu_mul"), (2305, 272, 2808, "none"), (100, 512, 39000, "none"), (70, 144, 39002, "silu_mul")])
@pytest.mark.parametrize("out_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_linear_in_large_tiles(T, K, N, act, out_type, pad):
    # enough outputs for the tiles of 256: an odd number of them along either axis, ups that cross a block of 128 rows (1371 and
    # 19501 gates), the last tiles ragged; rows of out on multiples of 16 bytes and not; base elsewhere and in place
    g = gen(T + N)
    n = N // 2 if act == "silu_mul" else N
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = make_weight(N, K, g)
    wide = n + -n % 8 + 8 + pad
    out = torch.full((T + 1, wide), 7.0, dtype=DT[out_type], device="cuda")
    M.moe_fp8_linear(x, w, act=act, out=out[:T, :n])
    assert (out[:T, n:] == 7.0).all() and (out[T:] == 7.0).all()
    check_linear(out[:T, :n], x, w, act)
    base = torch.randn((T + 1, wide), generator=g, device="cuda").to(DT[out_type])
    keep = base.clone()
    M.moe_fp8_linear(x, w, act=act, base=base[:T, :n], out=out[:T, :n])
    check_linear(out[:T, :n], x, w, act, keep[:T, :n])
    M.moe_fp8_linear(x, w, act=act, base=base[:T, :n], out=base[:T, :n])
    assert torch.equal(base[:T, :n], out[:T, :n]) and torch.equal(base[:T, n:], keep[:T, n:]) and torch.equal(base[T:], keep[T:])
    assert M.moe_get_fp8_linear_error() == 0


def test_linear_of_the_smallest_largest_and_empty_groups():
    # weights and activations of zero, of the largest code, of scales that are zero, tiny and large
    for T in (5, 150):
        x = torch.full((T, 256), 1.0, device="cuda")
        x[1], x[2], x[3] = 0.0, 3e38, 1e-30
        codes = torch.full((130, 256), 448.0, device="cuda").to(torch.float8_e4m3fn)
        codes[7] = 0.0
        scale = torch.tensor([[1.0, 0.0], [1e-36, 1e-3]], device="cuda")
        w = M.Fp8Weight(codes, scale)
        out = M.moe_fp8_linear(x, w, dtype=torch.float32)
        rows = [t for t in range(T) if t != 2]
        q, qs = plain_quantize(x)
        ref, tol = linear_reference(q.cuda(), qs.cuda(), w, "none", None, torch.float32)
        # a product of two scales below 2^-126 may be lost: 2^-126 for each of 256 products of codes up to 448^2
        assert ((out.double() - ref).abs() <= tol + 2.0 ** -126 * 256 * 448.0 ** 2)[rows].all()
        assert (out[:, 7] == 0).all() and (out[1] == 0).all() and out[2, 0].isinf()  # 3e38 448 128 is past fp32


@pytest.mark.parametrize("T,K,N,act", [(1, 256, 200, "none"), (5, 272, 256, "silu_mul"), (12, 256, 200, "silu_mul"), (16, 2048, 130, "none"), (24, 256, 200, "none"),
                                       (24, 2048, 200, "silu_mul"), (40, 2048, 3200, "none"), (150, 256, 256, "silu_mul"), (150, 256, 200, "silu_mul"),
                                       (600, 256, 4096, "none"), (600, 256, 4096, "silu_mul"), (700, 256, 3998, "silu_mul")])
@pytest.mark.parametrize("turn", range(4))
def test_linear_scales_whose_product_alone_leaves_the_range(T, K, N, act, turn):
    # rows and blocks of weight rows with scales from 2^-120 to 2^120, in every combination; codes of zero among them.  Sums that
    # fp32 holds come out within their bound, zeros as zeros
    g = gen(T + N + turn)
    G = (K + 127) // 128
    codes = lambda *s: (torch.randn(s, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    near = lambda *s: 0.75 + 0.25 * torch.rand(s, generator=g, device="cuda")  # noqa: E731
    x, w = codes(T, K), codes(N, K)
    x[T // 2] = 0.0
    w[3], w[N // 2 + 5] = 0.0, 0.0
    of_row = torch.tensor([1.0, 2.0 ** 100, 2.0 ** -100, 2.0 ** 120, 2.0 ** -120, 1e30, 2.0 ** -45, 0.0], device="cuda")
    of_block = torch.tensor([2.0 ** 100, 2.0 ** -100, 1e3, 2.0 ** -70, 1.0, 2.0 ** 70, 2.0 ** -120, 0.0], device="cuda")
    xs = near(T, G) * of_row[(torch.arange(T, device="cuda") * 5 + turn) % 8][:, None]
    ws = near((N + 127) // 128, G) * of_block[(torch.arange((N + 127) // 128, device="cuda") * 3 + 2 * turn) % 8][:, None]
    weight = M.Fp8Weight(w, ws)
    out = M.moe_fp8_linear(x, weight, x_scale=xs, act=act, dtype=torch.float32).double()
    a = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    b = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y, size = a @ b.t(), a.abs() @ b.abs().t()
    e = size * (K + 16) * 2.0 ** -23 + 2.0 ** -149 * (G + 1)  # a subnormal sum is rounded to 2^-150 at each step
    held = size < 2.0 ** 126
    if act == "silu_mul":
        n = N // 2
        v, u, ev, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
        sv = v * torch.sigmoid(v)
        held = held[:, :n] & held[:, n:]
        # past e^88.7 the exponential is an infinity and silu 0, 88.8 e^-88.7 < 3e-37 at most
        y, e = sv * u, 1.1 * ev * (u.abs() + eu) + sv.abs() * eu + 16 * U * (sv * u).abs() + 3e-37 * u.abs() + 2.0 ** -148 * (1.0 + u.abs())
        held &= y.abs() + e < 2.0 ** 126
    assert held.any() and (out[held] - y[held]).abs().le((e + U * (y.abs() + e))[held]).all()
    assert (out[(size[:, :out.shape[1]] == 0) & held] == 0).all()


def test_operators_beside_each_other():
    # the layer for few tokens, products and the layer for many, each on a stream of its own, again and again
    a = Layer("int4", 32, 256, 8, 512, 256, seed=43)
    b = Layer("nvfp4_w4a16", 5, 16, 4, 640, 384, seed=47)
    g = gen(53)
    x = torch.randn((1500, 512), generator=g, device="cuda").bfloat16()
    w, w2 = make_weight(3000, 512, g), make_weight(200, 512, g)
    y = torch.empty_like(x[:64])
    logits = torch.randn((64, 256), generator=g, device="cuda")
    ws = torch.empty(M.moe_workspace_size(a.desc, 64, 8), dtype=torch.uint8, device="cuda")
    calls = [lambda s: a.run(stream=s), lambda s: b.run(stream=s), lambda s: M.moe_fp8_linear(x, w, stream=s),
             lambda s: M.moe_fp8_linear(x[:100], w2, act="silu_mul", stream=s),
             lambda s: (M.moe_layer_forward_scored(x[:64], logits, M.Router(), a.desc, a.packed, 8, y, ws, stream=s), y)[1].clone()]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    a.check(want[0])
    b.check(want[1])
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(10):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(c(s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i % len(calls)]) for i, o in enumerate(got))
    assert M.moe_get_device_error(a.ws) == M.moe_get_device_error(b.ws) == M.moe_get_device_error(ws) == M.moe_get_fp8_linear_error() == 0


@pytest.mark.parametrize("T", [4, 64, 300])
def test_linear_rows_are_independent(T):
    g = gen(T)
    x = torch.randn((T, 512), generator=g, device="cuda").bfloat16()
    w = make_weight(256, 512, g)
    clean = M.moe_fp8_linear(x, w)
    x[1, 3], x[2, 300] = float("nan"), float("inf")
    x[3] = 0.0
    out = M.moe_fp8_linear(x, w)
    assert out[1].isnan().all() and out[2].isnan().all() and (out[3] == 0).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[4:], clean[4:])


@pytest.mark.parametrize("T", [1, 24, 200, 700])
def test_linear_streams_and_graphs(T):
    g = gen(T)
    x = torch.randn((T, 1024), generator=g, device="cuda").bfloat16()
    w = make_weight(640, 1024, g)
    want = M.moe_fp8_linear(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [(M.moe_fp8_linear(x, w, stream=side), M.moe_fp8_linear(x, w)) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want) for a, b in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = M.moe_fp8_linear(x, w)
    graph.replay()
    assert torch.equal(y, want)
    x.mul_(-1)
    graph.replay()
    assert torch.equal(y, -want)
    q, s = M.moe_fp8_quantize(x)
    assert torch.equal(M.moe_fp8_linear(q, w, x_scale=s), -want)


def test_linear_empty_and_refusals():
    g = gen(0)
    x = torch.randn((4, 256), generator=g, device="cuda").bfloat16()
    w = make_weight(64, 256, g)
    assert M.moe_fp8_linear(x[:0], w).shape == (0, 64)
    q, s = M.moe_fp8_quantize(x)

    def refused(*a, **kw):
        with pytest.raises(M.MoEError) as e:
            M.moe_fp8_linear(*a, **kw)
        assert e.value.status == 1

    refused(x[:, :128], w)
    refused(x.double(), w)
    refused(q, w)  # codes without their scales
    refused(q, w, x_scale=s[:, :1])
    refused(x, w, x_scale=s)
    refused(x, w, act="relu")
    refused(x, w, dtype=torch.float64)
    refused(x, w, out=torch.empty((4, 63), dtype=torch.bfloat16, device="cuda"))
    refused(x, w, out=torch.empty((4, 64), dtype=torch.bfloat16, device="cuda"), dtype=torch.float32)
    refused(x, w, base=torch.empty((4, 64), device="cuda"), out=torch.empty((4, 64), dtype=torch.bfloat16, device="cuda"))
    refused(x, make_weight(63, 256, g), act="silu_mul")
    refused(x, w, base=torch.empty((4, 64)))
    codes = torch.zeros((64, 256), dtype=torch.uint8, device="cuda")
    for bad in ((codes[:, :24], torch.ones((1, 1), device="cuda")), (codes.float(), w.scale_inv), (codes, w.scale_inv[:, :1]), (codes, w.scale_inv.double()),
                (codes[:, ::2], torch.ones((1, 1), device="cuda")), (codes.view(-1)[8:8 + 63 * 256].view(63, 256), w.scale_inv)):
        with pytest.raises(M.MoEError):
            M.Fp8Weight(*bad)


# ------------------------------------------------------------------------------------------ together
def test_block_with_a_shared_expert_and_few_tokens():
    g = gen(41)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    E, H, I, k = 16, 512, 256, 4
    layer = M.MoELayer("fp8", (rnd(E, 2 * I, H) / H ** 0.5).bfloat16(), (rnd(E, H, I) / I ** 0.5).bfloat16())
    shared = (make_weight(2 * I, H, g), make_weight(H, I, g))
    wr, router = (rnd(E, H) / H ** 0.5).bfloat16(), M.Router("sigmoid", groups=4, top_groups=2, group_top=2, scale=2.0)
    bias = 0.02 * rnd(E)
    pre, post = M.Norm("rms", (1 + 0.1 * rnd(H)).bfloat16()), M.Norm("rms", (1 + 0.1 * rnd(H)).bfloat16())
    blk = M.MoEBlock(layer, wr, router, k, pre, post, bias, beta=0.5, shared=shared, few_tokens=8)
    plain = M.MoEBlock(layer, wr, router, k, pre, post, bias, beta=0.5, shared=shared)
    for T in (1, 8, 9):
        x = rnd(T, H)
        out = blk.forward(x)
        h = M.moe_block_enter(x, pre, dtype=torch.bfloat16)
        if T <= 8:
            m = M.moe_layer_few(h, wr, router, layer.desc, layer.packed, k, layer.ensure_few_workspace(T, k), bias=bias)
        else:
            m = torch.empty_like(h)
            M.moe_layer_forward_scored(h, h @ wr.t(), router, layer.desc, layer.packed, k, m, layer.ensure_workspace(T, k), bias=bias)
        m = M.moe_fp8_linear(M.moe_fp8_linear(h, shared[0], act="silu_mul"), shared[1], base=m, out=m)
        assert torch.equal(out, M.moe_block_leave(x, m, post=post, beta=0.5))
        # against the block without the operator for few tokens: its logits are bf16, its h too; rows routed alike agree
        other = plain.forward(x)
        hd = h.double()
        same = (M.moe_route_scored((hd @ wr.double().t()).float(), router, k, bias=bias)[0].sort(1).values
                == M.moe_route_scored(h @ wr.t(), router, k, bias=bias)[0].sort(1).values).all(1)
        # the logits' rounding moves a score by 2^-8 |l| / 4 at most, so the weights by a few 2^-8
        assert ((out - other)[same].norm() <= 4 * 2.0 ** -8 * (other - x)[same].norm()) if same.any() else True
    with pytest.raises(M.MoEError):
        M.MoEBlock(layer, wr, router, k, pre, few_tokens=33)


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_block_takes_its_router_at_any_length(w_dtype):
    g = gen(61)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    E, H, I, k = 16, 512, 256, 4
    layer = M.MoELayer("fp8", (rnd(E, 2 * I, H) / H ** 0.5).bfloat16(), (rnd(E, H, I) / I ** 0.5).bfloat16())
    wr, router, pre = (rnd(E, H) / H ** 0.5).to(w_dtype), M.Router(), M.Norm("rms")
    blk = M.MoEBlock(layer, wr, router, k, pre, few_tokens=8)
    for T in (0, 1, 8, 9, 300):
        x = rnd(T, H)
        h = M.moe_block_enter(x, pre, dtype=torch.bfloat16)
        m = torch.empty_like(h)
        if 0 < T <= 8:
            m = M.moe_layer_few(h, wr, router, layer.desc, layer.packed, k, blk.few_workspace)
        else:
            logits = h @ wr.t() if w_dtype == torch.bfloat16 else h.float() @ wr.float().t()
            M.moe_layer_forward_scored(h, logits, router, layer.desc, layer.packed, k, m, layer.ensure_workspace(T, k))
        assert torch.equal(blk.forward(x), M.moe_block_leave(x, m))


@pytest.mark.parametrize("few_tokens", [0, 8])
def test_block_of_no_tokens(few_tokens):
    layer = M.MoELayer("fp8", torch.zeros((4, 256, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 256, 128), dtype=torch.bfloat16, device="cuda"))
    blk = M.MoEBlock(layer, torch.zeros((256, 4), dtype=torch.bfloat16, device="cuda").t(), M.Router(), 2, M.Norm("rms"), few_tokens=few_tokens)
    assert blk.forward(torch.zeros((0, 256), device="cuda")).shape == (0, 256)


def test_few_graph_outlives_a_larger_block_on_the_same_layer():
    g = gen(59)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    E, H, I, k = 16, 512, 256, 4
    layer = M.MoELayer("fp8", (rnd(E, 2 * I, H) / H ** 0.5).bfloat16(), (rnd(E, H, I) / I ** 0.5).bfloat16())
    wr = (rnd(E, H) / H ** 0.5).bfloat16()
    make = lambda n: M.MoEBlock(layer, wr, M.Router(), k, M.Norm("rms"), few_tokens=n)  # noqa: E731
    a = make(2)
    assert M.moe_get_device_error(a.few_workspace) == 0  # polled before its first call
    x = rnd(2, H)
    want = a.forward(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = a.forward(x)
    b = make(32)
    n = a.few_workspace.numel()
    assert b.few_workspace.numel() > n
    over = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]  # whatever was given back
    graph.replay()
    assert torch.equal(y, want) and all((o == 7).all() for o in over)
    assert torch.equal(b.forward(x), want) and torch.equal(a.forward(x), want)
    assert M.moe_get_device_error(a.few_workspace) == M.moe_get_device_error(b.few_workspace) == 0


def test_graph_outlives_a_larger_batch_on_the_same_layer():
    g = gen(79)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    E, H, I, k = 16, 512, 256, 4
    layer = M.MoELayer("fp8", (rnd(E, 2 * I, H) / H ** 0.5).bfloat16(), (rnd(E, H, I) / I ** 0.5).bfloat16())
    blk = M.MoEBlock(layer, (rnd(E, H) / H ** 0.5).bfloat16(), M.Router(), k, M.Norm("rms"))
    x, many = rnd(40, H), rnd(900, H)
    want = blk.forward(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = blk.forward(x)
    n = layer.workspace.numel()
    blk.forward(many)
    assert layer.workspace.numel() > n
    over = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]  # whatever was given back
    graph.replay()
    assert torch.equal(y, want) and all((o == 7).all() for o in over)
    assert torch.equal(blk.forward(x), want)


def test_example_runs_with_few_tokens():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block

    x = moe_block.main(["--hidden", "512", "--inner", "256", "--experts", "16", "--top-k", "4", "--steps", "2", "--few"])
    assert torch.isfinite(x).all()
