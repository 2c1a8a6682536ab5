"""The operators around the experts against plain 64-bit implementations (GPU).

Tolerances come from rounding analysis, elementwise, with u = 2^-24 (fp32) and the output's half unit
in the last place relative to the value (8, 11 and 24 bits of significand: 2^-8 for bf16, 2^-11 for fp16
plus half its smallest subnormal, u for fp32):
  sums       a value summed from n terms passes through at most C = 64 roundings here (a thread adds at
             most 32 terms in a row, then ten levels of a tree join the threads), the elementwise steps
             around it, rsqrtf and expf (2 units each) included: error <= C u * (sum of magnitudes).
             Rows longer than a block's registers give a thread up to 64 terms: C = 128 covers both.
  products   an inner product of n terms in fp32 has error <= n 2^-23 * sum |a||b| in whatever order
             (2^-23: tensor cores may truncate); the adapters' inner values are then held in two bf16
             terms: 2^-17 relative.
Choices (indices) are compared exactly on inputs whose deciding keys are further apart than the
keys' own rounding, and on exact ties.
"""
import math

import numpy as np
import pytest
import torch

import nvfp4_expert_gemms_gb300 as M

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = 128
HALF_ULP = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25), torch.float32: (U, 0.0)}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(T, H, dtype, g, pad=0, scale=1.0, mean=0.0):
    buf = torch.full((T, H + pad), float("nan"), dtype=dtype, device="cuda")
    v = buf[:, :H]
    v.copy_(torch.randn((T, H), generator=g, device="cuda") * scale + mean)
    return v


# ------------------------------------------------------------------------------------------ norms
def ref_norm(v, e, kind, w, b, off, eps):
    """(norm(v), bound of its fp32 error) in fp64, for v known to within e (elementwise)."""
    m = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    r = 1.0 / torch.sqrt(((v - m) ** 2).mean(-1, keepdim=True) + eps)
    yh = (v - m) * r
    mag = (v.abs() + (v.abs().mean(-1, keepdim=True) if kind == "layer" else 0.0)) * r
    em = e.mean(-1, keepdim=True) if kind == "layer" else 0.0
    err = (e + em) * r + C * U * mag + yh.abs() * (((e + em) ** 2).mean(-1, keepdim=True).sqrt() * r + C * U * (
        1.0 + (mag ** 2).mean(-1, keepdim=True).sqrt()))
    if w is not None:
        wf = w.double() + off
        yh, err = yh * wf, err * wf.abs()
    if b is not None:
        yh = yh + b.double()
        err = err + U * yh.abs()
    return yh, err + 4 * U * yh.abs()


def check(got, ref, err, what=""):
    rel, sub = HALF_ULP[got.dtype]
    bad = ~((got.double() - ref).abs() <= ref.abs() * rel + sub + err * (1 + rel))
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside, worst {float((got.double() - ref).abs().max()):.3e}"


def make_norm(kind, H, dtype, g, weight=True, bias=True, off=0.0, eps=1e-6):
    w = (torch.randn(H, generator=g, device="cuda") * 0.3 + 1.0 - off).to(dtype) if weight else None
    b = (torch.randn(H, generator=g, device="cuda") * 0.2).to(dtype) if bias else None
    return M.Norm(kind, w, b, eps=eps, offset=off), (kind, w, b, off, eps)


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 33), (5, 64), (1, 2048), (7, 2048), (300, 256), (4, 999), (9, 1000), (3, 4096),
          (2, 5001), (2, 8192), (2, 8200), (2, 9001), (1, 16384), (1, 40000), (1, 70000)]


@pytest.mark.parametrize("types", ["bf16/bf16", "f16/f16", "f32/f32", "f32/bf16", "f32/f16"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_enter(types, T, H):
    xt, yt = (DT[t] for t in types.split("/"))
    for i, (kind, weight, bias, off, pad) in enumerate([("rms", True, False, 0.0, 0), ("layer", True, True, 1.0, 3),
                                                        ("rms", False, False, 1.0, 8), ("layer", False, True, 0.0, 16)]):
        g = gen(17 * T + H + i)
        x = rows(T, H, xt, g, pad, 2.0, 0.7)
        norm, spec = make_norm(kind, H, DT["f32"] if i == 1 else yt, g, weight, bias, off)
        got = M.moe_block_enter(x, norm, dtype=yt)
        v = x.double()
        ref, err = ref_norm(v, torch.zeros_like(v), *spec)
        check(got, ref, err, f"{kind} {types} {T}x{H} pad {pad}")


@pytest.mark.parametrize("types", ["bf16/bf16", "f16/f16", "f32/f32", "f32/bf16", "f32/f16"])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 2048), (2, 40), (5, 999), (33, 1024), (3, 2056), (2, 9001), (2, 36000)])
def test_leave(types, gate, T, H):
    xt, at = (DT[t] for t in types.split("/"))
    for i, (kind, post, nxt, act, pad) in enumerate([("rms", True, True, "none", 0), ("layer", True, True, "sigmoid", 5),
                                                     ("layer", False, True, "tanh", 8), ("rms", True, False, "sigmoid", 0),
                                                     ("rms", False, False, "none", 16)]):
        g = gen(31 * T + H + i)
        x, b = rows(T, H, xt, g, pad, 1.5, 0.2), rows(T, H, at, g, pad, 0.4, -0.1)
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
        gt = None if shape is None else torch.randn(shape, generator=g, device="cuda").to(at if i % 2 else torch.float32)
        pn, ps = make_norm(kind, H, at, g) if post else (None, None)
        nn, ns = make_norm(kind, H, at, g, bias=False) if nxt else (None, None)
        alpha, beta = 0.9, -1.3
        got = M.moe_block_leave(x, b, post=pn, gate=gt, gate_act=act, alpha=alpha, beta=beta, next=nn)
        v = b.double()
        e = torch.zeros_like(v)
        if post:
            v, e = ref_norm(v, e, *ps)
        if gt is not None:
            gd = gt.double()
            f = {"none": gd, "sigmoid": torch.sigmoid(gd), "tanh": torch.tanh(gd)}[act]
            v, e = v * f, e * f.abs() + 8 * U * (v * f).abs()
        a32, b32 = float(np.float32(alpha)), float(np.float32(beta))
        e = abs(b32) * e + 4 * U * ((a32 * x.double()).abs() + (b32 * v).abs())
        o = a32 * x.double() + b32 * v
        out, y = got if nxt else (got, None)
        check(out, o, e, f"out {kind} {types} {gate} {act} {T}x{H}")
        if nxt:
            ry, ey = ref_norm(o, e, *ns)
            check(y, ry, ey, f"y {kind} {types} {gate} {act} {T}x{H}")


@pytest.mark.parametrize("H", [8200, 16384, 20001, 28928, 57856, 57864])
def test_long_rows(H):
    """Rows kept in shared memory, to the last column that fits and past it; in place."""
    for types, gate in (("bf16/bf16", "channel"), ("f16/f16", "full"), ("f32/f32", "token"), ("f32/bf16", "full"), ("f32/f16", "none")):
        test_enter(types, 2, H)
        test_leave(types, gate, 2, H)
    g = gen(H)
    for kind in ("rms", "layer"):
        x, b = rows(3, H, torch.float32, g, 16), rows(3, H, torch.bfloat16, g, 16)
        (p, _), (n, _) = make_norm(kind, H, torch.bfloat16, g), make_norm(kind, H, torch.bfloat16, g)
        out, y = M.moe_block_leave(x, b, post=p, next=n, beta=0.5)
        x2, b2 = x.clone(), b.clone()
        M.moe_block_leave(x2, b2, post=p, next=n, beta=0.5, out=x2, y=b2)
        assert torch.equal(x2, out) and torch.equal(b2, y)
        # parameters of two types
        (q, sq), (r, sr) = make_norm(kind, H, torch.float32, g), make_norm(kind, H, torch.bfloat16, g)
        got, y = M.moe_block_leave(x, b, post=q, next=r)
        v, e = ref_norm(b.double(), torch.zeros_like(b, dtype=torch.float64), *sq)
        o = x.double() + v
        e = e + 4 * U * (x.double().abs() + v.abs())
        check(got, o, e, f"out {kind} {H}")
        ry, ey = ref_norm(o, e, *sr)
        check(y, ry, ey, f"y {kind} {H}")


def test_leave_in_place_and_other_stream():
    g = gen(3)
    for T, H in ((6, 2048), (4, 1001), (1, 70000)):
        x, b = rows(T, H, torch.float32, g), rows(T, H, torch.bfloat16, g)
        (p, _), (n, _) = make_norm("layer", H, torch.bfloat16, g), make_norm("rms", H, torch.bfloat16, g)
        out, y = M.moe_block_leave(x, b, post=p, next=n, beta=0.5)
        x2, b2 = x.clone(), b.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        M.moe_block_leave(x2, b2, post=p, next=n, beta=0.5, out=x2, y=b2, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(x2, out) and torch.equal(b2, y)
        e = M.moe_block_enter(b, n)
        e2 = b.clone()
        assert torch.equal(M.moe_block_enter(e2, n, out=e2), e)


def test_norm_edges():
    """Rows of zeros, constants, infinities and NaN; neighbours keep their values; no rows at all."""
    g = gen(4)
    for H in (2048, 1003, 70000):
        x = rows(6, H, torch.float32, g)
        x[1] = 0.0
        x[2] = 5.0
        x[3, H // 2] = float("inf")
        x[4, 0] = float("nan")
        n, spec = make_norm("layer", H, torch.float32, g, bias=False)
        got = M.moe_block_enter(x, n)
        assert torch.equal(got[1], torch.zeros_like(got[1]))
        # a constant row: every difference from the mean is rounding of the mean, at most C u * 5
        lim = C * U * 5.0 / math.sqrt(1e-6) * (n.weight.abs() + 1)
        assert (got[2].abs() <= lim).all()
        assert torch.isnan(got[3]).all() and torch.isnan(got[4]).all()
        v = x[[0, 5]].double()
        ref, err = ref_norm(v, torch.zeros_like(v), *spec)
        check(got[[0, 5]], ref, err)
    n, _ = make_norm("rms", 64, torch.bfloat16, g)
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert M.moe_block_enter(empty, n).shape == (0, 64)
    assert M.moe_block_leave(empty, empty, next=n)[1].shape == (0, 64)


def test_layer_norm_keeps_the_variance_of_a_shifted_row():
    """Mean 1000 times the spread: the variance comes from differences, not from a difference of squares."""
    g = gen(5)
    x = rows(3, 2048, torch.float32, g, 0, 1.0, 1000.0)
    n, spec = make_norm("layer", 2048, torch.float32, g)
    v = x.double()
    ref, err = ref_norm(v, torch.zeros_like(v), *spec)
    got = M.moe_block_enter(x, n)
    check(got, ref, err)
    assert float(err.max()) < 0.2  # the bound itself says something


def test_offsets_past_32_bits():
    H, far = 2048, 2 ** 31 + 64
    buf = torch.empty(far + H, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, H), (far, 1))
    x.copy_(torch.randn((2, H), generator=gen(6), device="cuda"))
    n, _ = make_norm("rms", H, torch.bfloat16, gen(7))
    near = x.clone()
    assert torch.equal(M.moe_block_enter(x, n), M.moe_block_enter(near, n))
    lg = x[:, :128]
    r = M.Router("sigmoid", groups=4, top_groups=2, group_top=2)
    for p, q in zip(M.moe_route_scored(lg, r, 4), M.moe_route_scored(lg.contiguous(), r, 4)):
        assert torch.equal(p, q)
    a = torch.randn((1, 8, H), device="cuda").bfloat16()
    b = torch.randn((1, H, 8), device="cuda").bfloat16()
    starts, slot = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 2], [0]))
    want = M.moe_adapters_add(near, near, a, b, starts, slot)
    assert torch.equal(M.moe_adapters_add(x, x, a, b, starts, slot), want)
    M.moe_adapters_add(x, x, a, b, starts, slot, out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("types", ["bf16/bf16", "f16/f16", "f32/f32", "f32/bf16", "f32/f16"])
@pytest.mark.parametrize("T,H", [(16384, 264), (12000, 512), (5200, 776), (6000, 1024), (2700, 1032), (3000, 2048), (1500, 2056), (1500, 4096),
                                 (330, 4104), (400, 8192)])
def test_many_rows(types, T, H):
    """Rows that groups of warps walk with the grid's stride, several each: both slots of a group's ring and both of its
    sums' buffers come round.  Every gate, norm and bias, padded rows, parameters in fp32, out of place and in place."""
    xt, at = (DT[t] for t in types.split("/"))
    combos = [("rms", "none", "none", True, True, False, 0, False), ("layer", "channel", "sigmoid", True, True, True, 8, False),
              ("rms", "token", "sigmoid", True, True, True, 16, True), ("layer", "full", "tanh", True, True, True, 0, False),
              ("layer", "full", "none", False, True, False, 8, True), ("rms", "full", "sigmoid", True, False, False, 0, False),
              ("layer", "channel", "none", True, True, False, 0, True), ("layer", "token", "tanh", True, False, True, 24, False)]
    for i, (kind, gate, act, post, nxt, bias, pad, wide) in enumerate(combos):
        pt = torch.float32 if wide else at
        g = gen(7 * T + H + i)
        x, b = rows(T, H, xt, g, pad, 1.5, 0.2), rows(T, H, at, g, pad, 0.4, -0.1)
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
        gt = None if shape is None else torch.randn(shape, generator=g, device="cuda").to(pt)
        pn, ps = make_norm(kind, H, pt, g, bias=bias) if post else (None, None)
        nn, ns = make_norm(kind, H, pt, g, bias=bias, off=1.0) if nxt else (None, None)
        alpha, beta = 0.9, -1.3
        got = M.moe_block_leave(x, b, post=pn, gate=gt, gate_act=act, alpha=alpha, beta=beta, next=nn)
        v, e = b.double(), torch.zeros((1, 1), dtype=torch.float64, device="cuda").expand(T, H)
        if post:
            v, e = ref_norm(v, e, *ps)
        if gt is not None:
            gd = gt.double()
            f = {"none": gd, "sigmoid": torch.sigmoid(gd), "tanh": torch.tanh(gd)}[act]
            v, e = v * f, e * f.abs() + 8 * U * (v * f).abs()
        a32, b32 = float(np.float32(alpha)), float(np.float32(beta))
        e = abs(b32) * e + 4 * U * ((a32 * x.double()).abs() + (b32 * v).abs())
        o = a32 * x.double() + b32 * v
        out, y = got if nxt else (got, None)
        what = f"{kind} {types} {gate} {act} {T}x{H} pad {pad}"
        check(out, o, e, "out " + what)
        if nxt:
            ry, ey = ref_norm(o, e, *ns)
            check(y, ry, ey, "y " + what)
            got = M.moe_block_enter(x, nn, dtype=at)
            ry, ey = ref_norm(x.double(), torch.zeros_like(o), *ns)
            check(got, ry, ey, "enter " + what)
            M.moe_block_leave(x, b, post=pn, gate=gt, gate_act=act, alpha=alpha, beta=beta, next=nn, out=x, y=b)
            assert torch.equal(x, out) and torch.equal(b, y), "in place " + what
            M.moe_block_enter(b, nn, out=b)
            ry, ey = ref_norm(y.double(), torch.zeros_like(o), *ns)
            check(b, ry, ey, "enter in place " + what)


# ------------------------------------------------------------------------------------------ routing
def ref_route(lg, bias, score, k, groups, top_groups, group_top, renorm, scale):
    """Indices, weights and each row's smallest gap between keys that decide, in fp64."""
    T, E = lg.shape
    S = E // groups
    idx, w, gap = np.zeros((T, k), np.int64), np.zeros((T, k)), np.full(T, np.inf)
    for t in range(T):
        l = np.where(np.isnan(lg[t]), -np.inf, lg[t])
        mx = l.max()
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                p = 1.0 / (1.0 + np.exp(-l))
            else:
                e = np.exp(l - mx) if np.isfinite(mx) else np.zeros(E)
                p = e / e.sum() if e.sum() > 0 else e
        key = p + bias if bias is not None else l
        key = np.where(np.isnan(key), -np.inf, key)
        ok = np.ones(E, bool)
        if groups > 1:
            by = (p if bias is None and group_top == 2 else key).reshape(groups, S)
            top = -np.sort(-by, axis=1)[:, :group_top]
            val = top.sum(axis=1)
            order = sorted(range(groups), key=lambda i: (-val[i], i))
            if top_groups < groups:
                a, b = val[order[top_groups - 1]], val[order[top_groups]]
                gap[t] = min(gap[t], abs(a - b) if a != b else np.inf)
            ok = np.zeros(groups, bool)
            ok[order[:top_groups]] = True
            ok = np.repeat(ok, S)
        cand = sorted((i for i in range(E) if ok[i]), key=lambda i: (-key[i], i))
        for a, b in zip(cand[:k], cand[1:k + 1]):
            if key[a] != key[b]:
                gap[t] = min(gap[t], key[a] - key[b])
        idx[t] = cand[:k]
        s = p[cand[:k]]
        if renorm and score == "softmax":  # the chosen alone: their ratios need no common maximum
            lc = l[cand[:k]]
            s = np.exp(lc - lc.max()) if np.isfinite(lc.max()) else np.zeros(k)
        w[t] = (s / s.sum() if s.sum() > 0 else 0.0 * s) * scale if renorm else s * scale
    return idx, w, gap


def check_route(lg, k, score, bias=None, groups=1, top_groups=None, group_top=1, renorm=True, scale=1.0, gaps=True):
    top_groups = groups if top_groups is None else top_groups
    r = M.Router(score, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm, scale=scale)
    idx, w = M.moe_route_scored(lg, r, k, bias=bias)
    ri, rw, gap = ref_route(lg.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy(), score, k,
                            groups, top_groups, group_top, renorm, scale)
    # keys are within 8 u of their values (sums of two scores or a score and a bias below 4 in size)
    sure = gap > 32 * 8 * U if gaps else np.ones(len(gap), bool)
    assert sure.mean() > 0.5 or len(sure) < 8  # the inputs leave something to compare
    idx, w = idx.cpu().numpy(), w.cpu().numpy()
    assert (idx >= 0).all() and (idx < lg.shape[1]).all()
    assert all(len(set(row)) == k for row in idx.tolist())
    assert np.array_equal(idx[sure], ri[sure])
    # a weight: expf (2 u) and a division over a sum of at most 8 scores or, over all experts, 64 roundings
    np.testing.assert_allclose(w[sure], rw[sure], rtol=(80 if score == "softmax" and not renorm else 24) * U, atol=1e-37)


ROUTERS = [dict(score="softmax"), dict(score="sigmoid"), dict(score="softmax", renorm=False, scale=2.0),
           dict(score="sigmoid", renorm=False), dict(score="sigmoid", bias=True, scale=2.5),
           dict(score="softmax", bias=True, renorm=False)]


@pytest.mark.parametrize("E,groups", [(1, 1), (2, 2), (7, 1), (8, 8), (16, 4), (32, 32), (33, 3), (60, 6), (64, 1), (90, 5),
                                      (128, 1), (128, 8), (160, 8), (200, 1), (256, 1), (256, 2), (256, 8), (256, 32), (255, 17), (249, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route(E, groups, dtype):
    S = E // groups
    for i, spec in enumerate(ROUTERS):
        for T, k in ((1, 1), (37, min(8, E)), (5, min(3, E))):
            g = gen(1000 * E + 10 * groups + i)
            lg = rows(T, E, DT[dtype], g, pad=(0, 1, 4)[i % 3], scale=1.5)
            spec2 = dict(spec)
            if spec2.pop("bias", False):
                spec2["bias"] = 0.2 * torch.randn(E, generator=g, device="cuda")
            need = -(-k // S)
            for tg in {need, max(need, groups // 2), groups}:
                for gt in (1, 2):
                    check_route(lg, k, groups=groups, top_groups=tg, group_top=gt, **spec2)


def test_route_matches_the_layers_router():
    """The default router chooses and weighs as moe_layer_forward's own routing does."""
    for T, E, k in ((1, 128, 8), (100, 128, 8), (700, 256, 8), (50, 7, 7)):
        lg = rows(T, E, torch.float32, gen(T + E))
        idx, w = M.moe_route_scored(lg, M.Router(), k)
        ws = torch.empty(M.moe_workspace_size(M.moe_packed_size("fp8", E, 128, 128), T, k), dtype=torch.uint8, device="cuda")
        ri, rw = M.moe_debug_route(lg, k, ws)[:2]
        assert torch.equal(idx, ri)
        np.testing.assert_allclose(w.cpu().numpy(), rw.cpu().numpy(), rtol=1e-6)


def test_route_ties_and_masked_experts():
    """Equal keys go to the lower index, also across lanes and groups; -inf, lowest values, NaN and
    whole rows without an expert."""
    lo = torch.finfo(torch.float32).min
    inf = float("inf")
    for E, groups in ((64, 1), (64, 8), (60, 6), (256, 8)):
        S = E // groups
        lg = torch.zeros((9, E), device="cuda")
        lg[1, ::2] = 1.0
        lg[2] = -inf
        lg[3] = lo
        lg[4] = float("nan")
        lg[5] = -inf
        lg[5, E - 1] = 0.5
        lg[6] = lo
        lg[6, E // 2] = -inf
        lg[7, :] = -0.0
        lg[7, 1] = 0.0
        lg[8] = torch.arange(E, device="cuda") // 3 * 1.0
        for score in ("softmax", "sigmoid"):
            for tg in {groups, max(1, groups // 2)}:
                k = min(8, S * tg)
                check_route(lg, k, score, groups=groups, top_groups=tg, gaps=False)
                check_route(lg, k, score, groups=groups, top_groups=tg, renorm=False, gaps=False)
                r = M.Router(score, groups=groups, top_groups=tg)
                w = M.moe_route_scored(lg, r, k)[1]
                assert torch.equal(w[[2, 4]], torch.zeros_like(w[[2, 4]])) and torch.isfinite(w).all()
    # a bias of -inf takes an expert out; scores equal, biases tie
    bias = torch.zeros(64, device="cuda")
    bias[:30] = -inf
    idx, w = M.moe_route_scored(torch.zeros((2, 64), device="cuda"), M.Router("sigmoid"), 8, bias=bias)
    assert idx.tolist() == [list(range(30, 38))] * 2
    np.testing.assert_allclose(w.cpu().numpy(), 0.125, rtol=24 * U)
    idx, w = M.moe_route_scored(torch.empty((0, 64), device="cuda"), M.Router("sigmoid"), 8)
    assert idx.shape == (0, 8) and w.shape == (0, 8)


@pytest.mark.parametrize("E,groups", [(7, 1), (64, 8), (128, 1), (256, 8)])
def test_route_infinite_logit(E, groups):
    """A +inf logit: softmax is NaN for the whole row, so are its weights; its neighbours and sigmoid scores are not."""
    k = min(8, E)
    lg = rows(3, E, torch.float32, gen(E))
    lg[1, E // 2] = float("inf")
    for renorm in (False, True):
        idx, w = M.moe_route_scored(lg, M.Router("softmax", groups=groups, renormalize=renorm), k)
        assert int(idx[1, 0]) == E // 2 and torch.isnan(w[1]).all() and torch.isfinite(w[[0, 2]]).all()
        # with a bias every key of the row is NaN, hence -infinity: the lowest experts
        idx, w = M.moe_route_scored(lg, M.Router("softmax", groups=groups, renormalize=renorm), k, bias=torch.randn(E, device="cuda"))
        assert idx[1].tolist() == list(range(k)) and torch.isnan(w[1]).all() and torch.isfinite(w[[0, 2]]).all()
        if groups > 1:  # groups by two scores: all of them -infinity, the lowest are kept
            idx, w = M.moe_route_scored(lg, M.Router("softmax", groups=groups, top_groups=2, group_top=2, renormalize=renorm), k)
            assert int(idx[1].max()) < 2 * E // groups and torch.isnan(w[1]).all() and torch.isfinite(w[[0, 2]]).all()
    idx, w = M.moe_route_scored(lg, M.Router("sigmoid", groups=groups, renormalize=False), k)
    assert int(idx[1, 0]) == E // 2 and w[1, 0] == 1.0 and torch.isfinite(w).all()


@pytest.mark.parametrize("size", [64.0, 256.0, 4096.0])
def test_route_groups_whose_keys_cancel(size):
    """The choice does not depend on the kernel's path: the same experts among others that cannot win.  A group's best
    two keys are near +size and -size, its value their sum, and the groups' values are a few of the keys' roundings apart."""
    T, groups, S, wide = 200000, 8, 8, 32
    g = gen(int(size))
    # scores where a key's rounding turns, to within their own: half units of the keys, some 6 units apart
    ulp = size * 2.0 ** -23
    turn = 0.5 + (torch.randn((T, groups, S), generator=g, device="cuda").double() * 6).round() * ulp + ulp / 2
    lg = (torch.logit(turn) + torch.randn((T, groups, S), generator=g, device="cuda") * 2.0 ** -22).float()
    bias = torch.full((groups, S), -3.0 * size, device="cuda")
    bias[:, 0], bias[:, 1] = size, -size - 1.0
    r = M.Router("sigmoid", groups=groups, top_groups=4, group_top=2)
    idx, w = M.moe_route_scored(lg.reshape(T, -1), r, 4, bias=bias.reshape(-1))
    lg2, bias2 = torch.zeros((T, groups, wide), device="cuda"), torch.full((groups, wide), -9.0 * size, device="cuda")
    lg2[..., :S], bias2[:, :S] = lg, bias
    idx2, w2 = M.moe_route_scored(lg2.reshape(T, -1), r, 4, bias=bias2.reshape(-1))
    assert torch.equal(idx2 // wide * S + idx2 % wide, idx) and torch.equal(w, w2)


def test_norm_follows_its_parameters():
    """Parameters that are replaced, given other storage or written in place are the ones that the next call uses."""
    g = gen(12)
    x = rows(3, 64, torch.bfloat16, g)
    w = torch.nn.Parameter(torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    old = w.data
    n = M.Norm("rms", w)
    one = M.moe_block_enter(x, n)
    w.data = torch.full((64,), 2.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(M.moe_block_enter(x, n), 2 * one)
    n.weight = torch.full((64,), 4.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(M.moe_block_enter(x, n), 4 * one)
    n.weight.fill_(0.5)
    assert torch.equal(M.moe_block_enter(x, n), one / 2)
    n.weight, n.bias = None, torch.full((64,), 3.0, device="cuda")
    assert (M.moe_block_enter(x.float(), n).mean() - 3.0).abs() < 1.0
    n.bias = None
    assert torch.equal(M.moe_block_enter(x, n), one)
    n.weight = w
    w.data = w.data[:32].clone()
    refused(1, M.moe_block_enter, x, n)  # another length now
    w.data = old.float()
    assert torch.equal(M.moe_block_enter(x, n), one)
    w.data = torch.ones(128, dtype=torch.bfloat16, device="cuda")[::2]
    refused(1, M.moe_block_enter, x, n)
    with pytest.raises(M.MoEError):
        n.weight = torch.ones((2, 32), device="cuda")
    del old


def test_copies_of_norms_and_routers():
    """A copy has its own descriptor and outlives what it was copied from."""
    import copy
    import gc

    g = gen(13)
    x, lg = rows(3, 64, torch.bfloat16, g), rows(3, 64, torch.float32, g)
    n, _ = make_norm("layer", 64, torch.bfloat16, g, off=1.0)
    r = M.Router("sigmoid", groups=4, top_groups=2, scale=2.5)
    want, (idx, w) = M.moe_block_enter(x, n), M.moe_route_scored(lg, r, 4)
    pairs = [(copy.copy(n), copy.copy(r)), (copy.deepcopy(n), copy.deepcopy(r))]
    del n, r
    gc.collect()
    other = [M.Router("softmax", scale=9.0) for _ in range(100)]  # what the first one's memory may hold now
    for m, q in pairs:
        assert torch.equal(M.moe_block_enter(x, m), want)
        assert torch.equal(M.moe_route_scored(lg, q, 4)[0], idx) and torch.equal(M.moe_route_scored(lg, q, 4)[1], w)
    del other


# ------------------------------------------------------------------------------------------ adapters
@pytest.mark.parametrize("E,groups,tg", [(256, 8, 1), (256, 16, 2), (128, 8, 1), (240, 8, 1), (256, 8, 2)])
def test_route_few_groups(E, groups, tg):
    """Candidates in fewer lanes than are chosen, with a bias: keys apart by construction, experts that the bias or
    the logits rule out (the bias's have equal keys: the lower index goes first)."""
    S, k, inf = E // groups, 8, float("inf")
    g = gen(E + groups)
    bias = 0.0103 * torch.randperm(E, generator=g, device="cuda").float()
    lg = torch.zeros((6, E), device="cuda")
    lg[1] = -inf
    lg[2, ::2] = -inf
    lg[3] = inf
    lg[4, ::3] = float("nan")
    lg[5, : E // 2] = 40.0
    for only in (None, 0, groups - 1):  # a group that wins with three experts left
        b = bias.clone()
        if only is not None:
            b[only * S: only * S + 3] += 9.0
            b[only * S + 3: (only + 1) * S] = -inf
        for gt in (1, 2):
            check_route(lg, k, "sigmoid", bias=b, groups=groups, top_groups=tg, group_top=gt, gaps=False)


def ref_adapters(x, base, a, b, starts, slot, scale, rank):
    """base + scale B (A x) in fp64 and the bound of the error before the last rounding."""
    x, a, b, out = x.double(), a.double(), b.double(), base.double()
    err = out.abs() * (a.shape[1] + 2) * 2.0 ** -23
    for q, s in enumerate(slot):
        lo, hi = starts[q], starts[q + 1]
        if 0 <= s < a.shape[0] and hi > lo:
            r = a.shape[1] if rank is None else rank[s]
            f = 1.0 if scale is None else scale[s]
            A, B = a[s, :r], b[s, :, :r]
            v, vm = x[lo:hi] @ A.t(), x[lo:hi].abs() @ A.abs().t()
            ev = vm * a.shape[2] * 2.0 ** -23 + v.abs() * 2.0 ** -17
            out[lo:hi] += f * (v @ B.t())
            err[lo:hi] += abs(f) * (ev @ B.abs().t() + (v.abs() @ B.abs().t()) * (2 * r + 4) * 2.0 ** -23)
    return out, err


def run_adapters(lens, slot, H, N, n, r, seed, rank=None, scale=True, pad=0, junk=True, in_place=False):
    g = gen(seed)
    T = sum(lens)
    starts = [0]
    for v in lens:
        starts.append(starts[-1] + v)
    x, base = rows(T, H, torch.bfloat16, g, pad), rows(T, N, torch.bfloat16, g, pad)
    a = (torch.randn((n, r, H), generator=g, device="cuda") / math.sqrt(H)).bfloat16()
    b = (torch.randn((n, N, r), generator=g, device="cuda") / math.sqrt(r)).bfloat16()
    if rank is not None and junk:  # what stands past an adapter's rank is never used
        for s in range(n):
            a[s, rank[s]:] = float("nan")
            b[s, :, rank[s]:] = float("inf")
    sc = (0.5 + torch.rand(n, generator=g, device="cuda")) if scale else None
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ref, err = ref_adapters(x, base, a, b, starts, slot, None if sc is None else sc.double().tolist(), rank)
    out = base if in_place else None
    got = M.moe_adapters_add(x, base, a, b, i32(starts), i32(slot), scale=sc, rank=None if rank is None else i32(rank), out=out)
    check(got, ref, err, f"{lens} {slot} {H}->{N} r {r} {rank}")
    return got


@pytest.mark.parametrize("r", [8, 16, 24, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("H,N", [(8, 8), (40, 264), (256, 72), (2048, 2048), (1000, 1536)])
def test_adapters(r, H, N):
    run_adapters([1], [0], H, N, 1, r, 1)
    run_adapters([1, 1, 1, 1, 1], [2, 0, -1, 1, 2], H, N, 3, r, 2, pad=8)
    run_adapters([17, 0, 1, 200, 16, 5], [0, 1, 2, 1, -1, 0], H, N, 3, r, 3, rank=[r, 1, max(1, r - 3)])
    run_adapters([700, 530, 515], [1, -1, 0], H, N, 2, r, 4, rank=[max(1, r // 2), r], in_place=True, pad=16)


@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("H,N,pad", [(2048, 1536, 16), (1000, 320, 0), (512, 264, 8), (2048, 72, 0)])
def test_adapters_long_requests(r, H, N, pad):
    """Sizes whose requests fill whole tiles: every kernel for long requests (T r (H + N) large enough for it, and
    for a tile shared by four blocks, by two and by none), ranks and rows that end inside a tile, requests
    without an adapter among them."""
    n = 3
    rank = [r, max(1, r - 5), max(1, r // 2)]
    whole = next(v for v in (16, 32, 64, 128) if r <= v)
    T = max(9200, int(9e8 / (whole * (H + N))) + 1)
    run_adapters([T - 5000, 1, 128, 0, 127, 4096, 600], [0, 1, 2, 0, 1, -1, 2], H, N, n, r, 11, rank=rank, pad=pad)
    run_adapters([T, 129], [1, 2], H, N, n, r, 12, rank=rank, pad=pad, in_place=True, scale=False)
    run_adapters([200, T - 3000, 17000], [2, 7, 0], H, N, n, r, 13, pad=pad)
    if whole == 128 and H + N > 2048:  # few enough tiles for four blocks each
        run_adapters([2600, 500], [0, 1], H, N, n, r, 14, rank=rank, pad=pad)


@pytest.mark.parametrize("r", [8, 16])
@pytest.mark.parametrize("H,N,pad", [(2048, 1536, 16), (1000, 320, 0), (40, 264, 8)])
def test_adapters_tiles_of_32(r, H, N, pad):
    """Low ranks whose requests fill tiles of 32: shared by eight blocks, four, two and none, tiles of one to 32
    rows, requests without tokens or without an adapter."""
    rank = [r, max(1, r - 5), max(1, r // 2)]
    run_adapters([1232], [1], H, N, 3, r, 31, rank=rank, pad=pad)
    run_adapters([700, 33, 0, 1265], [0, 2, 1, -1], H, N, 3, r, 32, rank=rank, pad=pad, in_place=True)
    run_adapters([1, 3000, 40, 8, 959, 24, 17], [0, 1, 2, 0, 1, -1, 2], H, N, 3, r, 33, rank=rank, pad=pad, scale=False)
    run_adapters([31, 32, 33, 16, 15, 5000, 1007, 481], [2, 0, 1, 2, 0, 1, 7, 0], H, N, 3, r, 34, pad=pad)
    run_adapters([17 + (7 * i) % 13 for i in range(120)], [i % 4 - 1 for i in range(120)], H, N, 3, r, 35, rank=rank, pad=pad)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("H,N,pad", [(256, 264, 8), (1000, 72, 0)])
def test_adapters_shared_by_short_requests(r, H, N, pad):
    """Tiles that gather an adapter's tokens from many requests: one token each and ragged ones, more of one adapter
    than a tile holds, empty requests, slots out of range, none at all, the most requests the search takes and one more."""
    rank = [r, max(1, r - 3), max(1, r // 2), 0]
    run_adapters([1] * 64, [(i * i) % 5 - 1 for i in range(64)], H, N, 4, r, 41, rank=rank, pad=pad)
    run_adapters([(i * 7) % 12 for i in range(90)], [(i * 3) % 7 - 2 for i in range(90)], H, N, 4, r, 42, rank=rank, in_place=True)
    run_adapters([0, 31, 1, 16, 17] + [1] * 45, [2, 1, 1, 2, 1] + [0, 1, 2] * 15, H, N, 3, r, 43, pad=pad, scale=False)
    run_adapters([1] * 40, [-1] * 40, H, N, 2, r, 44)
    run_adapters([1] * 33, [0] * 33, H, N, 1, r, 45, rank=[r])
    run_adapters([1] * 512, [(i * 11) % 60 for i in range(512)], H, N, 60, r, 46, pad=pad)
    run_adapters([1] * 513, [(i * 11) % 60 for i in range(513)], H, N, 60, r, 47)


@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("R", [33, 40, 50, 90, 100, 257])
def test_gathered_adapters_among_requests_without_one(r, R):
    """Any number of requests, some without an adapter, out of place: every row its own, none outside the batch."""
    H, N, n = 256, 264, 2
    for ragged in (False, True):
        lens = [(i * 7 + R) % 12 for i in range(R)] if ragged else [1] * R
        slot = [-1 if i % 7 == 6 else i % n for i in range(R)]
        g, T = gen(R + r), sum(lens)
        starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
        x, base = rows(T, H, torch.bfloat16, g), rows(T, N, torch.bfloat16, g)
        a = (torch.randn((n, r, H), generator=g, device="cuda") / math.sqrt(H)).bfloat16()
        b = (torch.randn((n, N, r), generator=g, device="cuda") / math.sqrt(r)).bfloat16()
        buf = torch.full((T + 128, N), 7.0, dtype=torch.bfloat16, device="cuda")
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        M.moe_adapters_add(x, base, a, b, i32(starts), i32(slot), out=buf[64:64 + T])
        ref, err = ref_adapters(x, base, a, b, starts, slot, None, None)
        check(buf[64:64 + T], ref, err, f"{R} requests, rank {r}")
        assert (buf[:64] == 7.0).all() and (buf[64 + T:] == 7.0).all()


def test_gathered_adapters_repeat_and_capture():
    """NaN stays in its row among gathered ones, runs repeat, and a captured call follows its inputs."""
    g = gen(51)
    T, H, N, r = 96, 512, 264, 64
    x, base = rows(T, H, torch.bfloat16, g), rows(T, N, torch.bfloat16, g)
    a = torch.randn((3, r, H), generator=g, device="cuda").bfloat16()
    b = torch.randn((3, N, r), generator=g, device="cuda").bfloat16()
    starts = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([(i * 5) % 4 - 1 for i in range(T)], dtype=torch.int32, device="cuda")
    want = M.moe_adapters_add(x, base, a, b, starts, slot)
    assert torch.equal(want, M.moe_adapters_add(x, base, a, b, starts, slot))
    x2 = x.clone()
    x2[17, 3] = float("nan")
    got = M.moe_adapters_add(x2, base, a, b, starts, slot)
    keep = torch.arange(T, device="cuda") != 17
    assert slot[17] >= 0 and torch.isnan(got[17]).all() and torch.equal(got[keep], want[keep])
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(base)
    with torch.cuda.graph(graph):
        M.moe_adapters_add(x, base, a, b, starts, slot, out=out)
    slot.copy_(slot.flip(0))
    graph.replay()
    assert torch.equal(out, M.moe_adapters_add(x, base, a, b, starts, slot))


def test_adapters_first_call_of_a_process():
    """Each kernel and cluster size as the first launch of its process: nothing an earlier call has set up (the
    opt-in to more shared memory) may be needed.  A process per length; every rank class is new to it."""
    import os
    import subprocess
    import sys

    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [{!r}, {!r}]; import test_block_ops as t\n"
            "for r in (8, 24, 40, 128): t.run_adapters([{}], [0], 64, 64, 1, r, 21)\n"
            "for r in (8, 24, 40, 128): t.run_adapters([1] * 40, [0] * 40, 64, 64, 1, r, 22)")
    runs = [subprocess.Popen([sys.executable, "-c", code.format(here, os.path.dirname(here), T)], stdout=subprocess.PIPE,
                             stderr=subprocess.STDOUT, text=True) for T in (16, 464, 944, 1904, 3184)]
    outs = [p.communicate(timeout=300)[0] for p in runs]
    assert all(p.returncode == 0 for p in runs), outs


def test_adapters_many_requests_and_edges():
    # more requests than one pass of the tile search holds, empty ones among them; slots out of range
    lens = [(i * 7) % 4 for i in range(700)]
    slot = [(i * 5) % 9 - 2 for i in range(700)]
    run_adapters(lens, slot, 128, 136, 5, 16, 5, rank=[0, 1, 7, 15, 16])
    run_adapters([3, 2], [-1, -1], 64, 64, 1, 8, 6)
    run_adapters([0, 0, 4], [0, 0, 0], 64, 64, 1, 8, 7, scale=False)
    run_adapters([513] * 3 + [0, 1], [0, 1, 0, 1, 1], 128, 256, 2, 40, 8, rank=[39, 37])
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    a, b = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 64, 8), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert M.moe_adapters_add(x, x, a, b, z, z[:0]).shape == (0, 64)


def test_adapters_nan_stays_in_its_row_and_runs_repeat():
    g = gen(9)
    x, base = rows(600, 256, torch.bfloat16, g), rows(600, 256, torch.bfloat16, g)
    a = torch.randn((1, 16, 256), generator=g, device="cuda").bfloat16()
    b = torch.randn((1, 256, 16), generator=g, device="cuda").bfloat16()
    for lens in ([600], [3, 500, 1, 96], [300, 300]):
        starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        slot = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        want = M.moe_adapters_add(x, base, a, b, starts, slot)
        assert torch.equal(want, M.moe_adapters_add(x, base, a, b, starts, slot))
        x2 = x.clone()
        x2[77, 5] = float("nan")
        x2[300, 255] = float("inf")
        got = M.moe_adapters_add(x2, base, a, b, starts, slot)
        keep = torch.ones(600, dtype=torch.bool, device="cuda")
        keep[77] = keep[300] = False
        assert torch.equal(got[keep], want[keep])
        assert torch.isnan(got[77]).all() and not torch.isfinite(got[300]).any()
    # the same in tiles of 128 tokens, where neighbours share one product
    x, base = rows(4096, 1024, torch.bfloat16, g), rows(4096, 1024, torch.bfloat16, g)
    a = torch.randn((2, 128, 1024), generator=g, device="cuda").bfloat16()
    b = torch.randn((2, 1024, 128), generator=g, device="cuda").bfloat16()
    starts, slot = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1000, 4096], [1, 0]))
    want = M.moe_adapters_add(x, base, a, b, starts, slot)
    assert torch.equal(want, M.moe_adapters_add(x, base, a, b, starts, slot))
    x[999, 5] = float("nan")
    got = M.moe_adapters_add(x, base, a, b, starts, slot)
    assert torch.isnan(got[999]).all() and torch.equal(got[:999], want[:999]) and torch.equal(got[1000:], want[1000:])
    assert M.moe_get_adapter_error() == 0


@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_no_adapters_at_all(r):
    """n = 0: every request is one without an adapter, at any size."""
    H, N = 2048, 2048
    for lens in ([1], [1] * 40, [3, 0, 50], [4096, 4096], [500] * 33):
        g, T, R = gen(r), sum(lens), len(lens)
        x, base = rows(T, H, torch.bfloat16, g), rows(T, N, torch.bfloat16, g)
        a = torch.empty((0, r, H), dtype=torch.bfloat16, device="cuda")
        b = torch.empty((0, N, r), dtype=torch.bfloat16, device="cuda")
        starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        slot = torch.tensor([i % 3 - 1 for i in range(R)], dtype=torch.int32, device="cuda")
        assert torch.equal(M.moe_adapters_add(x, base, a, b, starts, slot), base)


@pytest.mark.parametrize("lens,r", [([4], 8), ([4], 64), ([4], 128), ([1] * 40, 16), ([1] * 40, 64), ([400, 800], 16),
                                    ([9000, 7000], 16), ([2000, 2000], 32), ([4096, 4096], 64), ([4096, 4096], 128), ([3000, 100], 128)])
def test_adapters_keep_infinities(lens, r):
    """A x infinite, or past bf16's largest value: what fp32 gives, not NaN; the other rows as they are."""
    H, N, T = 1024, 1536, sum(lens)
    g = gen(r)
    x, base = rows(T, H, torch.bfloat16, g), rows(T, N, torch.bfloat16, g)
    a, b = torch.ones((2, r, H), dtype=torch.bfloat16, device="cuda"), torch.randn((2, N, r), generator=g, device="cuda").bfloat16()
    a[:, :, 1] = 0.0
    a[:, 0, 1] = 2.0 ** -20
    a[:, 1:, 0] = -1.0
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts, slot = i32(np.concatenate([[0], np.cumsum(lens)])), i32([i % 2 for i in range(len(lens))])
    s = int(np.repeat(np.arange(len(lens)) % 2, lens)[T // 2])  # the changed row's adapter
    for rank in (1, r):  # alone: its sign.  All: infinities of both signs, NaN
        args = dict(scale=torch.full((2,), 1.0035, device="cuda"), rank=i32([rank, rank]))
        want = M.moe_adapters_add(x, base, a, b, starts, slot, **args)
        assert torch.isfinite(want).all()
        y = x.clone()
        y[T // 2, 0] = float("inf")
        got = M.moe_adapters_add(y, base, a, b, starts, slot, **args)
        keep = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(got[keep], want[keep])
        ref = (float("inf") * b[s, :, 0].float()).bfloat16()
        if rank == 1:
            assert torch.equal(got[T // 2].isnan(), ref.isnan()) and torch.equal(got[T // 2].nan_to_num(7.0), ref.nan_to_num(7.0))
        else:
            assert not torch.isfinite(got[T // 2]).any()
    # finite, but bf16's rounding alone would make it infinite
    top = torch.finfo(torch.bfloat16).max
    y = x.clone()
    y[T // 2] = 0.0
    y[T // 2, 2] = top
    args = dict(scale=torch.full((2,), 1.0035, device="cuda"), rank=i32([1, 1]))
    bt = b * 2.0 ** -120
    got = M.moe_adapters_add(y, base, a, bt, starts, slot, **args)[T // 2].double()
    exact = base[T // 2].double() + float(np.float32(1.0035)) * top * bt[s, :, 0].double()
    assert ((got - exact).abs() <= exact.abs() * 2.0 ** -8 + base[T // 2].double().abs() * 2.0 ** -20 + (exact - base[T // 2].double()).abs() * 2.0 ** -16).all()


@pytest.mark.parametrize("lens,r", [([4], 8), ([4], 64), ([4], 128), ([1] * 40, 16), ([1] * 40, 64), ([400, 800], 16),
                                    ([9000, 7000], 16), ([2000, 2000], 32), ([4096, 4096], 64), ([4096, 4096], 128), ([3000, 100], 128)])
def test_adapters_hold_all_bits_of_the_inner_product(lens, r):
    """A x of 23 bits, and outputs that are differences of two of them: whole numbers, exact in fp32 from end to end."""
    H, N, T = 1024, 1536, sum(lens)
    g = gen(r + 1)
    x = torch.zeros((T, H), device="cuda")
    x[:, :64] = torch.randint(1, 256, (T, 64), generator=g, device="cuda").float()
    a = torch.zeros((2, r, H), device="cuda")
    a[:, 0::2, 0], a[:, 0::2, 1], a[:, 0::2, 2] = 2.0 ** 14, 2.0 ** 7, 1.0  # 22 bits
    a[:, 1::2, 0], a[:, 1::2, 1] = 2.0 ** 14, 2.0 ** 7  # the same without the last
    b = torch.zeros((2, N, r), device="cuda")
    n = torch.arange(N, device="cuda")
    b[:, n, n % (r // 2) * 2], b[:, n, n % (r // 2) * 2 + 1] = 1.0, -1.0
    base = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts, slot = i32(np.concatenate([[0], np.cumsum(lens)])), i32([i % 2 for i in range(len(lens))])
    got = M.moe_adapters_add(x.bfloat16(), base, a.bfloat16(), b.bfloat16(), starts, slot)
    assert torch.equal(got, x[:, 2:3].bfloat16().expand(T, N))


def test_adapters_without_requests():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    a, b = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 64, 8), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    refused(1, M.moe_adapters_add, x, x, a, b, z, z[:0])  # four tokens of no request: nothing would write them
    assert M.moe_adapters_add(x[:0], x[:0], a, b, z, z[:0]).shape == (0, 64)


# ------------------------------------------------------------------------------------------ together
def bf16_experts(E, H, I, g):
    wgu = (0.05 * torch.randn((E, 2 * I, H), generator=g, device="cuda")).bfloat16()
    wd = (0.05 * torch.randn((E, H, I), generator=g, device="cuda")).bfloat16()
    return wgu, wd


def ref_layer(x, idx, w, wgu, wd):
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    I = wd.shape[2]
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            h = wgu[e].double() @ x[t].double()
            h = torch.nn.functional.silu(h[:I]) * h[I:]
            out[t] += float(w[t, j]) * (wd[e].double() @ h)
    return out


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4", "nvfp4_w4a16", "nvfp4_w4a4", "fp8_w8a8"])
def test_layer_forward_scored_default_is_layer_forward(fmt):
    g = gen(11)
    E, H, I, k = 16, 256, 128, 4
    wgu, wd = bf16_experts(E, H, I, g)
    layer = M.MoELayer(fmt, wgu, wd)
    for T in (0, 1, 30, 300):
        x, lg = rows(T, H, torch.bfloat16, g).contiguous(), rows(T, E, torch.float32, g).contiguous()
        want = layer.forward(x, lg, k)
        got = torch.empty_like(x)
        M.moe_layer_forward_scored(x, lg, M.Router(), layer.desc, layer.packed, k, got, layer.workspace)
        # the same experts and weights within expf's rounding, so sums of bf16 rows within one rounding each
        if T:
            assert (got.double() - want.double()).norm() <= 2.0 ** -8 * want.double().norm()
            assert M.moe_get_device_error(layer.workspace) == 0


@pytest.mark.parametrize("T", [1, 7, 150])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_layer_forward_scored(T, score):
    g = gen(T)
    E, H, I, k = 32, 256, 128, 4
    wgu, wd = bf16_experts(E, H, I, g)
    layer = M.MoELayer("bf16", wgu, wd)
    x = rows(T, H, torch.bfloat16, g).contiguous()
    lg = rows(T, E, torch.bfloat16, g, pad=8)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    r = M.Router(score, groups=4, top_groups=2, group_top=2, renormalize=score == "sigmoid", scale=2.5)
    out = torch.empty_like(x)
    M.moe_layer_forward_scored(x, lg, r, layer.desc, layer.packed, k, out, layer.ensure_workspace(T, k), bias=bias)
    idx, w = M.moe_route_scored(lg, r, k, bias=bias)
    ref = ref_layer(x, idx.cpu(), w.cpu(), wgu, wd)
    d = out.double() - ref
    assert d.norm() <= 1e-2 * ref.norm() and d.abs().max() <= 2e-2 * ref.abs().max()


@pytest.mark.parametrize("T,stream_type", [(1, "bf16"), (9, "f32"), (200, "f32")])
def test_moe_block(T, stream_type):
    """The whole block against its formula in 64 bits (given the experts it chose: bf16 router logits tie)."""
    g = gen(T + 50)
    E, H, I, k, n, r = 16, 256, 128, 4, 3, 16
    wgu, wd = bf16_experts(E, H, I, g)
    (pre, ps), (post, qs), (nxt, ns) = (make_norm("rms", H, torch.bfloat16, g, bias=False) for _ in range(3))
    router = M.Router("sigmoid", groups=4, top_groups=2, group_top=2, scale=2.5)
    wr = (torch.randn((E, H), generator=g, device="cuda") / 16).bfloat16()
    block = M.MoEBlock(M.MoELayer("bf16", wgu, wd), wr, router, k, pre, post, beta=0.5)
    x = rows(T, H, DT[stream_type], g)
    cut = T // 3
    ad = dict(a=(torch.randn((n, r, H), generator=g, device="cuda") / 16).bfloat16(),
              b=(torch.randn((n, H, r), generator=g, device="cuda") / 4).bfloat16(),
              starts=torch.tensor([0, cut, T], dtype=torch.int32, device="cuda"),
              slot=torch.tensor([-1, 2], dtype=torch.int32, device="cuda"))
    gate = torch.randn((T, 1), generator=g, device="cuda")
    out, y = block.forward(x, adapters=ad, gate=gate, gate_act="sigmoid", next=nxt)
    z = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    h = ref_norm(x.double(), z, *ps)[0]
    hb = M.moe_block_enter(x, pre, dtype=torch.bfloat16)
    idx, w = M.moe_route_scored(hb @ wr.t(), router, k)
    m = ref_layer(h, idx.cpu(), w.cpu(), wgu, wd)
    m = ref_adapters(h, m, ad["a"], ad["b"], [0, cut, T], [-1, 2], None, None)[0]
    o = x.double() + 0.5 * torch.sigmoid(gate.double()) * ref_norm(m, z, *qs)[0]
    ry = ref_norm(o, z, *ns)[0]
    for got, ref in ((out, o), (y, ry)):
        assert (got.double() - ref).norm() <= 1e-2 * ref.norm()
    # the next block starts from y: nothing is normed twice
    again = block.forward(x, h=hb, adapters=ad, gate=gate, gate_act="sigmoid")
    assert torch.equal(again, out)


def test_example_runs():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    x = example.main(["--format", "fp8", "--hidden", "256", "--inner", "128", "--experts", "16", "--top-k", "4", "--steps", "1"])
    assert x.shape == (5, 256) and torch.isfinite(x).all()


def test_operators_in_a_graph():
    """Captured once, replayed on new inputs: the same results as direct calls."""
    g = gen(21)
    T, H, E, r = 4000, 1024, 64, 128
    x, b = rows(T, H, torch.float32, g), rows(T, H, torch.bfloat16, g)
    (pre, _), (post, _) = make_norm("rms", H, torch.bfloat16, g), make_norm("layer", H, torch.bfloat16, g)
    lg = rows(T, E, torch.float32, g)
    router = M.Router("sigmoid", groups=8, top_groups=4, group_top=2)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    A = torch.randn((2, r, H), generator=g, device="cuda").bfloat16()
    B = torch.randn((2, H, r), generator=g, device="cuda").bfloat16()
    starts, slot = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1000, 4000], [1, 0]))

    def work():
        h = M.moe_block_enter(x, pre, dtype=torch.bfloat16)
        idx, w = M.moe_route_scored(lg, router, 4, bias=bias)
        m = M.moe_adapters_add(h, b, A, B, starts, slot)
        few = M.moe_adapters_add(h[:64], b[:64], A, B, starts.clamp(max=64), slot)
        return (idx, w, m, few) + M.moe_block_leave(x, m, post=post, next=pre)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for t in (x, b, lg):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    graph.replay()
    for p, q in zip(got, work()):
        assert torch.equal(p, q)


# ------------------------------------------------------------------------------------------ refusals
def refused(status, f, *args, **kw):
    with pytest.raises(M.MoEError) as e:
        f(*args, **kw)
    assert e.value.status == status


def test_refusals():
    g = gen(1)
    x = rows(4, 64, torch.bfloat16, g)
    n = M.Norm("rms", torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    refused(1, M.moe_block_enter, x.cpu(), n)
    refused(1, M.moe_block_enter, x.t(), n)
    refused(1, M.moe_block_enter, x[0], n)
    refused(1, M.moe_block_enter, x[:, :32], n)  # the norm's parameters are longer
    refused(1, M.moe_block_enter, x, n, dtype=torch.int8)
    refused(1, M.moe_block_enter, x.to(torch.int16), n)
    refused(2, M.moe_block_enter, x, n, dtype=torch.float32)  # a narrow stream, wide output
    refused(1, M.moe_block_enter, x, n, out=torch.empty((4, 63), dtype=torch.bfloat16, device="cuda"))
    refused(1, M.moe_block_enter, torch.as_strided(x, (2, 64), (8, 1)), n)
    refused(1, M.Norm, "batch")
    refused(1, M.Norm, "rms", eps=0.0)
    refused(1, M.Norm, "rms", torch.ones(4, device="cuda"), torch.ones(5, device="cuda"))
    refused(1, M.moe_block_leave, x, x[:3])
    refused(2, M.moe_block_leave, x, x.half())
    refused(1, M.moe_block_leave, x, x, gate=torch.ones(63, device="cuda"))
    refused(1, M.moe_block_leave, x, x, gate=torch.ones(64, device="cuda"), gate_act="relu")
    refused(1, M.moe_block_leave, x, x, next=n, y=torch.empty((4, 64), device="cuda"))
    lg = rows(4, 64, torch.float32, g)
    refused(1, M.Router, "relu")
    for bad in (dict(groups=3), dict(groups=0), dict(groups=64), dict(groups=8, top_groups=9), dict(groups=8, top_groups=0),
                dict(group_top=3), dict(scale=float("nan"))):
        refused(1, M.moe_route_scored, lg, M.Router("sigmoid", **bad), 4)
    refused(1, M.moe_route_scored, lg, M.Router("sigmoid", groups=32, top_groups=2), 5)  # 4 candidates
    refused(1, M.moe_route_scored, lg, M.Router(), 9)
    refused(1, M.moe_route_scored, lg, M.Router(), 0)
    refused(1, M.moe_route_scored, lg[:, :4], M.Router(), 5)
    refused(1, M.moe_route_scored, rows(2, 257, torch.float32, g), M.Router(), 4)
    refused(1, M.moe_route_scored, lg, M.Router(), 4, bias=torch.zeros(64, dtype=torch.bfloat16, device="cuda"))
    refused(1, M.moe_route_scored, lg, M.Router(), 4, topk_idx=torch.empty((4, 4), dtype=torch.int64, device="cuda"))
    a, b = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 64, 8), dtype=torch.bfloat16, device="cuda")
    st, sl = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 4], [0]))
    M.moe_adapters_add(x, x, a, b, st, sl)
    refused(1, M.moe_adapters_add, x.half(), x, a, b, st, sl)
    refused(1, M.moe_adapters_add, x, x[:, :32], a, b, st, sl)
    refused(1, M.moe_adapters_add, x, x, a[:, :4], b, st, sl)
    refused(1, M.moe_adapters_add, x, x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), st, sl)  # rank 4
    refused(1, M.moe_adapters_add, x, x, a, b, st.long(), sl)
    refused(1, M.moe_adapters_add, x, x, a, b, sl, sl)
    refused(1, M.moe_adapters_add, x, x, a, b, st, sl, scale=torch.ones(3, device="cuda"))
    refused(1, M.moe_adapters_add, x, x, a, b, st, sl, rank=torch.ones(2, device="cuda"))
    off = torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda")
    refused(1, M.moe_adapters_add, off[:, 4:68], x, a, b, st, sl)  # rows not on 16-byte boundaries
