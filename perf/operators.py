"""The operators around a layer of quantized experts, as cases to measure.

A block of a mixture-of-experts model runs, per token: a norm of the residual stream, the router's
choice of experts, the experts, the low-rank adapter of the token's request added to the layer's
output, and the way back into the stream (norm of the block's output, gate, residual scales) with
the next block's norm.  The cases cover the three operators around the experts:

  enter / leave   nvfp4_expert_gemms_gb300.moe_block_enter / moe_block_leave
  route           nvfp4_expert_gemms_gb300.moe_route_scored
  adapt           nvfp4_expert_gemms_gb300.moe_adapters_add

With `own` false, run() computes them from elementary torch operations in fp32.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
ALPHA, BETA = 1.0, 0.22  # residual scales: the stream's and the block's


def enter(name, T, H, stream="bf16", act="bf16", kind="rms", pad=0):
    return {"name": name, "op": "enter", "T": T, "H": H, "stream": stream, "act": act, "kind": kind, "pad": pad}


def leave(name, T, H, stream="bf16", act="bf16", kind="rms", gate="none", gate_act="none", next=True, pad=0):
    return {"name": name, "op": "leave", "T": T, "H": H, "stream": stream, "act": act, "kind": kind, "gate": gate,
            "gate_act": gate_act, "next": next, "pad": pad}


def route(name, T, E, k, score, bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, logits="f32"):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "group_top": group_top, "renorm": renorm, "scale": scale, "logits": logits}


def adapt(name, T, requests, H, N, slots, rank, mix=0, mixed_ranks=False, none_every=0):
    return {"name": name, "op": "adapt", "T": T, "requests": requests, "H": H, "N": N, "slots": slots, "rank": rank,
            "mix": mix, "mixed_ranks": mixed_ranks, "none_every": none_every}


def listed():
    return [
        # one token of one request: the norm in front of the router and the experts, at decode
        enter("enter_decode_1", 1, 2048),
        # a decode step of 256 requests: back into the stream, gated per token (the sigmoid gate of an
        # always-active expert), with the next block's norm in the same pass
        leave("leave_decode_256", 256, 2048, gate="token", gate_act="sigmoid"),
        # a 16k-token prefill with the stream kept in fp32: norm after the block, a gate per channel,
        # residual scales, norm before the next block
        leave("leave_prefill_16384", 16384, 2048, stream="f32", gate="channel"),
        # rows of odd length with padded row strides, fp16, layer norms with biases, a gate per element
        leave("leave_odd_layer", 1237, 1999, stream="f16", act="f16", kind="layer", gate="full", gate_act="tanh", pad=6),
        # one token: sigmoid scores, a balance bias, 4 of 8 groups
        route("route_decode_1", 1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # a 4096-token batch, softmax router over 128 experts, all groups
        route("route_softmax_4096", 4096, 128, 8, "softmax"),
        # a 16k-token prefill, sigmoid scores, bias, groups
        route("route_prefill_16384", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # ragged expert count, bf16 logits (a bf16 router product: many ties), best expert per group,
        # weights left as they are
        route("route_odd_60", 5003, 60, 4, "softmax", False, 6, 3, 1, False, 16.0, "bf16"),
        # one token of one request with its adapter
        adapt("adapt_decode_1", 1, 1, 2048, 2048, 4, 16),
        # a decode step of 64 requests over 32 adapters of mixed rank, some requests without one
        adapt("adapt_decode_64", 64, 64, 2048, 2048, 32, 32, 1, True, 7),
        # a mixed step: 37 requests of uneven length (decodes and prefills together), a projection
        # of the experts' fused gate/up width
        adapt("adapt_ragged_4001", 4001, 37, 2048, 1536, 12, 16, 2, True, 5),
        # a 16k-token prefill of 16 requests, rank 64
        adapt("adapt_prefill_16384", 16384, 16, 2048, 2048, 16, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _length(rng, lo, hi):
    n = _log(rng, lo, hi)
    return n - 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(["enter", "leave", "leave", "route", "route", "adapt", "adapt"])
    if op in ("enter", "leave"):
        T = _log(rng, 1, 16384)
        H = _length(rng, 64, min(8192, max(65, 2048 * 16384 // T)))
        if rng.random() < 0.7:
            H = max(64, H // 64 * 64)
            H = 2944 if H == 3072 else H
        stream, act = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f16"), ("f32", "f32")])
        kind, pad = rng.choice(["rms", "rms", "layer"]), rng.choice([0, 0, 8, 13])
        if op == "enter":
            c = enter("", T, H, stream, act, kind, pad)
        else:
            g = rng.choice(["none", "token", "channel", "full"])
            c = leave("", T, H, stream, act, kind, g, rng.choice(["none", "sigmoid", "tanh"]) if g != "none" else "none",
                      rng.random() < 0.7, pad)
    elif op == "route":
        T = _log(rng, 1, 16384)
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(max(2, 8 // groups), 256 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(8, per * top_groups))
        score = rng.choice(["softmax", "sigmoid"])
        c = route("", T, groups * per, k, score, score == "sigmoid" and rng.random() < 0.7, groups, top_groups,
                  rng.randint(1, 2), rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]), rng.choice(["f32", "f32", "bf16", "f16"]))
    else:
        T = _log(rng, 1, 16384)
        requests = _log(rng, 1, min(T, 256))
        H, N = 8 * _log(rng, 16, 256), 8 * _log(rng, 16, 256)
        c = adapt("", T, requests, H, N, _log(rng, 1, 64), 8 * rng.randint(1, 8), rng.randrange(1 << 20), rng.random() < 0.5,
                  rng.choice([0, 0, 3, 9]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------- inputs
def _requests(case):
    """Request lengths, adapter slots (-1: none) and each slot's rank: the same for every seed."""
    T, R, n, rank = case["T"], case["requests"], case["slots"], case["rank"]
    r = random.Random(case["mix"])
    if case["mix"] == 0 or R == T:  # even lengths
        cuts = [T * i // R for i in range(R + 1)]
    else:  # uneven: a few tokens to most of the batch, empty requests among them
        share = [r.lognormvariate(0.0, 2.0) for _ in range(R)]
        run, cuts = 0.0, [0]
        for s in share:
            run += s
            cuts.append(min(T, int(T * run / sum(share))))
        cuts[-1] = T
    slot = [i % n if case["mix"] == 0 else r.randrange(n) for i in range(R)]
    if case["none_every"]:
        slot = [-1 if i % case["none_every"] == case["none_every"] - 1 else s for i, s in enumerate(slot)]
    ranks = [r.randint(1, rank) if case["mixed_ranks"] else rank for _ in range(n)]
    return cuts, slot, ranks


def _row(shape, pad, dtype):
    """An uninitialised [T, H] view whose rows lie `pad` elements further apart than H."""
    return torch.empty((shape[0], shape[1] + pad), dtype=dtype, device="cuda")[:, :shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] in ("enter", "leave"):
        T, H, pad = case["T"], case["H"], case["pad"]
        stream, act = DTYPES[case["stream"]], DTYPES[case["act"]]
        channel = torch.exp(0.8 * normal(H))  # a few channels carry most of a stream's energy
        s["x"] = _row((T, H), pad, stream).copy_(normal(T, H) * channel * torch.exp(0.5 * normal(T, 1)))
        norms = ["norm"] if case["op"] == "enter" else ["post", "next"] if case["next"] else ["post"]
        for n in norms:
            s[n + "_w"] = (1.0 + 0.2 * normal(H)).to(act)
            s[n + "_b"] = (0.1 * normal(H)).to(act) if case["kind"] == "layer" else None
        if case["op"] == "leave":
            s["block"] = _row((T, H), pad, act).copy_(0.3 * normal(T, H))
            shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[case["gate"]]
            s["gate"] = None if shape is None else normal(*shape).to(act)
        if own:
            import nvfp4_expert_gemms_gb300 as M

            for n in norms:
                s[n] = M.Norm(case["kind"], s[n + "_w"], s[n + "_b"], eps=EPS)
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        popular = -0.6 * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda"))
        s["logits"] = (1.2 * normal(T, E) + popular).to(DTYPES[case["logits"]])
        s["bias"] = 0.05 * normal(E) - 0.1 * popular if case["bias"] else None
        if own:
            import nvfp4_expert_gemms_gb300 as M

            s["router"] = M.Router(case["score"], groups=case["groups"], top_groups=case["top_groups"],
                                   group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"])
    else:
        T, H, N, n, rank = case["T"], case["H"], case["N"], case["slots"], case["rank"]
        cuts, slot, ranks = _requests(case)
        s["x"], s["base"] = normal(T, H).bfloat16(), normal(T, N).bfloat16()
        s["a"] = (normal(n, rank, H) / math.sqrt(H)).bfloat16()
        s["b"] = (normal(n, N, rank) / math.sqrt(rank)).bfloat16()
        s["scale"] = 0.5 + 1.5 * torch.rand(n, generator=g, device="cuda")
        s["starts"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        s["slot"] = torch.tensor(slot, dtype=torch.int32, device="cuda")
        s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _norm(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()
    return v if b is None else v + b.float()


def _plain_enter(s):
    c = s["case"]
    return _norm(s["x"].float(), c["kind"], s["norm_w"], s["norm_b"]).to(DTYPES[c["act"]])


def _plain_leave(s):
    c = s["case"]
    v = _norm(s["block"].float(), c["kind"], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        gate = s["gate"].float()
        v = v * {"none": lambda t: t, "sigmoid": lambda t: 1.0 / (1.0 + torch.exp(-t)), "tanh": torch.tanh}[c["gate_act"]](gate)
    out = ALPHA * s["x"].float() + BETA * v
    if not c["next"]:
        return out.to(s["x"].dtype)
    return out.to(s["x"].dtype), _norm(out, c["kind"], s["next_w"], s["next_b"]).to(DTYPES[c["act"]])


def _plain_route(s):
    c, logits = s["case"], s["logits"].float()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(-1, keepdim=True))  # over their sum below
    key = logits if s["bias"] is None else score + s["bias"]  # without a bias the logits have the scores' order
    if c["groups"] > 1:
        per = c["E"] // c["groups"]
        member = (score if s["bias"] is None and c["group_top"] == 2 else key).view(-1, c["groups"], per)
        best = torch.sort(member, dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        key = key.masked_fill(~mask.repeat_interleave(per, dim=1), -math.inf)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    elif c["score"] == "softmax":
        w = w / score.sum(-1, keepdim=True)
    return idx.int(), w * c["scale"]


def _plain_adapt(s):
    c = s["case"]
    T, N, n, rank = c["T"], c["N"], c["slots"], c["rank"]
    slot = torch.repeat_interleave(s["slot"], s["starts"].diff(), output_size=T)  # each token's adapter
    ids = torch.arange(n, device="cuda")
    live = (torch.arange(rank, device="cuda") < s["ranks"][:, None]).float() * s["scale"][:, None]  # [n, rank]
    v = s["x"].float() @ s["a"].view(n * rank, -1).float().t()  # every adapter's inner products
    v = v.view(T, n, rank) * (slot[:, None] == ids).float()[..., None] * live  # its own stay
    return (s["base"].float() + v.view(T, n * rank) @ s["b"].transpose(1, 2).reshape(n * rank, N).float()).bfloat16()


def run(s):
    c = s["case"]
    if not own:
        return {"enter": _plain_enter, "leave": _plain_leave, "route": _plain_route, "adapt": _plain_adapt}[c["op"]](s)
    import nvfp4_expert_gemms_gb300 as M

    if c["op"] == "enter":
        return M.moe_block_enter(s["x"], s["norm"], dtype=DTYPES[c["act"]])
    if c["op"] == "leave":
        return M.moe_block_leave(s["x"], s["block"], post=s["post"], gate=s["gate"], gate_act=c["gate_act"], alpha=ALPHA,
                                 beta=BETA, next=s["next"] if c["next"] else None)
    if c["op"] == "route":
        return M.moe_route_scored(s["logits"], s["router"], c["k"], bias=s["bias"])
    return M.moe_adapters_add(s["x"], s["base"], s["a"], s["b"], s["starts"], s["slot"], scale=s["scale"], rank=s["ranks"])


# ---------------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    T = case["T"]
    if case["op"] in ("enter", "leave"):
        H, st, ac = case["H"], SIZE[case["stream"]], SIZE[case["act"]]
        par = ac * H * (2 if case["kind"] == "layer" else 1)
        if case["op"] == "enter":
            return {"bytes": T * H * (st + ac) + par, "flops": 6 * T * H}
        gate = {"none": 0, "token": T, "channel": H, "full": T * H}[case["gate"]] * ac
        nxt = 1 if case["next"] else 0
        return {"bytes": T * H * (2 * st + ac * (1 + nxt)) + gate + par * (1 + nxt), "flops": (9 + 6 * nxt) * T * H}
    if case["op"] == "route":
        E = case["E"]
        return {"bytes": T * E * SIZE[case["logits"]] + 8 * T * case["k"] + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    H, N = case["H"], case["N"]
    cuts, slot, ranks = _requests(case)
    used = {s for i, s in enumerate(slot) if s >= 0 and cuts[i + 1] > cuts[i]}
    flops = sum(2 * (cuts[i + 1] - cuts[i]) * ranks[s] * (H + N) for i, s in enumerate(slot) if s >= 0)
    rows = sum(cuts[i + 1] - cuts[i] for i, s in enumerate(slot) if s >= 0)
    return {"bytes": 2 * rows * H + 4 * T * N + sum(2 * ranks[s] * (H + N) for s in used) + 4 * (2 * len(slot) + 1), "flops": flops + T * N}


# ---------------------------------------------------------------------------------------- the definitions in 64 bits
def _f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _exact_norm(v, kind, w, b):
    mean = v.sum(axis=1, keepdims=True) / v.shape[1] if kind == "layer" else 0.0
    power = ((v - mean) ** 2).sum(axis=1, keepdims=True) / v.shape[1]
    y = (v - mean) / np.sqrt(power + EPS) * w
    return y if b is None else y + b


def _exact_route(c, logits, bias):
    idx, w = np.zeros((c["T"], c["k"]), np.int32), np.zeros((c["T"], c["k"]))
    per = c["E"] // c["groups"]
    for t in range(c["T"]):
        l = logits[t]
        p = 1.0 / (1.0 + np.exp(-l)) if c["score"] == "sigmoid" else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        key = p + bias if bias is not None else l
        if c["groups"] > 1:
            by = (p if bias is None and c["group_top"] == 2 else key).reshape(c["groups"], per)
            best = np.sort(by, axis=1)[:, ::-1][:, :c["group_top"]].sum(axis=1)
            allowed = np.zeros(c["groups"], bool)
            allowed[np.argsort(-best, kind="stable")[:c["top_groups"]]] = True
            key = np.where(np.repeat(allowed, per), key, -np.inf)
        order = np.argsort(-key, kind="stable")[:c["k"]]
        idx[t], w[t] = order, p[order] / (p[order].sum() if c["renorm"] else 1.0) * c["scale"]
    return idx, w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "enter":
        return _exact_norm(_f64(s["x"]), case["kind"], _f64(s["norm_w"]), _f64(s["norm_b"]))
    if case["op"] == "leave":
        v = _exact_norm(_f64(s["block"]), case["kind"], _f64(s["post_w"]), _f64(s["post_b"]))
        if s["gate"] is not None:
            gate = _f64(s["gate"])
            v *= np.tanh(gate) if case["gate_act"] == "tanh" else 1.0 / (1.0 + np.exp(-gate)) if case["gate_act"] == "sigmoid" else gate
        out = ALPHA * _f64(s["x"]) + BETA * v
        return (out, _exact_norm(out, case["kind"], _f64(s["next_w"]), _f64(s["next_b"]))) if case["next"] else out
    if case["op"] == "route":
        return _exact_route(case, _f64(s["logits"]), _f64(s["bias"]))
    cuts, slot, ranks = _requests(case)
    x, out, scale = _f64(s["x"]), _f64(s["base"]), _f64(s["scale"])
    for i, k in enumerate(slot):
        if k >= 0:
            rows = slice(cuts[i], cuts[i + 1])
            a, b = _f64(s["a"][k, :ranks[k]]), _f64(s["b"][k, :, :ranks[k]])
            out[rows] += scale[k] * ((x[rows] @ a.T) @ b.T)
    return out
