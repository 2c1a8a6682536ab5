"""Two mixture-of-experts blocks of a serving loop on one GPU: a ragged prefill, then decode steps.

Each block: norm -> router (sigmoid scores, balance bias, expert groups) -> quantized experts, with the
low-rank adapter of each request added -> norm, sigmoid gate per token and residual scale back into an
fp32 stream, with the following block's norm in the same pass.  Weights are random.

    python examples/moe_block.py [--format nvfp4_w4a16] [--hidden 2048] [--experts 64] [--few]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_expert_gemms_gb300 as M  # noqa: E402


def fp8_weight(N, K, g):
    """A random weight in the FP8 block format: E4M3 codes and a scale per 128 x 128 block."""
    w = torch.randn((N, K), generator=g, device="cuda")
    scale = torch.full(((N + 127) // 128, (K + 127) // 128), 1.0 / (100.0 * K ** 0.5), device="cuda")
    return M.Fp8Weight((100.0 * w).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale)


def make_block(fmt, E, H, I, k, g, few=False):
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    layer = M.MoELayer(fmt, (rnd(E, 2 * I, H) / H ** 0.5).bfloat16(), (rnd(E, H, I) / I ** 0.5).bfloat16())
    router = M.Router("sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5)
    norm = lambda: M.Norm("rms", (1.0 + 0.1 * rnd(H)).bfloat16())  # noqa: E731
    # --few: decode steps through one call per layer, and an always-active FP8 expert beside the routed ones
    extra = {"few_tokens": 32, "shared": (fp8_weight(2 * I, H, g), fp8_weight(H, I, g))} if few else {}
    return M.MoEBlock(layer, (rnd(E, H) / H ** 0.5).bfloat16(), router, k, norm(), norm(), 0.02 * rnd(E), beta=0.5, **extra)


def make_adapters(n, r, H, g):
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return {"a": (rnd(n, r, H) / H ** 0.5).bfloat16(), "b": (0.1 * rnd(n, H, r)).bfloat16(),
            "scale": torch.full((n,), 2.0, device="cuda"),
            "rank": torch.tensor([r if i % 2 else r // 2 for i in range(n)], dtype=torch.int32, device="cuda")}


def step(blocks, adapters, lengths, slots, x):
    """One step over a ragged batch: x [sum(lengths), H] fp32 in, the stream and the last norm's output back."""
    cuts = [0]
    for n in lengths:
        cuts.append(cuts[-1] + n)
    batch = {"starts": torch.tensor(cuts, dtype=torch.int32, device="cuda"),
             "slot": torch.tensor(slots, dtype=torch.int32, device="cuda")}
    gate = torch.zeros((x.shape[0], 1), dtype=torch.bfloat16, device="cuda")
    h = None
    for i, (b, ad) in enumerate(zip(blocks, adapters)):
        following = blocks[(i + 1) % len(blocks)].pre
        x, h = b.forward(x, h=h, adapters={**ad, **batch}, gate=gate, gate_act="sigmoid", next=following)
    return x, h


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--format", default="nvfp4_w4a16", choices=sorted(M.FORMATS))
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=768)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--steps", type=int, default=3)
    p.add_argument("--few", action="store_true", help="decode through moe_layer_few, with an always-active FP8 expert")
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    blocks = [make_block(a.format, a.experts, a.hidden, a.inner, a.top_k, g, a.few) for _ in range(2)]
    adapters = [make_adapters(4, 16, a.hidden, g) for _ in range(2)]
    slots = [0, -1, 3, 1, 1]  # the requests' adapters; the second has none
    lengths = [37, 5, 300, 1, 128]
    x, h = step(blocks, adapters, lengths, slots, torch.randn((sum(lengths), a.hidden), generator=g, device="cuda"))
    print(f"prefill of {sum(lengths)} tokens: stream {tuple(x.shape)} rms {x.square().mean().sqrt().item():.3f}")
    last = torch.tensor([sum(lengths[:i + 1]) - 1 for i in range(len(lengths))], device="cuda")
    x = x[last]
    for i in range(a.steps):
        x, h = step(blocks, adapters, [1] * len(slots), slots, x)
        print(f"decode {i}: rms {x.square().mean().sqrt().item():.3f}, next input {tuple(h.shape)} {h.dtype}")
    for b in blocks:
        for w in (b.layer.workspace, b.few_workspace):
            if w is not None and M.moe_get_device_error(w):
                raise RuntimeError("device error flag set")
    if M.moe_get_adapter_error():
        raise RuntimeError("adapter error flag set")
    if M.moe_get_fp8_linear_error():
        raise RuntimeError("product error flag set")
    if not torch.isfinite(x).all():
        raise RuntimeError("the stream is not finite")
    return x


if __name__ == "__main__":
    main()
