"""A whole MoE layer with NVFP4 experts: quantise the weights once, then serve batches of one token to a full prefill.

Needs a GB300 and the built library (python -m combine_moe_route_meta_gb300.build):

    python examples/moe_layer_nvfp4.py [--tokens 1,32,512,4096] [--experts 64] [--hidden 4096] [--inter 1024] [--topk 8]

Batches of up to four pairs an expert (and MOE_LAYER_MAX_TOKENS tokens) go through moe_layer_few_tokens; larger ones
through route metadata, NVFP4 dispatch, gate/up product with SwiGLU, down product and combine. Each is timed and compared with the layer's bf16
weights in 32-bit arithmetic.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_moe_route_meta_gb300 as moe  # noqa: E402


def reference(x, ids, weights, w13, w2):
    out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    for e in range(w13.shape[0]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            gate, up = (x[t].float() @ w13[e].float().T).chunk(2, dim=1)
            out.index_add_(0, t, (torch.nn.functional.silu(gate) * up) @ w2[e].float().T * weights[t, k, None])
    return out


def microseconds(fn, steps=20):
    for _ in range(3):
        fn()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        fn()
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end) * 1000 / steps


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", default="1,32,512,4096")
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inter", type=int, default=1024)
    p.add_argument("--topk", type=int, default=8)
    a = p.parse_args()
    sizes = [int(t) for t in a.tokens.split(",")]
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    w13 = (randn(a.experts, 2 * a.inter, a.hidden) * a.hidden ** -0.5).bfloat16()
    w2 = (randn(a.experts, a.hidden, a.inter) * a.inter ** -0.5).bfloat16()
    weights = moe.quantize_experts(w13, w2)
    # scales of the activations: 448 * 6 over the largest value to expect (from a calibration run, in earnest)
    layer = moe.MoELayer(weights, a.topk, max(sizes), input_scale=2688.0 / 6.0, inter_scale=2688.0 / 16.0)

    for t in sizes:
        x = randn(t, a.hidden).bfloat16()
        logits, ids = randn(t, a.experts).topk(a.topk, dim=1)
        ids, gates = ids.int().contiguous(), logits.softmax(dim=1).contiguous()
        y = layer(x, ids, gates)
        layer.check()
        want = reference(x, ids, gates, w13, w2)
        off = ((y.float() - want).norm() / want.norm()).item()
        us = microseconds(lambda: layer(x, ids, gates))
        print(f"{t:6d} tokens: {us:9.1f} us, {100 * off:.1f} % off the bf16 layer (NVFP4's own rounding)")


if __name__ == "__main__":
    main()
