"""Decode steps through a stack of sparse blocks: x = x + MoE(norm(x)), a few tokens at a time.

Each block is two calls: moe_rmsnorm (the residual stream and its normalised rows) and
moe_forward_few (the whole layer, the residual added).  The step is captured once in a CUDA
graph and replayed for every token.

    python examples/decode_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_expert_ffn_moe_gb300 as moe  # noqa: E402

EPS = 1e-6


class Block:
    """One sparse block with 8-bit experts (E4M3, a scale a weight row)."""

    def __init__(self, T, d, E, K, inter, inter_shared, g):
        self.shape = moe.make_shape(T, d, E, K, inter, inter_shared, "bf16", "sigmoid")
        self.workspace = moe.alloc_few_workspace(self.shape)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.weight = (1 + 0.1 * rnd(d)).bfloat16()
        self.w_g = (rnd(E, d) / d ** 0.5).bfloat16()
        self.bias = 0.1 * rnd(E)
        self.q = {}
        for name, shape in (("w_gate", (E, inter, d)), ("w_up", (E, inter, d)),
                            ("w_down", (E, d, inter)), ("ws_gate", (inter_shared, d)),
                            ("ws_up", (inter_shared, d)), ("ws_down", (d, inter_shared))):
            w = (rnd(*shape) / shape[-1] ** 0.5).bfloat16()
            self.q[name] = torch.empty(shape, dtype=torch.uint8, device="cuda")
            scales = ("s" if name.startswith("w_") else "ss") + name[name.index("_"):]
            self.q[scales] = torch.empty(shape[:-1], device="cuda")
            moe.moe_quantize_fp8_rows(w, self.q[name], self.q[scales])
        self.experts = moe.make_fp8_experts(self.q)

    def __call__(self, x, normed):
        """x (the residual stream, in place) += MoE(norm(x))"""
        moe.moe_rmsnorm(x, None, self.weight, EPS, None, normed, None, None)
        moe.moe_forward_few_fp8(self.shape, normed, self.w_g, self.bias, self.experts, x, x,
                                self.workspace)


def main(T=4, d=1024, E=32, K=4, inter=512, inter_shared=512, layers=4, steps=8, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [Block(T, d, E, K, inter, inter_shared, g) for _ in range(layers)]
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    normed = torch.empty_like(x)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            for block in blocks:
                block(x, normed)
    out = []
    for _ in range(steps):
        x.copy_(torch.randn(T, d, generator=g, device="cuda"))  # the next tokens' rows
        graph.replay()
        out.append(x.clone())
    torch.cuda.synchronize()
    errors = [moe.moe_get_device_error(b.workspace) for b in blocks]
    if any(errors):
        raise RuntimeError(f"device errors {errors}")
    return blocks, torch.stack(out)


if __name__ == "__main__":
    _, rows = main()
    print(f"{len(rows)} steps, rows of RMS {rows.float().square().mean().sqrt().item():.3f}")
