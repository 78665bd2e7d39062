"""Trains the router of a sparse MoE layer over frozen 8-bit experts.

The experts (E4M3 codes with row scales) stay as they are; the router's matrix
w_g learns to imitate a teacher layer that uses the same experts with another
router, and the balance loss keeps the experts evenly used.  A step runs the
library's operators the way a training program does:

    scores = x w_g^T                      (torch, so that autograd carries d_scores on)
    moe_route, moe_permute, moe_expert_ffn_fp8       forward, frozen experts
    moe_combine_dropout                              y = x + dropout(sum of the experts)
    moe_balance_loss                                 loss and per-expert counts
    moe_combine_backward                             d_y -> d_topk_w
    moe_route_backward                               d_topk_w and the balance loss -> d_scores
    scores.backward(d_scores)                        -> gradient of w_g

    python examples/train_router.py --steps 60
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_expert_ffn_moe_gb300 as moe  # noqa: E402


class FrozenExperts:
    """E experts of width d and inner width inter, quantised once to E4M3."""

    def __init__(self, d, E, inter, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = {}
        for name, shape, fan in (("gate", (E, inter, d), d), ("up", (E, inter, d), d),
                                 ("down", (E, d, inter), inter)):
            w = (torch.randn(shape, generator=g, device="cuda") * fan ** -0.5).bfloat16()
            q[f"w_{name}"] = torch.empty(shape, dtype=torch.uint8, device="cuda")
            q[f"s_{name}"] = torch.empty(shape[:-1], device="cuda")
            moe.moe_quantize_fp8_rows(w, q[f"w_{name}"], q[f"s_{name}"])
        self.tensors, self.handle = q, moe.make_fp8_experts(q)


class RouterTrainer:
    """One layer's buffers, and a step of its router's training."""

    def __init__(self, T, d, E, K, inter, p=0.1, alpha=0.05, sequences=4, seed=0):
        self.shape = moe.make_shape(T, d, E, K, inter, 0, "bf16")
        self.T, self.p, self.alpha = T, p, alpha
        self.experts = FrozenExperts(d, E, inter, seed)
        new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.topk_idx, self.topk_w = new(T, K, dt=torch.int32), new(T, K)
        self.offsets, self.count = new(E + 1, dt=torch.int32), new(E, dt=torch.int32)
        self.inv_perm = new(T * K, dt=torch.int32)
        self.x_perm, self.y_perm = (new(T * K, d, dt=torch.bfloat16) for _ in range(2))
        self.y = new(T, d, dt=torch.bfloat16)
        self.counts = new(sequences, E, dt=torch.int32)
        self.mean_probs, self.balance = new(sequences, E), new(1)
        self.d_topk_w, self.d_scores = new(T, K), new(T, E)
        self.workspace = moe.alloc_workspace(self.shape)
        self.balance_workspace = moe.alloc_balance_workspace(self.shape, sequences)
        # packed sequences of the batch, and the generator's {seed, offset}
        self.seq_offsets = torch.linspace(0, T, sequences + 1).to(torch.int32).cuda()
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")

    def forward(self, x, scores, p):
        """y = x + dropout(the layer's output with the given scores)."""
        s, ws = self.shape, self.workspace
        moe.moe_route(s, None, None, None, scores, None, self.topk_idx, self.topk_w, ws)
        moe.moe_permute(s, self.topk_idx, x, self.count, self.offsets, None, self.inv_perm,
                        self.x_perm, ws)
        moe.moe_expert_ffn_fp8(s, self.x_perm, self.offsets, self.experts.handle, self.y_perm, ws)
        moe.moe_combine_dropout(s, self.y_perm, self.inv_perm, self.topk_w, None, x, p, self.rng,
                                self.y)
        return self.y

    def step(self, x, target, w_g):
        """Task and balance loss of one batch; w_g.grad gets their gradient."""
        s = self.shape
        scores = x.float() @ w_g.t()
        y = self.forward(x, scores.detach(), self.p)
        moe.moe_balance_loss(s, scores.detach(), self.topk_idx, None, self.seq_offsets, self.alpha,
                             self.counts, self.mean_probs, self.balance, self.balance_workspace)
        err = y.float() - target.float()
        task = err.square().mean()
        d_y = (err * (2.0 / err.numel())).bfloat16()
        moe.moe_combine_backward(s, d_y, self.y_perm, self.inv_perm, self.topk_w, self.p, self.rng,
                                 None, self.d_topk_w, None)
        moe.moe_route_backward(s, scores.detach(), self.topk_idx, self.d_topk_w, None,
                               self.seq_offsets, self.alpha, self.counts, None, self.d_scores)
        scores.backward(self.d_scores)
        self.rng[1] += 1  # the next step's masks
        return task, self.balance


def train(steps=60, T=2048, d=512, E=16, K=2, inter=256, lr=3e-2, seed=0, log=print):
    """Returns the task losses and balance losses of the steps (floats)."""
    layer = RouterTrainer(T, d, E, K, inter, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher = torch.randn(E, d, generator=g, device="cuda") * d ** -0.5
    w_g = (torch.randn(E, d, generator=g, device="cuda") * d ** -0.5).requires_grad_()
    opt = torch.optim.Adam([w_g], lr=lr)
    tasks, balances = [], []
    for i in range(steps):
        x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
        target = layer.forward(x, x.float() @ teacher.t(), 0.0).clone()
        opt.zero_grad()
        task, balance = layer.step(x, target, w_g)
        opt.step()
        tasks.append(task.item())
        balances.append(balance.item())
        if log and (i % 10 == 0 or i == steps - 1):
            used = (layer.counts.sum(0) > 0).sum().item()
            log(f"step {i:3d}  task {tasks[-1]:.5f}  balance {balances[-1]:.5f}  "
                f"experts used {used}/{E}")
    if moe.moe_get_device_error(layer.workspace) or moe.moe_get_device_error(layer.balance_workspace):
        raise RuntimeError("device error")
    return tasks, balances


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    a = ap.parse_args()
    train(steps=a.steps, T=a.tokens, E=a.experts)
