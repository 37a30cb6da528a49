"""Train a router in front of frozen FP8 experts (scales per block of 128).

    python examples/train_router.py [--tokens T] [--steps N]

Each step routes a batch (top-k, weights, counts and the balance loss in one
call), runs the experts' products on the permuted rows, combines them with the
routing weights, and takes the gate's gradient from the task loss (through the
routing weights) and from the balance loss.  The experts stay as they are.
The task: follow a teacher, the same experts behind another gate; the student
starts with a gate that prefers a few experts.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_expert_layer_histogram_gb300 import (blockscale_experts, router_balance,  # noqa: E402
                                              router_balance_backward, router_order)


def quantize_weight(w):
    """bf16-like weights [E, N, K] (N, K multiples of 128) -> e4m3 codes and one
    fp32 scale per 128 x 128 block."""
    E, N, K = w.shape
    v = w.float().view(E, N // 128, 128, K // 128, 128)
    s = v.abs().amax(dim=(2, 4)) / 448.0
    return (v / s[:, :, None, :, None]).view(E, N, K).to(torch.float8_e4m3fn), s


def expert_order(routing):
    """The routed slots t * K + k in expert order, as blockscale_experts takes
    them: slots int32 [T * K], offsets int32 [E + 1].  Slots of tokens that are
    not live (id -1) come last and belong to no expert."""
    order = router_order(routing.ids, routing.counts.numel())
    return order.slots, order.offsets


class FrozenExperts:
    """Routed FP8 experts: forward keeps what the gate's gradient needs."""

    def __init__(self, E, top_k, H, I, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.K = E, top_k
        self.w13, self.s13 = quantize_weight(
            torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5)
        self.w2, self.s2 = quantize_weight(
            torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5)

    def forward(self, x, logits, coef, mask=None):
        """Any number of tokens, logits f32 or bf16; mask as router_balance
        takes it: padding goes through no expert and gives zero rows."""
        T, dev = x.shape[0], x.device
        routing = router_balance(logits, self.K, coef, mask=mask)
        slots, off = expert_order(routing)
        # (rows of no expert, padding's, are left as they are: zero)
        y = torch.zeros(T * self.K, x.shape[1], dtype=torch.bfloat16, device=dev)
        blockscale_experts(x, slots, off, self.K, self.w13, self.s13, self.w2, self.s2, out=y)
        row_of_slot = torch.empty(T * self.K, dtype=torch.int64, device=dev)
        row_of_slot[slots.long()] = torch.arange(T * self.K, device=dev)
        rows = y[row_of_slot].view(T, self.K, -1).float()      # each token's expert outputs
        out = (routing.weights.unsqueeze(-1) * rows).sum(1)
        return out, routing, rows

    @staticmethod
    def gate_gradient(logits, routing, rows, d_out, d_loss):
        """Gradient of the logits from d_out [T, H] and the balance loss's d_loss."""
        d_weights = (d_out.unsqueeze(1) * rows).sum(-1)
        return router_balance_backward(logits, routing, d_loss=d_loss, d_weights=d_weights)


def train(tokens=512, steps=60, E=64, top_k=6, H=512, I=256, coef=0.05, lr=20.0, seed=0):
    """Returns a list of (task loss, balance loss / coef, largest load / mean load)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    experts = FrozenExperts(E, top_k, H, I, seed)
    teacher = torch.randn(H, E, generator=g, device="cuda") * H ** -0.5 * 2
    gate = teacher + torch.randn(H, E, generator=g, device="cuda") * H ** -0.5
    bias = torch.zeros(E, device="cuda")
    bias[: E // 8] = 2.0                                       # a few experts preferred
    one = torch.ones((), device="cuda")
    history = []
    for _ in range(steps):
        x = torch.randn(tokens, H, generator=g, device="cuda").bfloat16()
        target, _, _ = experts.forward(x, x.float() @ teacher, coef)
        logits = x.float() @ gate + bias
        out, routing, rows = experts.forward(x, logits, coef)
        err = out - target
        d_logits = experts.gate_gradient(logits, routing, rows, 2 * err / err.numel(), one)
        gate -= lr * (x.float().t() @ d_logits)
        bias -= lr * d_logits.sum(0)
        load = routing.counts.float()
        history.append((float((err * err).mean()), float(routing.loss) / coef,
                        float(load.max() / load.mean())))
    return history


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--steps", type=int, default=60)
    a = p.parse_args()
    for i, (task, balance, peak) in enumerate(train(a.tokens, a.steps)):
        if i % 10 == 0 or i + 1 == a.steps:
            print("step %3d  task loss %.4f  balance loss %.4f  largest load %.2f x mean"
                  % (i, task, balance, peak))


if __name__ == "__main__":
    main()
