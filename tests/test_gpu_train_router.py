"""The router-training example: it learns, and its gate gradient is the
gradient of the loss (against differences of a plain 64-bit evaluation)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "train_router", os.path.join(ROOT, "examples", "train_router.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_both_losses():
    h = example().train(tokens=256, steps=40)
    first, last = h[0], [sum(v) / 5 for v in zip(*h[-5:])]
    assert last[0] < 0.8 * first[0], (first, last)      # task
    assert last[1] < first[1], (first, last)            # balance: 1 is even
    assert last[2] < first[2], (first, last)            # largest load


def test_gate_gradient_against_differences():
    # loss(logits) = <c, out> + d_loss * balance with the experts' outputs fixed:
    # exact in the weights, so central differences of step 1e-5 in 64 bits
    # agree to about their square; the kernels' fp32 adds 1e-5 of the terms
    m = example()
    ex = m.FrozenExperts(8, 2, 256, 128)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(24, 256, generator=g, device="cuda").bfloat16()
    logits = torch.randn(24, 8, generator=g, device="cuda")
    c = torch.randn(24, 256, generator=g, device="cuda")
    coef = 2.0
    _, routing, rows = ex.forward(x, logits, coef)
    d = ex.gate_gradient(logits, routing, rows, c, torch.ones((), device="cuda")).double().cpu()
    ids, rows64, c64 = routing.ids.long().cpu(), rows.double().cpu(), c.double().cpu()
    counts = routing.counts.double().cpu()

    def loss(z):
        w = torch.softmax(z.gather(1, ids), 1)
        out = (w.unsqueeze(-1) * rows64).sum(1)
        p = torch.softmax(z, 1)
        return (c64 * out).sum() + coef * (counts * 8 / (2 * 24) * p.mean(0)).sum()

    z = logits.double().cpu()
    for seed in range(4):
        v = torch.randn(24, 8, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        num = (loss(z + 1e-5 * v) - loss(z - 1e-5 * v)) / 2e-5
        got = (d * v).sum()
        assert abs(float(num - got)) <= 1e-5 * float((d * v).abs().sum()) + 1e-6
