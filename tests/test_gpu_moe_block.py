"""A whole MoE block of the operators together: gate, expert order, the experts'
products, the join with its norms, and the next projection; served in 8 bits, and
in training with the gate's gradient.

Tolerances as in the operators' own tests (test_gpu_int8.py, test_gpu_join.py,
test_gpu_gate.py): each step is compared with 64 bits on what the step before gave.
"""
import pytest
import torch

from .test_gpu_int8 import close, codes_of, matmul_reference, randn, scales_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8


def block(T, E, K, H, I, seed=0, masked=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mask = torch.rand(T, generator=g, device="cuda") >= masked
    return dict(x=randn(T, H, seed=seed), mask=mask,
                logits=randn(T, E, seed=seed + 1, dtype=torch.float32),
                bias=randn(E, seed=seed + 2, dtype=torch.float32, scale=0.05),
                w13=codes_of(E, 2 * I, H, seed=seed + 3), s13=scales_of(E, 2 * I) * 0.02,
                w2=codes_of(E, H, I, seed=seed + 4), s2=scales_of(E, H) * 0.1,
                shared=randn(T, H, seed=seed + 5), gate=randn(T, seed=seed + 6, dtype=torch.float32),
                norm=1 + randn(H, seed=seed + 7, dtype=torch.float32, scale=0.1))


@pytest.mark.parametrize("T,E,K,H,I,N", [(1, 16, 4, 512, 128, 300), (45, 16, 3, 1024, 256, 512),
                                         (2000, 8, 2, 256, 128, 100)])
def test_a_served_block_in_8_bits(T, E, K, H, I, N):
    from moe_expert_layer_histogram_gb300 import (block_join, int8_experts, int8_matmul, router_gate,
                                                  router_order)
    b = block(T, E, K, H, I, masked=0.2 if T > 1 else 0.0)
    wn, sn = codes_of(N, H, seed=20), scales_of(N)
    r = router_gate(b["logits"], K, score="sigmoid", bias=b["bias"], groups=4, group_top=2,
                    scale=2.0, mask=b["mask"])
    o = router_order(r.ids, E)
    rows = int8_experts(b["x"], o.slots, o.offsets, K, b["w13"], b["s13"], b["w2"], b["s2"])
    j = block_join(b["x"], expert_rows=rows, order=o, weights=r.weights, shared=b["shared"],
                   gate=b["gate"], scale=0.5, norm_weight=b["norm"], quantize=True)
    y = int8_matmul(j.codes, j.code_scales, wn, sn)
    # every live slot's row is its expert's; padding has none
    place = o.rows.view(T, K)
    assert bool((place[~b["mask"]] == -1).all()) and bool((place[b["mask"]] >= 0).all())
    expert = torch.bucketize(place[b["mask"]], o.offsets[1:], right=True)
    assert torch.equal(expert.int(), r.ids[b["mask"]])
    assert torch.equal(o.slots[place[b["mask"]].flatten().long()].view(-1, K),
                       torch.arange(T * K, device="cuda", dtype=torch.int32).view(T, K)[b["mask"]])
    z = torch.where((place >= 0)[:, :, None], rows.double()[place.clamp(min=0).long()], 0.0)
    w = r.weights.double()[:, :, None]
    s = torch.sigmoid(b["gate"].double())[:, None]
    want = b["x"].double() + 0.5 * ((w * z).sum(1) + s * b["shared"].double())
    mag = b["x"].double().abs() + (w * z).abs().sum(1) + (s * b["shared"].double()).abs()
    assert bool(((j.x.double() - want).abs() <= 100 * U * mag + BF16 * (want.abs() + mag * U)).all())
    x = j.x.double()
    h = x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * b["norm"].double()
    q = h / j.code_scales.double()[:, None]
    assert bool(((j.codes.double() - q).abs() <= 0.5 + 128 * 110 * U).all())
    close(y, *matmul_reference(j.codes, j.code_scales, wn, sn), H)


@pytest.mark.parametrize("score,normalize", [("sigmoid", True), ("softmax", False)])
def test_a_training_step_of_the_gate(score, normalize):
    """Frozen FP8 experts; the gradient of the logits through the norms and the join, against
    torch's own differentiation of the same function in 64 bits (the experts' rows and the choice
    are constants of it)."""
    from moe_expert_layer_histogram_gb300 import (blockscale_experts, block_join,
                                                  block_join_backward, router_gate,
                                                  router_gate_backward, router_order)
    T, E, K, H, I = 61, 16, 3, 256, 128
    b = block(T, E, K, H, I, seed=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    w13 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 20).to(torch.float8_e4m3fn)
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * 20).to(torch.float8_e4m3fn)
    s13 = torch.full((E, 2, 2), 3e-3, device="cuda")
    s2 = torch.full((E, 2, 1), 3e-3, device="cuda")
    kw = dict(score=score, normalize=normalize, bias=b["bias"], groups=4, group_top=2, scale=1.5)
    post, norm = 1 + randn(H, seed=9, dtype=torch.float32, scale=0.1), b["norm"]
    r = router_gate(b["logits"], K, mask=b["mask"], **kw)
    o = router_order(r.ids, E)
    x32 = b["x"].float()
    rows = torch.zeros(T * K, H, dtype=torch.bfloat16, device="cuda")
    blockscale_experts(b["x"], o.slots, o.offsets, K, w13, s13, w2, s2, out=rows)
    j = block_join(x32, expert_rows=rows, order=o, weights=r.weights, shared=b["shared"],
                   gate=b["gate"], post_weight=post, scale=0.7, norm_weight=norm)
    dx, dh = randn(T, H, seed=11, dtype=torch.float32), randn(T, H, seed=12)
    grads = block_join_backward(j, d_x=dx, d_h=dh)
    d_logits = router_gate_backward(b["logits"], r, grads.weights)

    logits = b["logits"].double().requires_grad_()
    gate = b["gate"].double().requires_grad_()
    s = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    picked = s.gather(1, r.ids.clamp(min=0).long())
    w = 1.5 * (picked / picked.sum(1, keepdim=True) if normalize else picked) * b["mask"][:, None]
    place = o.rows.view(T, K)
    z = torch.where((place >= 0)[:, :, None], rows.double()[place.clamp(min=0).long()], 0.0)
    y = (w[:, :, None] * z).sum(1) + torch.sigmoid(gate)[:, None] * b["shared"].double()

    def norm_of(v, weight):
        return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * weight.double()
    x = x32.double() + 0.7 * norm_of(y, post)
    ((x * dx.double()).sum() + (norm_of(x, norm) * dh.double()).sum()).backward()
    # Both gradients are sums over the width of d y times a row (z_k, or the shared
    # expert's), and d y, off by 400 u = 2.4e-5 of its terms' magnitudes
    # (test_gpu_join.py), is orthogonal to y behind the norm: a token whose y is its
    # shared row alone has a gate gradient of almost 0 from terms of order 1.  So 1e-4
    # of the sum of the terms' magnitudes, times what the weights do with it (scale
    # 1.5, derivatives of at most 1)
    s = torch.sigmoid(b["gate"].double())[:, None]
    dy = (grads.shared.double() / s).abs() * (1 + BF16)
    of_rows = 1.5 * (dy[:, None] * z.abs()).sum(2).amax(1, keepdim=True)
    of_gate = (dy * b["shared"].double().abs()).sum(1, keepdim=True)
    for got, want, size in ((d_logits, logits.grad, of_rows),
                            (grads.gate[:, None], gate.grad[:, None], of_gate)):
        assert bool(((got.double() - want).abs() <= 1e-4 * size + 1e-9).all())
    assert bool((d_logits[~b["mask"]] == 0).all())
