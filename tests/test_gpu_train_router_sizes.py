"""The router-training example beyond 4096 tokens, with padding and bf16 logits."""
import numpy as np
import pytest
import torch

from .test_gpu_blockscale import dequant_rows, dequant_weight, round_e4m3, swiglu_ref
from .test_gpu_train_router import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,K", [(1, 4, 2), (300, 64, 6), (4096, 8, 3)])
def test_expert_order_is_the_layers_permutation(T, E, K):
    from moe_expert_layer_histogram_gb300 import moe_route_permute_static, router_balance
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).cuda()
    r = router_balance(logits, K)
    slots, offsets = example().expert_order(r)
    ids, w = torch.empty_like(r.ids), torch.empty_like(r.weights)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * K, dtype=torch.int32, device="cuda")
    moe_route_permute_static(logits, T, E, K, ids, w, off, perm,
                             torch.cuda.current_stream().cuda_stream)
    assert torch.equal(slots, perm) and torch.equal(offsets, off)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [600, 5000])
def test_padding_goes_through_no_expert(T, dtype):
    # live tokens against 64 bits (the tolerance of test_experts_match_64_bits:
    # a weighted sum of rows is as near as the rows are); padding, here NaN, gives
    # zeros and no gradient
    from moe_expert_layer_histogram_gb300 import blockscale_quantize
    E, K, H, I = 16, 2, 256, 128
    ex = example().FrozenExperts(E, K, H, I)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    logits = torch.randn(T, E, generator=g).to(dtype).cuda()
    mask = (torch.rand(T, generator=g) < 0.8).cuda()
    mask[0] = False
    x[~mask] = float("nan")
    out, routing, rows = ex.forward(x, logits, 0.1, mask)
    assert not bool(out[~mask].any()) and not bool(rows[~mask].any())
    assert int(routing.counts.sum()) == int(mask.sum()) * K
    pick = mask.nonzero()[::37, 0]
    a = dequant_rows(*blockscale_quantize(x[pick])).cpu()
    want = torch.zeros(len(pick), H, dtype=torch.float64)
    for i, t in enumerate(pick.tolist()):
        for k in range(K):
            e = int(routing.ids[t, k])
            h = swiglu_ref(a[i:i + 1], ex.w13[e], ex.s13[e], 0.0).numpy()
            s = (np.abs(h.reshape(1, -1, 128)).max(2) / 448).repeat(128, 1)
            hq = torch.from_numpy(round_e4m3(h / s) * s)
            want[i] += float(routing.weights[t, k]) * (hq @ dequant_weight(ex.w2[e], ex.s2[e]).cpu().t())[0]
    assert float((out[pick].double().cpu() - want).norm() / want.norm()) <= 1e-2
    d = ex.gate_gradient(logits, routing, rows, torch.ones_like(out), torch.ones((), device="cuda"))
    assert not bool(d[~mask].any()) and bool(torch.isfinite(d).all())
