"""Block-scaled FP8 operators on unusual inputs: offsets out of order and
values at the ends of fp32's range.  Helpers and tolerances as in
test_gpu_blockscale.py."""
import pytest
import torch

from .test_gpu_blockscale import draw_w, draw_x, no_wait_gave_up  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- offsets
def in_order(offsets, M):
    """What the offsets mean: clamped into [0, M], none below one before it."""
    out, top = [], 0
    for o in offsets:
        top = max(top, min(max(o, 0), M))
        out.append(top)
    return out


def hostile_offsets(E, M, seed):
    g = torch.Generator().manual_seed(seed)
    some = torch.randint(-M, 2 * M + 1, (E + 1,), generator=g).tolist()
    return {"alternating": [0 if e % 2 == 0 else M for e in range(E + 1)],
            "falling": [M - e * M // E for e in range(E + 1)],
            "any": some,
            "extreme": [(2 ** 31 - 1, -2 ** 31, 0, M)[v % 4] for v in some],
            "late": [0] * (E // 2) + [M // 2] * (E - E // 2) + [0]}


# up to 16 rows the reduction is split (one item per cluster); 60 rows: several
# chunks' worth of experts per CTA; 2100 and 3300: wide items, alone and in pairs
@pytest.mark.parametrize("E,M,N,K", [(2, 3, 256, 1024), (20, 16, 256, 1024), (64, 16, 144, 2064),
                                     (512, 9, 128, 528), (512, 60, 130, 256), (33, 300, 144, 272),
                                     (2, 2100, 1552, 272), (3, 3300, 1552, 272)])
@pytest.mark.parametrize("kind", ["alternating", "falling", "any", "extreme", "late"])
def test_offsets_out_of_order(kind, E, M, N, K):
    # the plan goes by the sizes alone, so the offsets put in order give the same
    # bits; nothing around the result is written
    from moe_expert_layer_histogram_gb300 import blockscale_matmul, blockscale_quantize
    off = hostile_offsets(E, M, E + M)[kind]
    want_off = in_order(off, M)
    w, s = draw_w(E, N, K, E)
    codes, scales = blockscale_quantize(draw_x(M, K, M))

    def call(offsets):
        store = torch.full((M + 2, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        blockscale_matmul(codes, scales, w, s, torch.tensor(offsets, dtype=torch.int32).cuda(),
                          out=store[1:M + 1, 8:N + 8])
        return store

    got, want = call(off), call(want_off)
    assert torch.equal(got, want)
    assert bool((got[0] == 7).all()) and bool((got[-1] == 7).all())
    assert bool((got[:, :8] == 7).all()) and bool((got[:, N + 8:] == 7).all())
    inside = got[1:M + 1, 8:N + 8]
    assert bool((inside[:want_off[0]] == 7).all()) and bool((inside[want_off[-1]:] == 7).all())


@pytest.mark.parametrize("E,M", [(20, 16), (64, 16), (512, 9), (40, 200)])
@pytest.mark.parametrize("kind", ["alternating", "falling", "any", "extreme", "late"])
def test_experts_with_offsets_out_of_order(kind, E, M):
    from moe_expert_layer_histogram_gb300 import blockscale_experts
    H, I = 528, 128
    off = hostile_offsets(E, M, E + M)[kind]
    w13, s13 = draw_w(E, 2 * I, H, 1)
    w2, s2 = draw_w(E, H, I, 2)
    x = draw_x(M, H, 3)
    slots = torch.arange(M, dtype=torch.int32, device="cuda")

    def call(offsets):
        out = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
        return blockscale_experts(x, slots, torch.tensor(offsets, dtype=torch.int32).cuda(), 1, w13,
                                  s13, w2, s2, out=out)

    assert torch.equal(call(off), call(in_order(off, M)))
