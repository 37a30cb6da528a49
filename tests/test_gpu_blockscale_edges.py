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


# ---------------------------------------------------------------- non-finite values
# rows split over a cluster, rows of one chunk, several chunks, CTA pairs
@pytest.mark.parametrize("clamp", [0.0, 7.0])
@pytest.mark.parametrize("M,K", [(6, 1040), (100, 256), (300, 272), (3000, 272)])
def test_swiglu_keeps_non_finite_rows(M, K, clamp):
    from moe_expert_layer_histogram_gb300 import blockscale_quantize, moe_blockscale_swiglu
    I = 256
    w, s = draw_w(1, 2 * I, K, 3)
    s = s * (8.5 / K ** 0.5)
    x = draw_x(M, K, 1)
    bad = sorted({2, M // 2, M - 1})
    for r, v in zip(bad, (float("inf"), float("nan"), -float("inf"))):
        x[r, 3 + r % 100] = v
    codes, scales = blockscale_quantize(x)
    h = torch.empty(M, I, dtype=torch.float8_e4m3fn, device="cuda")
    hs = torch.empty(I // 128, M, device="cuda")
    moe_blockscale_swiglu(codes, codes.stride(0), scales, M, w, w.stride(1), s, None, 1, M, I, K,
                          clamp, h, I, hs, M, torch.cuda.current_stream().cuda_stream)
    is_bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    is_bad[bad] = True
    assert torch.equal(torch.isnan(hs).all(0), is_bad) and torch.equal(torch.isnan(hs).any(0), is_bad)
    nan = torch.isnan(h.float())
    assert torch.equal(nan.all(1), is_bad) and torch.equal(nan.any(1), is_bad)


@pytest.mark.parametrize("clamp", [0.0, 7.0])
@pytest.mark.parametrize("T,E,topk", [(3, 8, 2), (60, 4, 2), (1500, 3, 2)])
def test_experts_keep_non_finite_tokens(T, E, topk, clamp):
    # a token with an infinity or NaN gives NaN rows, the others stay as they are
    from moe_expert_layer_histogram_gb300 import blockscale_experts
    H, I = 400, 256
    w13, s13 = draw_w(E, 2 * I, H, 1)
    w2, s2 = draw_w(E, H, I, 2)
    s13 = s13 * (8.5 / H ** 0.5)
    g = torch.Generator().manual_seed(T)
    ids = torch.rand(T, E, generator=g).topk(topk, 1).indices.reshape(-1)
    slots = torch.sort(ids, stable=True).indices.to(torch.int32).cuda()
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    x = draw_x(T, H, 5)
    want = blockscale_experts(x, slots, off.cuda(), topk, w13, s13, w2, s2, clamp=clamp)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[0] = bad[T - 1] = True
    x[0, 399], x[T - 1, 0] = float("nan"), float("inf")
    y = blockscale_experts(x, slots, off.cuda(), topk, w13, s13, w2, s2, clamp=clamp)
    rows = bad[slots.long() // topk]
    assert bool(torch.isfinite(want).all())
    assert bool(torch.isnan(y[rows]).all()) and torch.equal(y[~rows], want[~rows])
