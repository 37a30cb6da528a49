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


# ---------------------------------------------------------------- tiny values
def tiny_rows(M, K, seed):
    """Rows whose gate and up shrink row by row: h's block maxima run from about
    2^-120 through fp32's subnormal range to 0."""
    x = draw_x(M, K, seed).float()
    x = x * torch.exp2(-torch.linspace(57, 78, M, device="cuda"))[:, None]
    return x.bfloat16()


@pytest.mark.parametrize("clamp", [0.0, 7.0])
@pytest.mark.parametrize("M", [7, 60, 300, 3000])
def test_swiglu_of_tiny_values(M, clamp):
    # h is stored as code * s: s = RN(amax / 448) is off by up to 2^-150, which
    # moves (and at the top cuts) a value by up to 448 times that; a code is off
    # by 2^-4 of its value, or 2^-10 s, twice that where h's own error moves it
    # across a rounding boundary; h's error is 2^-13 of it and a few 2^-149.
    from moe_expert_layer_histogram_gb300 import blockscale_quantize, moe_blockscale_swiglu
    from .test_gpu_blockscale import dequant_rows, swiglu_ref
    I, K = 256, 272
    w, s = draw_w(1, 2 * I, K, 3)
    s = s * (8.5 / K ** 0.5)
    codes, scales = blockscale_quantize(tiny_rows(M, K, 1))
    h = torch.empty(M, I, dtype=torch.float8_e4m3fn, device="cuda")
    hs = torch.empty(I // 128, M, device="cuda")
    moe_blockscale_swiglu(codes, codes.stride(0), scales, M, w, w.stride(1), s, None, 1, M, I, K,
                          clamp, h, I, hs, M, torch.cuda.current_stream().cuda_stream)
    ref = swiglu_ref(dequant_rows(codes, scales).cpu(), w[0], s[0], clamp)
    top = ref.abs().amax(1)
    assert float(top.max()) > 2.0 ** -126 and float(top.min()) < 2.0 ** -149
    assert bool(torch.isfinite(hs).all()) and bool(torch.isfinite(h.float()).all())
    amax = ref.abs().view(M, 2, 128).amax(2)
    got_s = hs.t().double().cpu()
    assert bool(((got_s - amax / 448).abs() <= 2.0 ** -13 * amax / 448 + 2.0 ** -149).all())
    err = (dequant_rows(h, hs).cpu() - ref).abs()
    tol = (2.0 ** -3 + 2.0 ** -13) * ref.abs() + 2.0 ** -9 * got_s.repeat_interleave(128, 1) + 2.0 ** -141
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("M", [7, 60, 300])
def test_experts_of_tiny_values(M):
    # the tokens' h is far below bf16's normal range: finite and next to nothing
    from moe_expert_layer_histogram_gb300 import blockscale_experts
    H, I = 272, 256
    w13, s13 = draw_w(2, 2 * I, H, 1)
    w2, s2 = draw_w(2, H, I, 2)
    x = tiny_rows(M, H, 4)
    off = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    slots = torch.arange(M, dtype=torch.int32, device="cuda")
    y = blockscale_experts(x, slots, off, 1, w13, s13 * (8.5 / H ** 0.5), w2, s2)
    assert bool(torch.isfinite(y).all()) and float(y.abs().max()) < 2.0 ** -90


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("M,N,K", [(3, 9856, 11264), (16, 20000, 144)])
def test_few_rows_into_many_columns(M, N, K):
    # more tiles than can be split: a row's codes fill most of the shared memory,
    # and more CTAs than run at a time quantise the same rows
    from moe_expert_layer_histogram_gb300 import blockscale_linear, blockscale_quantize
    from .test_gpu_blockscale import assert_product, product_ref
    x = draw_x(M, K, M + N + K)
    w, s = draw_w(1, N, K, N)
    codes, scales = blockscale_quantize(x)
    assert_product(blockscale_linear(x, w[0], s[0]), *product_ref(codes, scales, w[0], s[0]), K)


@pytest.mark.parametrize("transpose", [False, True])
def test_one_weight_row_an_expert(transpose):
    from moe_expert_layer_histogram_gb300 import blockscale_matmul, blockscale_quantize
    from .test_gpu_blockscale import assert_product, dequant_rows, dequant_weight, offsets_of
    counts, cols = [3, 0, 20, 9], 272
    w, s = draw_w(4, 1, cols, 5)
    K = 1 if transpose else cols
    codes, scales = blockscale_quantize(draw_x(32, K, 2))
    out = blockscale_matmul(codes, scales, w, s, offsets_of(counts), transpose_w=transpose)
    a, r = dequant_rows(codes, scales).cpu(), 0
    for e, c in enumerate(counts):
        b = dequant_weight(w[e], s[e]).cpu()
        b = b if transpose else b.t()
        assert_product(out[r:r + c], a[r:r + c] @ b, a[r:r + c].abs() @ b.abs(), K)
        r += c


# ---------------------------------------------------------------- many tokens
# Sizes for which the experts' call quantises the tokens once and copies their
# codes to the rows (test_operators_devices_cpu.py holds them to that).
COPIED = [(2100, 5, 4, 2064, 640), (9000, 5, 2, 1040, 640), (1300, 4, 3, 4400, 1664)]


@pytest.mark.parametrize("T,E,topk,H,I", COPIED)
def test_experts_copy_the_tokens_codes(T, E, topk, H, I):
    # the same bits as the quantiser's gather and the two products one by one;
    # slots outside the tokens give zero rows; some rows against 64 bits (as in
    # test_experts_match_64_bits)
    import numpy as np
    from moe_expert_layer_histogram_gb300 import (blockscale_experts, blockscale_matmul,
                                                  blockscale_quantize, moe_blockscale_swiglu)
    from .test_gpu_blockscale import dequant_rows, dequant_weight, round_e4m3, swiglu_ref
    R = T * topk
    x = draw_x(T, H, T)
    w13, s13 = draw_w(E, 2 * I, H, 1)
    w2, s2 = draw_w(E, H, I, 2)
    s13 = s13 * (8.5 / H ** 0.5)
    g = torch.Generator().manual_seed(T)
    ids = torch.rand(T, E, generator=g).topk(topk, 1).indices.reshape(-1)
    slots = torch.sort(ids, stable=True).indices.to(torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    out_of = torch.tensor([0, 77, R // 2, R - 1])
    slots[out_of] = torch.tensor([-1, R, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    slots, off_gpu = slots.cuda(), off.cuda()
    y = blockscale_experts(x, slots, off_gpu, topk, w13, s13, w2, s2)
    codes, scales = blockscale_quantize(x, slots, topk)
    h = torch.empty(R, I, dtype=torch.float8_e4m3fn, device="cuda")
    hs = torch.empty(I // 128, R, device="cuda")
    moe_blockscale_swiglu(codes, H, scales, R, w13, H, s13, off_gpu, E, R, I, H, 0.0, h, I, hs, R,
                          torch.cuda.current_stream().cuda_stream)
    assert torch.equal(y, blockscale_matmul(h, hs, w2, s2, off_gpu))
    assert not bool(y[out_of].any()) and bool(y.any(1).sum() == R - 4)
    for e in range(E):
        rows = torch.arange(int(off[e]), int(off[e + 1]))[5::131]
        a = dequant_rows(codes[rows], scales[:, rows]).cpu()
        hr = swiglu_ref(a, w13[e], s13[e], 0.0).numpy()
        s = (np.abs(hr.reshape(len(rows), -1, 128)).max(2) / 448).repeat(128, 1)
        ref = torch.from_numpy(round_e4m3(hr / np.where(s == 0, 1, s)) * s) @ dequant_weight(w2[e], s2[e]).cpu().t()
        err = float((y[rows].double().cpu() - ref).norm() / ref.norm())
        assert err <= 1e-2, err
