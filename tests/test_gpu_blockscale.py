"""Block-scaled FP8 operators against plain 64-bit implementations.

Quantisation is exact by definition (two roundings to fp32 and one to e4m3),
so codes and scales are compared bit for bit.

A product of exact fp8 values, summed in fp32 in any order with additions that
may truncate (2^-23 each), is off by at most (K + 8) 2^-23 of the sum of its
terms' magnitudes; the scale product and the scaled additions are among the
8.  The result's rounding to bf16 (8 significant bits) adds 2^-8 of itself.

The fused SwiGLU's fp32 values carry the product's error, so a few codes near
a rounding boundary may fall on the other side: each must be within one e4m3
step, and a value moves across a boundary only if it lies within its error of
one.  With errors below 2^-13 of the value and steps of at least 2^-4 of it,
that is at most a fraction 2^-13 * 2 / 2^-4 = 2^-8 of the codes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    from moe_expert_layer_histogram_gb300 import moe_blockscale_status
    yield
    assert moe_blockscale_status() == 0


def cdiv(a, b):
    return (a + b - 1) // b


def dequant_rows(codes, scales):
    """codes [R, C], scales [ceil(C/128), R] -> float64."""
    C = codes.shape[1]
    s = scales.double().t().repeat_interleave(128, 1)[:, :C]
    return codes.double() * s


def dequant_weight(w, s):
    N, K = w.shape[-2:]
    s = s.double().repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]
    return w.double() * s


def ref_quantize(x):
    """Independent restatement in numpy: x float64 [R, C] of fp32 or bf16 values."""
    R, C = x.shape
    codes, scales = np.zeros((R, C)), np.zeros((cdiv(C, 128), R), np.float32)
    for b in range(cdiv(C, 128)):
        blk = x[:, b * 128:(b + 1) * 128]
        amax = np.abs(blk).max(1).astype(np.float32)
        s = (amax / np.float32(448)).astype(np.float32)
        scales[b] = s
        with np.errstate(divide="ignore", invalid="ignore"):
            q = (blk.astype(np.float32) / s[:, None]).astype(np.float32)
        q[s == 0] = 0
        codes[:, b * 128:(b + 1) * 128] = round_e4m3(q.astype(np.float64))
    return codes, scales


def round_e4m3(q):
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -30))), -6)
    step = 2.0 ** (e - 3)
    return np.clip(np.round(q / step) * step, -448, 448)


def draw_x(M, K, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, K, generator=g) * scale).bfloat16().cuda()


def draw_w(E, N, K, seed, ldw=None):
    """Codes [E, N, K] (views of padded rows where K % 16) and block scales."""
    g = torch.Generator().manual_seed(seed)
    ld = ldw or cdiv(K, 16) * 16
    store = torch.randn(E, N, ld, generator=g).mul_(60).clamp(-448, 448).to(torch.float8_e4m3fn)
    store = store.view(torch.uint8)
    store[:, :, K:] = 0x7F                                   # NaN in the padding: must not matter
    w = store.cuda().view(torch.float8_e4m3fn)[:, :, :K]
    s = (torch.rand(E, cdiv(N, 128), cdiv(K, 128), generator=g) + 0.5) * 2.0 ** -9
    return w, s.cuda()


def product_ref(codes, scales, w, s):
    """(y, sum of magnitudes) in 64 bits; w [N, K]."""
    a, b = dequant_rows(codes, scales).cpu(), dequant_weight(w, s).cpu()
    return a @ b.t(), a.abs() @ b.abs().t()


def assert_product(out, y, mag, K):
    err = (out.double().cpu() - y).abs()
    tol = (K + 8) * 2.0 ** -23 * mag + 2.0 ** -8 * y.abs() + 1e-38
    assert bool((err <= tol).all()), float((err / tol).max())


# ---------------------------------------------------------------- quantise
@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (3, 7), (5, 127), (5, 129), (17, 144),
                                 (64, 256), (33, 1000), (130, 2048), (257, 640), (2, 7168)])
def test_quantize_bit_exact(R, C):
    from moe_expert_layer_histogram_gb300 import blockscale_quantize
    x = draw_x(R, C, R * 1000 + C)
    codes, scales = blockscale_quantize(x)
    want_c, want_s = ref_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.double().cpu().numpy(), want_c)


def crafted_rows():
    """128-column rows with hard scales and quotients."""
    rows = []
    base = torch.linspace(-1, 1, 128)
    for amax in (448.0, 447.0, 1.0, 3.5, 2.0 ** -60, 2.0 ** -100, 2.0 ** -120, 2.0 ** -126,
                 2.0 ** -133, 3.0e38, 1e38, 1.0078125, 1.9921875, 0.875, 7.0, 21.0):
        rows.append(base * amax)
        r = torch.zeros(128)
        r[5], r[77] = amax, -amax * 0.75                     # 21/16 in e4m3 terms: a rounding tie
        r[9] = amax * 2.0 ** -9
        r[10] = -amax * 2.0 ** -17
        rows.append(r)
    rows.append(torch.zeros(128))
    rows.append(-torch.zeros(128))
    return torch.stack(rows).bfloat16().cuda()


def test_quantize_hard_blocks():
    from moe_expert_layer_histogram_gb300 import blockscale_quantize
    x = crafted_rows()
    codes, scales = blockscale_quantize(x)
    want_c, want_s = ref_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.double().cpu().numpy(), want_c)


def test_quantize_all_significands():
    """Every pair of a block maximum's and a value's significand, the value at
    every exponent that has a code."""
    from moe_expert_layer_histogram_gb300 import blockscale_quantize
    a = torch.arange(128, 256).double() / 128
    m = torch.arange(128, 256).double() / 128
    e = 2.0 ** -torch.arange(1, 21).double()
    x = m[None, None, :] * e[None, :, None] * torch.ones(128, 1, 1)     # [a, e, m]
    x = torch.cat([x[..., :64], a[:, None, None].expand(128, 20, 1), -x[..., 64:],
                   torch.zeros(128, 20, 127)], 2).reshape(-1, 256)
    x[:, 255] = x[:, 64]                                                # (its own block's maximum)
    x[:, 129:255] = -x[:, 1:127]
    x = x.bfloat16().cuda()
    codes, scales = blockscale_quantize(x)
    want_c, want_s = ref_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.double().cpu().numpy(), want_c)


def test_quantize_non_finite_blocks_are_nan():
    from moe_expert_layer_histogram_gb300 import blockscale_quantize
    x = draw_x(4, 300, 1)
    x[0, 5], x[1, 200], x[2, 299] = float("inf"), float("nan"), -float("inf")
    codes, scales = blockscale_quantize(x)
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(torch.isnan(scales), bad)
    want = bad.t().repeat_interleave(128, 1)[:, :300]
    assert torch.equal(torch.isnan(codes.float()), want)


def test_quantize_gathers_slots_and_strided_rows():
    from moe_expert_layer_histogram_gb300 import blockscale_quantize
    big = draw_x(20, 500, 2)
    for x in (big[:, :384], big[:, 3:388], big[:, 8:264], big[::2, 1:130]):
        n = x.shape[0]
        slots = torch.randint(0, 4 * n, (53,), dtype=torch.int32)
        codes, scales = blockscale_quantize(x, slots.cuda(), 4)
        c2, s2 = blockscale_quantize(x[(slots.long() // 4).cuda()].contiguous())
        assert torch.equal(codes.float(), c2.float()) and torch.equal(scales, s2)
    slots = torch.tensor([0, -1, 19, 20, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    codes, scales = blockscale_quantize(big, slots, 1)
    assert not bool(codes[[1, 3, 4, 5]].float().any()) and not bool(scales[:, [1, 3, 4, 5]].any())
    assert bool(codes[[0, 2]].float().any(1).all())


# ---------------------------------------------------------------- product
SIZES = [(1, 1, 1), (1, 128, 128), (1, 300, 1024), (2, 7, 129), (3, 64, 16), (5, 513, 2064),
         (15, 100, 100), (16, 127, 127), (17, 128, 500), (31, 129, 144), (33, 255, 640),
         (64, 256, 384), (65, 257, 1000), (127, 96, 256), (128, 128, 128), (129, 384, 130),
         (200, 1001, 272), (300, 320, 2000), (513, 64, 400), (1, 1024, 7168), (40, 72, 3000),
         (700, 520, 528)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_matches_64_bits(M, N, K):
    from moe_expert_layer_histogram_gb300 import blockscale_linear, blockscale_quantize
    x = draw_x(M, K, M + N + K)
    w, s = draw_w(1, N, K, N)
    codes, scales = blockscale_quantize(x)
    out = blockscale_linear(x, w[0], s[0])
    assert_product(out, *product_ref(codes, scales, w[0], s[0]), K)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_dx_matches_64_bits(M, N, K):
    # dy [M, N], w [N, K]: the reduction runs over N
    from moe_expert_layer_histogram_gb300 import blockscale_linear_dx, blockscale_quantize
    dy = draw_x(M, N, M + N + K + 1, 0.01)
    w, s = draw_w(1, N, K, N + 1)
    codes, scales = blockscale_quantize(dy)
    out = blockscale_linear_dx(dy, w[0], s[0])
    a, b = dequant_rows(codes, scales).cpu(), dequant_weight(w[0], s[0]).cpu()
    assert_product(out, a @ b, a.abs() @ b.abs(), N)


# enough 256-column items for every SM: the wide kernels, in CTA pairs and alone
LARGE = [(2570, 2000, 272), (4900, 1030, 130), (2561, 4100, 400), (130, 39000, 144)]


@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_products_match_64_bits(M, N, K):
    from moe_expert_layer_histogram_gb300 import (blockscale_linear, blockscale_linear_dx,
                                                  blockscale_quantize)
    x = draw_x(M, K, M + N + K)
    w, s = draw_w(1, N, K, N)
    codes, scales = blockscale_quantize(x)
    assert_product(blockscale_linear(x, w[0], s[0]), *product_ref(codes, scales, w[0], s[0]), K)
    w, s = draw_w(1, K, N, N)                  # the reduction along the stored rows
    out = blockscale_linear_dx(x, w[0], s[0])
    a, b = dequant_rows(codes, scales).cpu(), dequant_weight(w[0], s[0]).cpu()
    assert_product(out, a @ b, a.abs() @ b.abs(), K)


def test_gradient_against_differences():
    # Rows whose blocks quantise exactly (multiples of 2^-3 up to 14 with 14
    # in every block: s = 2^-5, codes are e4m3 values), so y is linear in x:
    # <dy, y(x + d) - y(x)> = <dx, d>.
    from moe_expert_layer_histogram_gb300 import blockscale_linear, blockscale_linear_dx
    M, N, K = 24, 200, 300
    g = torch.Generator().manual_seed(5)
    w, s = draw_w(1, N, K, 9)
    s = torch.full_like(s, 2.0 ** -9)

    def exact_rows(cols):
        v = torch.randint(-7, 8, (M, cols), generator=g).float()
        v[:, ::128] = 14.0
        return v

    dy = exact_rows(N)
    x0, x1 = exact_rows(K), exact_rows(K)
    y0, y1 = (blockscale_linear(v.bfloat16().cuda(), w[0], s[0]).double().cpu() for v in (x0, x1))
    dx = blockscale_linear_dx(dy.bfloat16().cuda(), w[0], s[0]).double().cpu()
    lhs = (dy.double() * (y1 - y0)).sum()
    rhs = (dx * (x1 - x0).double()).sum()
    # each y and dx is rounded to bf16 once: 2^-8 of its terms
    tol = 2.0 ** -8 * ((dy.double().abs() * (y1.abs() + y0.abs())).sum()
                       + (dx.abs() * (x1 - x0).double().abs()).sum())
    assert abs(float(lhs - rhs)) <= float(tol)
    assert abs(float(rhs)) > 0


def test_strides_and_unaligned_outputs():
    from moe_expert_layer_histogram_gb300 import blockscale_linear
    big = draw_x(70, 700, 3)
    w, s = draw_w(1, 130, 321, 4, ldw=352)
    x = big[:, 5:326]
    want = blockscale_linear(x.contiguous(), w[0], s[0])
    for start, width in ((0, 130), (1, 150), (3, 137), (8, 144)):
        store = torch.full((70, width + 9), 7.0, dtype=torch.bfloat16, device="cuda")
        blockscale_linear(x, w[0], s[0], out=store[:, start:start + 130])
        torch.cuda.synchronize()
        assert torch.equal(store[:, start:start + 130], want)
        assert bool((store[:, :start] == 7).all()) and bool((store[:, start + 130:] == 7).all())


def test_nan_stays_in_its_row_and_block():
    from moe_expert_layer_histogram_gb300 import blockscale_linear
    x = draw_x(140, 256, 3)
    w, s = draw_w(1, 200, 256, 4)
    want = blockscale_linear(x, w[0], s[0])
    x[3, 7] = float("inf")
    x[133, 255] = float("nan")
    got = blockscale_linear(x, w[0], s[0])
    keep = [m for m in range(140) if m not in (3, 133)]
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[133]).all())


# ---------------------------------------------------------------- grouped
def offsets_of(counts, first=0):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    return (off + first).cuda()


GROUPS = [[700, 0, 513, 1, 1500, 129, 257, 640], [1025, 128, 1], [0, 5, 1, 0, 130, 17, 0],
          [1, 1, 1, 1], [128, 129, 127, 256], [0, 0, 0, 3], [300, 0, 0, 1], [2] * 40,
          [0] * 511 + [9], [33, 64, 65, 31, 32, 16, 15], [2100, 77], [1, 3300, 129], [0, 2049],
          [30, 0, 34], [1] * 3 + [0] * 5, [63], [0, 16, 0, 0], [8, 8], [3, 14]]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: "E%d_M%d" % (len(c), sum(c)))
def test_grouped_matches_64_bits(counts, transpose):
    from moe_expert_layer_histogram_gb300 import blockscale_matmul, blockscale_quantize
    E, M, N, K = len(counts), sum(counts), 144, 272
    N = 1552 if M > 1000 else N                # wide items
    w, s = draw_w(E, *((K, N) if transpose else (N, K)), seed=E)
    codes, scales = blockscale_quantize(draw_x(M, K, M))
    off = offsets_of(counts)
    out = blockscale_matmul(codes, scales, w, s, off, transpose_w=transpose)
    r = 0
    a = dequant_rows(codes, scales).cpu()
    for e, c in enumerate(counts):
        b = dequant_weight(w[e], s[e]).cpu()
        b = b if transpose else b.t()
        assert_product(out[r:r + c], a[r:r + c] @ b, a[r:r + c].abs() @ b.abs(), K)
        r += c


def test_rows_of_no_expert_are_left_alone():
    from moe_expert_layer_histogram_gb300 import blockscale_matmul, blockscale_quantize
    w, s = draw_w(3, 160, 256, 2)
    codes, scales = blockscale_quantize(draw_x(60, 256, 2))
    want = blockscale_matmul(codes, scales, w, s, offsets_of([20, 20, 20]))
    out = torch.full((60, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    blockscale_matmul(codes, scales, w, s, torch.tensor([4, 20, 40, 50], dtype=torch.int32).cuda(),
                      out=out)
    assert torch.equal(out[4:50], want[4:50])
    assert bool((out[:4] == 7).all()) and bool((out[50:] == 7).all())


def test_bad_offsets_stay_in_range():
    from moe_expert_layer_histogram_gb300 import blockscale_matmul, blockscale_quantize
    w, s = draw_w(4, 130, 256, 2)
    codes, scales = blockscale_quantize(draw_x(60, 256, 2))
    for off in ([-5, 10, 8, 40, 2000], [70, 80, 90, 100, 110], [2 ** 31 - 1, -2 ** 31, 5, 3, 60]):
        store = torch.full((62, 130), 7.0, dtype=torch.bfloat16, device="cuda")
        blockscale_matmul(codes, scales, w, s, torch.tensor(off, dtype=torch.int32).cuda(),
                          out=store[1:61])
        torch.cuda.synchronize()
        assert bool((store[0] == 7).all()) and bool((store[61] == 7).all())


# ---------------------------------------------------------------- SwiGLU
def swiglu_ref(a, w13, s13, clamp):
    gu = a @ dequant_weight(w13, s13).cpu().t()
    if clamp:
        gu = gu.clamp(-clamp, clamp)
    I = gu.shape[1] // 2
    return gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]


@pytest.mark.parametrize("clamp", [0.0, 1.5])
@pytest.mark.parametrize("counts,I,K", [([1], 128, 128), ([7, 0, 20], 256, 400),
                                        ([0, 129, 1, 64], 384, 272), ([300, 33], 128, 1040),
                                        ([2] * 20, 640, 256), ([600, 257, 0, 300], 256, 272),
                                        ([1025], 384, 400), ([64], 256, 1040), ([37], 128, 528),
                                        ([65], 256, 1040), ([2500, 300], 256, 272),
                                        ([5, 3200, 0], 128, 144), ([1, 0, 1, 3], 256, 1040),
                                        ([0, 9, 4], 256, 528), ([16, 0, 1], 256, 528), ([1, 0, 0, 0, 0, 0, 1], 128, 2000)])
def test_swiglu_codes(counts, I, K, clamp):
    from moe_expert_layer_histogram_gb300 import blockscale_quantize, moe_blockscale_swiglu
    E, M = len(counts), sum(counts)
    w, s = draw_w(E, 2 * I, K, E)
    # gate and up of order one: a K-term sum of order sqrt(K) * 60 * 2^-9
    s = s * (8.5 / K ** 0.5)
    codes, scales = blockscale_quantize(draw_x(M, K, M))
    h = torch.empty(M, I, dtype=torch.float8_e4m3fn, device="cuda")
    hs = torch.empty(I // 128, M, device="cuda")
    moe_blockscale_swiglu(codes, codes.stride(0), scales, M, w, w.stride(1), s, offsets_of(counts),
                          E, M, I, K, clamp, h, I, hs, M, torch.cuda.current_stream().cuda_stream)
    a = dequant_rows(codes, scales).cpu()
    r = flips = 0
    for e, c in enumerate(counts):
        if c:
            ref = swiglu_ref(a[r:r + c], w[e], s[e], clamp).numpy()
            amax = np.abs(ref.reshape(c, -1, 128)).max(2)
            got_s = hs[:, r:r + c].double().cpu().numpy().T
            assert np.all(np.abs(got_s - amax / 448) <= 2.0 ** -13 * amax / 448)
            q = ref / np.repeat(got_s, 128, 1)
            want = round_e4m3(q)
            got = h[r:r + c].double().cpu().numpy()
            step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -30))), -6) - 3)
            assert np.all(np.abs(got - want) <= 2 * step)
            assert np.all(np.abs(got - q) <= 0.51 * 2 * step)
            flips += int((got != want).sum())
        r += c
    assert flips <= max(2, M * I * 2.0 ** -8)


def test_swiglu_non_finite_rows():
    from moe_expert_layer_histogram_gb300 import blockscale_quantize, moe_blockscale_swiglu
    w, s = draw_w(1, 512, 256, 3)
    x = draw_x(6, 256, 1)
    x[2, 3] = float("inf")
    codes, scales = blockscale_quantize(x)
    h = torch.empty(6, 256, dtype=torch.float8_e4m3fn, device="cuda")
    hs = torch.empty(2, 6, device="cuda")
    moe_blockscale_swiglu(codes, 256, scales, 6, w, 256, s, None, 1, 6, 256, 256, 0.0, h, 256, hs,
                          6, torch.cuda.current_stream().cuda_stream)
    assert bool(torch.isnan(hs[:, 2]).all()) and bool(torch.isnan(h[2].float()).all())
    keep = [0, 1, 3, 4, 5]
    assert bool(torch.isfinite(hs[:, keep]).all()) and bool(torch.isfinite(h[keep].float()).all())


# ---------------------------------------------------------------- experts
@pytest.mark.parametrize("T,E,topk,H,I,clamp", [(1, 8, 2, 256, 128, 0.0), (5, 16, 4, 400, 256, 0.0),
                                                (64, 8, 2, 512, 256, 7.0), (300, 4, 2, 384, 384, 0.0),
                                                (40, 64, 6, 640, 128, 1.0)])
def test_experts_match_64_bits(T, E, topk, H, I, clamp):
    # relative L2: bf16's rounding (at most 2^-8 = 4e-3) and at most 2^-8 of
    # h's codes one step (at most 2^-3 of the value) off: 2^-3 * 2^-4 = 8e-3
    from moe_expert_layer_histogram_gb300 import (blockscale_experts, blockscale_quantize,
                                                  moe_route_permute_static)
    x = draw_x(T, H, T)
    w13, s13 = draw_w(E, 2 * I, H, 1)
    w2, s2 = draw_w(E, H, I, 2)
    s13 = s13 * (8.5 / H ** 0.5)
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=g).cuda()
    ids = torch.empty(T, topk, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, topk, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    moe_route_permute_static(logits, T, E, topk, ids, wt, off, perm,
                             torch.cuda.current_stream().cuda_stream)
    y = blockscale_experts(x, perm, off, topk, w13, s13, w2, s2, clamp=clamp)
    codes, scales = blockscale_quantize(x, perm, topk)
    a, o = dequant_rows(codes, scales).cpu(), off.tolist()
    ref = torch.zeros(T * topk, H, dtype=torch.float64)
    for e in range(E):
        if o[e] < o[e + 1]:
            h = swiglu_ref(a[o[e]:o[e + 1]], w13[e], s13[e], clamp).numpy()
            s = (np.abs(h.reshape(h.shape[0], -1, 128)).max(2) / 448).repeat(128, 1)
            hq = torch.from_numpy(round_e4m3(h / s) * s)
            ref[o[e]:o[e + 1]] = hq @ dequant_weight(w2[e], s2[e]).cpu().t()
    err = float((y.double().cpu() - ref).norm() / ref.norm())
    assert err <= 1e-2, err


def _route(T, E, topk, seed):
    from moe_expert_layer_histogram_gb300 import moe_route_permute_static
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g).cuda()
    ids = torch.empty(T, topk, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, topk, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    moe_route_permute_static(logits, T, E, topk, ids, wt, off, perm,
                             torch.cuda.current_stream().cuda_stream)
    return off, perm


@pytest.mark.parametrize("T,E,topk,H,I", [(700, 2, 1, 400, 256), (1500, 3, 2, 272, 128),
                                          (90, 5, 3, 1040, 128)])
def test_experts_however_their_rows_are_gathered(T, E, topk, H, I):
    # all rows against the slices of one
    # expert each, beside an empty one (fewer rows than tokens: gathered by the
    # quantiser), and against the two products called one by one: the same
    # sums in the same order, so the same bits
    from moe_expert_layer_histogram_gb300 import (blockscale_experts, blockscale_matmul,
                                                  blockscale_quantize, moe_blockscale_swiglu)
    x = draw_x(T, H, T)
    w13, s13 = draw_w(E, 2 * I, H, 1)
    w2, s2 = draw_w(E, H, I, 2)
    s13 = s13 * (8.5 / H ** 0.5)
    off, perm = _route(T, E, topk, 7)
    y = blockscale_experts(x, perm, off, topk, w13, s13, w2, s2)
    o = off.tolist()
    for e in range(E):
        n, pick = o[e + 1] - o[e], [e, (e + 1) % E]
        own = torch.tensor([0, n, n], dtype=torch.int32, device="cuda")
        # (indexing drops the padding of the rows, which H is a multiple of 16 without)
        part = blockscale_experts(x, perm[o[e]:o[e + 1]].clone(), own, topk,
                                  w13.view(torch.uint8)[pick].view(torch.float8_e4m3fn), s13[pick],
                                  w2.view(torch.uint8)[pick].view(torch.float8_e4m3fn), s2[pick])
        assert torch.equal(part, y[o[e]:o[e + 1]])
    R = T * topk
    codes, scales = blockscale_quantize(x, perm, topk)
    h = torch.empty(R, I, dtype=torch.float8_e4m3fn, device="cuda")
    hs = torch.empty(I // 128, R, device="cuda")
    moe_blockscale_swiglu(codes, H, scales, R, w13, H, s13, off, E, R, I, H, 0.0, h, I, hs, R,
                          torch.cuda.current_stream().cuda_stream)
    assert torch.equal(blockscale_matmul(h, hs, w2, s2, off), y)


def test_slots_outside_the_tokens_give_zero_rows():
    from moe_expert_layer_histogram_gb300 import blockscale_experts
    T, E, topk, H, I = 40, 4, 2, 256, 128
    x = draw_x(T, H, 1)
    w13, s13 = draw_w(E, 2 * I, H, 1)
    w2, s2 = draw_w(E, H, I, 2)
    off, perm = _route(T, E, topk, 3)
    want = blockscale_experts(x, perm, off, topk, w13, s13, w2, s2)
    bad = perm.clone()
    rows = [0, 5, 33, 79]
    bad[rows] = torch.tensor([-1, T * topk, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = blockscale_experts(x, bad, off, topk, w13, s13, w2, s2)
    keep = [r for r in range(T * topk) if r not in rows]
    assert torch.equal(got[keep], want[keep]) and not bool(got[rows].any())


def test_same_bits_every_time_streams_and_graphs():
    from moe_expert_layer_histogram_gb300 import blockscale_linear
    x = draw_x(37, 1024, 1)
    w, s = draw_w(1, 500, 1024, 2)
    want = blockscale_linear(x, w[0], s[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            assert torch.equal(blockscale_linear(x, w[0], s[0]), want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = blockscale_linear(x, w[0], s[0])
    x2 = draw_x(37, 1024, 5)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, blockscale_linear(x2, w[0], s[0]))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (16, 1024, 2000), (48, 2048, 2048),
                                   (300, 600, 1536)])
def test_many_calls_in_a_row(M, N, K):
    # launches that find the weights in L2 and launches that do not: the copies
    # and the tensor pipe take turns in being first
    from moe_expert_layer_histogram_gb300 import blockscale_linear
    x = draw_x(M, K, 1)
    w, s = draw_w(1, N, K, 2)
    want = blockscale_linear(x, w[0], s[0])
    flush = torch.empty(1 << 27, dtype=torch.int16, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            flush.fill_(i)
        assert torch.equal(blockscale_linear(x, w[0], s[0]), want)


def test_back_to_back_calls_do_not_disturb_each_other():
    # many small dependent calls in a row: each reads what the one before wrote
    from moe_expert_layer_histogram_gb300 import blockscale_linear
    w, s = draw_w(1, 256, 256, 3)
    s = s * (8.5 / 16)
    x = draw_x(3, 256, 1)
    y = x
    for _ in range(50):
        y = blockscale_linear(y, w[0], s[0])
        y = y / y.float().abs().amax().bfloat16()
    z = x
    for _ in range(50):
        z = blockscale_linear(z, w[0], s[0])
        torch.cuda.synchronize()
        z = z / z.float().abs().amax().bfloat16()
    assert torch.equal(y, z) and bool(torch.isfinite(y).all())


def test_empty_inputs():
    from moe_expert_layer_histogram_gb300 import (blockscale_experts, blockscale_linear,
                                                  blockscale_linear_dx)
    w, s = draw_w(1, 256, 128, 3)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert blockscale_linear(x, w[0], s[0]).shape == (0, 256)
    dy = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    assert blockscale_linear_dx(dy, w[0], s[0]).shape == (0, 128)
    w2, s2 = draw_w(1, 128, 128, 3)
    y = blockscale_experts(x, torch.empty(0, dtype=torch.int32, device="cuda"),
                           torch.zeros(2, dtype=torch.int32, device="cuda"), 1, w, s, w2, s2)
    assert y.shape == (0, 128)


def test_wrapper_refusals():
    from moe_expert_layer_histogram_gb300 import (MoEError, blockscale_experts, blockscale_linear,
                                                  blockscale_matmul, blockscale_quantize)
    w, s = draw_w(2, 256, 128, 3)
    x = draw_x(4, 128, 0)
    with pytest.raises(ValueError):
        blockscale_linear(x.float(), w[0], s[0])
    with pytest.raises(ValueError):
        blockscale_linear(x[:, :64], w[0], s[0])
    with pytest.raises(ValueError):
        blockscale_linear(x, w[0], s[0, :1])
    with pytest.raises(ValueError):
        blockscale_linear(x, w, s)                              # two experts, no offsets
    with pytest.raises(ValueError):
        blockscale_linear(x, w[0], s[0], out=torch.empty(4, 256, device="cuda"))
    with pytest.raises(MoEError) as e:                          # rows at a stride of 120 bytes
        bad = torch.zeros(256 * 120 + 8, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        blockscale_linear(x[:, :100], bad.as_strided((256, 100), (120, 1)), s[0])
    assert e.value.code == 1
    with pytest.raises(MoEError) as e:                          # codes start at an odd byte
        store = torch.zeros(256 * 128 + 16, dtype=torch.uint8, device="cuda")
        blockscale_linear(x, store.view(torch.float8_e4m3fn)[1:].as_strided((256, 128), (128, 1)),
                          s[0])
    assert e.value.code == 1
    with pytest.raises(MoEError) as e:                          # overlapping rows
        blockscale_linear(x[:1].expand(4, 128), w[0], s[0])
    assert e.value.code == 1
    codes, scales = blockscale_quantize(x)
    with pytest.raises(ValueError):
        blockscale_matmul(codes, scales[:, :3], w[0], s[0])
    with pytest.raises(ValueError):
        blockscale_matmul(codes, scales, w, s, torch.zeros(3, dtype=torch.int64, device="cuda"))
    w2, s2 = draw_w(2, 128, 64, 3)
    with pytest.raises(ValueError):                             # I = 64
        blockscale_experts(x, torch.zeros(4, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, dtype=torch.int32, device="cuda"), 1, w[:, :128],
                           s[:, :1].contiguous(), w2, s2)
