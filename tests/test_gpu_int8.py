"""8-bit integer products with a scale per token and per output channel: codes
against the format's definition, products and the experts' MLPs against plain
implementations in 64 bits.

Tolerances.  u = 2^-24.  Products of codes are exact and a sum of K of them is off
by at most K u of the sum of their magnitudes; the two scales add 2 u, the store
2^-8 of the result.  h = silu(gate) up is off by 3 times the gate's and up's
errors and 8 u; its codes may each differ by one step where the quotient lies
within that of a half, so an expert's output is off by at most the steps of the
codes that lie so near (none, a few or, for the test, those that a 64-bit
quotient puts within 1e-4 of a half).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    from moe_expert_layer_histogram_gb300 import moe_int8_status
    assert moe_int8_status() == 0


def randn(*shape, seed=0, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def codes_of(*shape, seed=0, low=-127):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales_of(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    return torch.rand(*shape, generator=g, device="cuda") * 0.01 + 1e-4


def quantized(x):
    """Codes and scales of rows, by the definition (IEEE quotients in fp32)."""
    v = x.float()
    amax = v.abs().amax(1)
    s = torch.where(torch.isfinite(amax), amax / torch.full_like(amax, 127.0), float("nan"))
    q = v / torch.where(s > 0, s, 1.0)[:, None]
    q = torch.where((s > 0)[:, None], torch.round(q).clamp(-127, 127), 0.0)
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 255), (70, 2001), (33, 7168),
                                       (4, 8192), (3, 8200), (2, 30001)])
def test_quantize(rows, cols):
    from moe_expert_layer_histogram_gb300 import int8_quantize
    x = randn(rows, cols, seed=cols)
    codes, s = int8_quantize(x)
    want, ws = quantized(x)
    assert torch.equal(s, ws) and torch.equal(codes.float(), want)
    assert codes.stride(0) % 16 == 0 or rows == 1


def test_quantize_every_half():
    # quotients that lie on halves and next to them: all pairs of significands
    from moe_expert_layer_histogram_gb300 import int8_quantize
    sig = torch.arange(128, 256, device="cuda", dtype=torch.float32)
    x = torch.cat([sig[:, None], sig[None].repeat(128, 1) / 2, -sig[None].repeat(128, 1) / 4,
                   sig[None].repeat(128, 1) / 64], 1).bfloat16()
    for scale in (1.0, 2.0 ** -100, 2.0 ** 100):
        codes, s = int8_quantize((x.float() * scale).bfloat16())
        want, ws = quantized((x.float() * scale).bfloat16())
        assert torch.equal(s, ws) and torch.equal(codes.float(), want)


def test_quantize_special_rows():
    from moe_expert_layer_histogram_gb300 import int8_quantize
    x = randn(6, 300)
    x[1] = 0
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    x[4] = 2.0 ** -133                      # the smallest bf16 numbers
    codes, s = int8_quantize(x)
    want, ws = quantized(x)
    assert float(s[1]) == 0 and bool(torch.isnan(s[2:4]).all())
    assert bool((codes[1:4] == 0).all())
    keep = [0, 4, 5]
    assert torch.equal(s[keep], ws[keep]) and torch.equal(codes[keep].float(), want[keep])


def test_quantize_by_slots_and_strides():
    from moe_expert_layer_histogram_gb300 import int8_quantize
    big = randn(20, 100)
    slots = torch.tensor([3, 0, 59, 7, 60, -1, 2 ** 31 - 1, 31], dtype=torch.int32, device="cuda")
    for x in (big[:, :96], big[:, 1:98], big[:, 4:68]):
        codes, s = int8_quantize(x, slots, 3)
        for r, slot in enumerate(slots.tolist()):
            if 0 <= slot < 60:
                want, ws = quantized(x[slot // 3:slot // 3 + 1])
                assert torch.equal(codes[r].float(), want[0]) and float(s[r]) == float(ws[0])
            else:
                assert bool((codes[r] == 0).all()) and float(s[r]) == 0


def matmul_reference(a, s, w, ws, offsets=None):
    """(result, the magnitudes of its terms) in 64 bits."""
    if offsets is None:
        scale = s.double()[:, None] * ws.double()
        return (a.double() @ w.double().t()) * scale, (a.double().abs() @ w.double().abs().t()) * scale
    M, N = a.shape[0], w.shape[1]
    out = torch.full((M, N), float("nan"), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    last = 0
    for e in range(w.shape[0]):
        r0 = min(max(offsets[e], last, 0), M)
        last = max(last, offsets[e])
        r1 = min(max(offsets[e + 1], r0), M)
        if r1 > r0:
            out[r0:r1], mag[r0:r1] = matmul_reference(a[r0:r1], s[r0:r1], w[e], ws[e])
    return out, mag


def close(got, want, mag, K):
    tol = (K + 4) * U * mag
    tol = tol + BF16 * (want.abs() + tol)
    err = (got.double() - want).abs()
    assert bool((err <= tol + 1e-30).all()), float((err - tol).max())


SHAPES = [(1, 1, 16), (1, 4096, 7168), (2, 256, 128), (3, 300, 48), (16, 257, 130), (17, 1001, 2000),
          (33, 512, 1024), (64, 640, 4096), (65, 255, 144), (128, 256, 512), (129, 1000, 272),
          (333, 1001, 2000), (500, 3000, 64), (1300, 2100, 1040), (2048, 4096, 256), (40, 20000, 32)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K):
    from moe_expert_layer_histogram_gb300 import int8_matmul
    ld = (K + 15) // 16 * 16
    a, w = codes_of(M, K, seed=1), codes_of(N, ld, seed=2)[:, :K]
    s, ws = scales_of(M), scales_of(N, seed=1)
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    got = int8_matmul(a, s, w, ws, out=out[1:M + 1])
    assert torch.equal(out[0], out[-1]) and bool((out[0] == 7).all())
    close(got, *matmul_reference(a, s, w, ws), K)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 33), (130, 512), (257, 1000), (1001, 2500),
                                 (64, 20000), (300, 4113)])
def test_few_rows(M, N, K):
    from moe_expert_layer_histogram_gb300 import int8_linear, int8_matmul, int8_quantize
    ld = (K + 15) // 16 * 16
    flat = codes_of((N - 1) * ld + K, seed=2)               # (nothing behind the last row)
    w, ws = torch.as_strided(flat, (N, K), (ld, 1)), scales_of(N)
    if N == 1:
        w = flat.view(1, K)
    for lead in (0, 3):
        a, s = codes_of(M, K + 5 + lead, seed=1)[:, lead:lead + K], scales_of(M)
        got = int8_matmul(a, s, w, ws)
        want, mag = matmul_reference(a, s, w, ws)
        close(got, want, mag, K)
        x = randn(M, K + 8 + lead)[:, lead:lead + K]
        assert torch.equal(int8_linear(x, w, ws), int8_matmul(*int8_quantize(x), w, ws))


def test_few_rows_of_the_largest_codes():
    # 131072 products of 127 x -128: int32 sums at their limit, then fp32 ones
    from moe_expert_layer_histogram_gb300 import int8_matmul
    for K in (131072, 131088):
        for M in (1, 8):
            a = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
            w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
            got = int8_matmul(a, torch.ones(M, device="cuda"), w, torch.ones(5, device="cuda"))
            want = torch.full((M, 5), -127.0 * 128 * K, dtype=torch.float64, device="cuda")
            close(got, want, -want, K)


@pytest.mark.parametrize("K", [131056, 131072, 131088])
@pytest.mark.parametrize("M", [1, 4, 5])
def test_largest_sums(M, K):
    # K products of -128 x -128, 2^31 of them at K = 2^17; every partial sum is a
    # multiple of 2^14 below 2^38, so exact in fp32
    from moe_expert_layer_histogram_gb300 import int8_matmul
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    got = int8_matmul(a, torch.ones(M, device="cuda"), w, torch.ones(5, device="cuda"))
    assert torch.equal(got, torch.full((M, 5), 16384.0 * K, device="cuda").bfloat16())


@pytest.mark.parametrize("M,N,K", [(4864, 1024, 400), (5000, 1025, 130), (9728, 500, 64),
                                   (2049, 9800, 1000), (20000, 256, 16)])
def test_matmul_of_many_rows(M, N, K):
    test_matmul(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 300, 1008), (100, 300, 1008), (400, 300, 1008),
                                   (5000, 1000, 1008)])
def test_sums_that_fp32_holds_are_exact(M, N, K):
    # scales 1 and at most 1008 products of up to 127 x 128: whole numbers below 2^24,
    # so the result is the exact sum rounded to bf16
    from moe_expert_layer_histogram_gb300 import int8_matmul
    a, w = codes_of(M, K, seed=3), codes_of(N, K, seed=4, low=-128)
    got = int8_matmul(a, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"))
    want = a.double() @ w.double().t()
    assert torch.equal(got, want.float().bfloat16())


@pytest.mark.parametrize("offset,ldo", [(0, 301), (1, 302), (2, 304), (0, 320)])
def test_results_of_any_alignment(offset, ldo):
    from moe_expert_layer_histogram_gb300 import int8_matmul
    for M in (5, 200, 700):
        N, K = 301, 256
        a, w = codes_of(M, K, seed=5), codes_of(N, K, seed=6)
        s, ws = scales_of(M), scales_of(N, seed=1)
        flat = torch.full((M * ldo + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = torch.as_strided(flat, (M, N), (ldo, 1), offset)
        keep = torch.ones_like(flat, dtype=torch.bool)
        torch.as_strided(keep, (M, N), (ldo, 1), offset).fill_(False)
        int8_matmul(a, s, w, ws, out=out)
        close(out, *matmul_reference(a, s, w, ws), K)
        assert bool((flat[keep] == 7).all())


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (7, 100, 130), (333, 1001, 2000), (1000, 512, 512)])
@pytest.mark.parametrize("lead", [0, 1])
def test_linear(M, N, K, lead):
    from moe_expert_layer_histogram_gb300 import int8_linear, int8_matmul, int8_quantize
    ld = (K + 15) // 16 * 16
    x, w, ws = randn(M, K + lead)[:, lead:], codes_of(N, ld, seed=2)[:, :K], scales_of(N)
    got = int8_linear(x, w, ws)
    q, s = quantized(x)
    close(got, *matmul_reference(q, s, w, ws), K)
    assert torch.equal(got, int8_matmul(*int8_quantize(x), w, ws))


GROUPS = [
    ([0, 5, 5, 130, 131, 400, 400, 433, 433], 433),
    ([0, 1, 1, 2, 2, 3, 3, 3, 3], 3),                 # a token: split
    ([0, 0, 0, 0, 0, 0, 0, 0, 0], 6),                 # rows of no expert only
    ([10, 20, 300, 300, 300, 310, 310, 320, 325], 330),
    ([-5, 20, 15, 60, 2 ** 31 - 1, 7, 80, 90, 100], 64),   # not a table: clamped
    ([0, 1200, 1200, 2500, 2500, 2500, 2600, 2601, 2700], 2700),
    ([0, 257, 257, 258, 513, 4000, 12001, 19990, 20001], 20010),
]


@pytest.mark.parametrize("offsets,M", GROUPS)
@pytest.mark.parametrize("N,K", [(256, 512), (333, 144), (1300, 272)])
def test_experts_rows(offsets, M, N, K):
    from moe_expert_layer_histogram_gb300 import int8_matmul
    E = len(offsets) - 1
    a, w = codes_of(M, K, seed=7), codes_of(E, N, K, seed=8)
    s, ws = scales_of(M), scales_of(E, N, seed=1)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    int8_matmul(a, s, w, ws, offsets=off, out=out)
    want, mag = matmul_reference(a, s, w, ws, offsets)
    mine = ~torch.isnan(want[:, 0])
    close(out[mine], want[mine], mag[mine], K)
    assert bool((out[~mine] == 7).all())


FEW = [
    (list(range(17)), 16),                            # a row each
    ([0] * 3 + list(range(0, 25)) + [24] * 2, 24), ([0] * 12 + [24] * 13, 24),
    ([0] * 6 + [16] * 11, 16),                        # all rows of one expert
    ([0, 0, 1, 3, 3, 6, 6, 10] + [15] * 10, 16),      # 1, 2, 3, 4 and 5 rows, one of none
    ([4, 4, 5] + [8] * 14, 12),                       # rows of no expert on either side
    ([0] * 17, 1), ([0] * 16 + [1], 1), ([0] * 511 + [1, 2], 2),
    ([5, 3, 9, 2, -1, 2 ** 31 - 1, 7, 11, 20, -2 ** 31, 14, 14, 15, 16, 90, 12, 16], 16),
]


@pytest.mark.parametrize("offsets,M", FEW)
@pytest.mark.parametrize("N,K", [(1, 16), (33, 130), (256, 512), (301, 2500), (90, 7168)])
def test_few_rows_of_experts(offsets, M, N, K):
    from moe_expert_layer_histogram_gb300 import int8_matmul
    E, ld = len(offsets) - 1, (K + 15) // 16 * 16
    w = codes_of(E, N, ld, seed=8, low=-128)[:, :, :K]
    s, ws = scales_of(M), scales_of(E, N, seed=1)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for lead, ldo in ((0, N), (3, N + 5)):
        a = codes_of(M, K + 7, seed=7, low=-128)[:, lead:lead + K]
        out = torch.full((M, ldo), 7.0, dtype=torch.bfloat16, device="cuda")
        int8_matmul(a, s, w, ws, offsets=off, out=out[:, :N])
        want, mag = matmul_reference(a, s, w, ws, offsets)
        mine = ~torch.isnan(want[:, 0])
        close(out[mine][:, :N], want[mine], mag[mine], K)
        assert bool((out[~mine] == 7).all()) and bool((out[:, N:] == 7).all())


def test_experts_of_tokens_quantised_once():
    # 8.4 M codes and more: the same bits as every expert's rows by themselves, also for
    # slots outside the tokens (rows of zeros)
    from moe_expert_layer_histogram_gb300 import int8_experts, int8_matmul, int8_quantize
    T, E, k, H, I = 4200, 4, 4, 512, 144
    x = randn(T, H)
    w13, w2 = codes_of(E, 2 * I, H, seed=1), codes_of(E, H, I, seed=2)
    s13, s2 = scales_of(E, 2 * I) * 0.02, scales_of(E, H, seed=1)
    _, o = route(T, E, k, masked=0.1)
    slots = o.slots.clone()
    slots[3], slots[7], slots[-1] = -1, T * k, 2 ** 31 - 1
    out = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    int8_experts(x, slots, o.offsets, k, w13, s13, w2, s2, out=out)
    live = int(o.offsets[-1])
    codes, scales = int8_quantize(x, slots, k)
    gu = int8_matmul(codes, scales, w13, s13, offsets=o.offsets)[:live]
    assert bool((out[[3, 7]] == 0).all()) and bool((out[live:] == 7).all())
    # h from products rounded to bf16: within 2^-8 of gate and up each, and a code's
    # half step of the largest |h| a row
    gate, up = gu[:, :I].double(), gu[:, I:].double()
    h = gate * torch.sigmoid(gate) * up
    dh = (h.abs() * (1 + gate.abs()) + 1e-30) * 3 * BF16 + h.abs().amax(1, keepdim=True) / 127
    off = o.offsets.tolist()
    for e in range(E):
        a, b = off[e], off[e + 1]
        w = w2[e].double() * s2[e].double()[:, None]
        want, tol = h[a:b] @ w.t(), dh[a:b] @ w.abs().t()
        assert bool(((out[a:b].double() - want).abs() <= tol + BF16 * want.abs() + 1e-30).all())


@pytest.mark.parametrize("T,E,k,H,I,clamp,masked", [
    (1, 64, 8, 7168, 2048, 7.0, 0.0), (1, 2, 1, 16, 16, 0.0, 0.0), (2, 16, 8, 272, 144, 0.5, 0.0),
    (5, 64, 3, 528, 16, 0.0, 0.4), (4, 16, 4, 2048, 1040, 7.0, 0.0), (16, 512, 1, 144, 272, 0.0, 0.0)])
def test_experts_of_few_rows(T, E, k, H, I, clamp, masked):
    test_experts(T, E, k, H, I, clamp, masked)


def route(T, E, k, seed=0, masked=0.0):
    from moe_expert_layer_histogram_gb300 import router_gate, router_order
    mask = None
    if masked:
        mask = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(seed + 9),
                          device="cuda") >= masked
    r = router_gate(randn(T, E, seed=seed, dtype=torch.float32), k, mask=mask)
    return r, router_order(r.ids, E)


@pytest.mark.parametrize("T,E,k,H,I,clamp,masked", [
    (1, 8, 2, 256, 128, 0.0, 0.0), (2, 64, 6, 2048, 1024, 7.0, 0.0), (40, 16, 3, 272, 144, 0.0, 0.2),
    (64, 64, 8, 1024, 512, 0.0, 0.0), (700, 8, 2, 512, 256, 0.5, 0.1), (300, 4, 4, 144, 16, 0.0, 0.0),
    (1500, 8, 4, 256, 400, 7.0, 0.0), (4000, 4, 2, 1024, 720, 0.0, 0.0),
    (6000, 8, 4, 528, 256, 1.0, 0.1)])
def test_experts(T, E, k, H, I, clamp, masked):
    from moe_expert_layer_histogram_gb300 import int8_experts
    x = randn(T, H)
    w13, w2 = codes_of(E, 2 * I, H, seed=1), codes_of(E, H, I, seed=2)
    s13, s2 = scales_of(E, 2 * I) * 0.02, scales_of(E, H, seed=1)
    _, o = route(T, E, k, masked=masked)
    out = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    int8_experts(x, o.slots, o.offsets, k, w13, s13, w2, s2, clamp=clamp, out=out)
    q, s = quantized(x)
    off = o.offsets.tolist()
    rows = o.slots.long() // k
    for e in range(E):
        r = rows[off[e]:off[e + 1]]
        if not len(r):
            continue
        gu, _ = matmul_reference(q[r], s[r], w13[e], s13[e])
        gate, up = gu[:, :I], gu[:, I:]
        if clamp:
            gate, up = gate.clamp(-clamp, clamp), up.clamp(-clamp, clamp)
        h = gate * torch.sigmoid(gate) * up
        sh = h.abs().amax(1) / 127
        quot = h / torch.where(sh > 0, sh, 1.0)[:, None]
        c = torch.round(quot).clamp(-127, 127)
        near = ((quot - torch.floor(quot)) - 0.5).abs() < 1e-4
        want, mag = matmul_reference(c, sh, w2[e], s2[e])
        # (a scale that is off by 1e-5 of itself, and the codes next to a half)
        step = (near.double() @ w2[e].double().abs().t()) * sh[:, None] * s2[e].double()
        got = out[off[e]:off[e + 1]].double()
        tol = step + 1e-5 * mag + (I + 4) * U * mag
        tol = tol + BF16 * (want.abs() + tol)
        err = (got - want).abs()
        assert bool((err <= tol + 1e-30).all()), float((err - tol).max())
    assert bool((out[off[E]:] == 7).all())


def test_rows_with_nan_keep_to_themselves():
    from moe_expert_layer_histogram_gb300 import int8_experts, int8_linear
    x = randn(200, 256)
    w, ws = codes_of(300, 256), scales_of(300)
    good = int8_linear(x, w, ws)
    bad = x.clone()
    bad[3, 5], bad[150, 0] = float("nan"), float("inf")
    got = int8_linear(bad, w, ws)
    other = [t for t in range(200) if t not in (3, 150)]
    assert bool(torch.isnan(got[[3, 150]]).all()) and torch.equal(got[other], good[other])
    w13, w2 = codes_of(2, 256, 256, seed=1), codes_of(2, 256, 128, seed=2)
    s13, s2 = scales_of(2, 256) * 0.02, scales_of(2, 256)
    slots = torch.arange(200, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 120, 200], dtype=torch.int32, device="cuda")
    a = int8_experts(x, slots, off, 1, w13, s13, w2, s2)
    b = int8_experts(bad, slots, off, 1, w13, s13, w2, s2)
    assert bool(torch.isnan(b[[3, 150]]).all()) and torch.equal(a[other], b[other])


def test_same_bits_every_time_on_streams_and_in_graphs():
    from moe_expert_layer_histogram_gb300 import int8_experts, int8_linear
    x = randn(300, 512)
    w, ws = codes_of(1000, 512), scales_of(1000)
    w13, w2 = codes_of(8, 512, 512, seed=1), codes_of(8, 512, 256, seed=2)
    s13, s2 = scales_of(8, 512) * 0.02, scales_of(8, 512)
    _, o = route(300, 8, 2)

    def once():
        return (int8_linear(x, w, ws), int8_linear(x[:4], w, ws),
                int8_experts(x, o.slots, o.offsets, 2, w13, s13, w2, s2))
    want = once()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(once())
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = once()
        graphs.append((g, held))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for _, held in graphs for p, q in zip(held, want))


def test_no_rows():
    from moe_expert_layer_histogram_gb300 import int8_experts, int8_linear, int8_matmul, int8_quantize
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w, ws = codes_of(32, 64), scales_of(32)
    assert int8_linear(x, w, ws).shape == (0, 32)
    assert int8_matmul(*int8_quantize(x), w, ws).shape == (0, 32)
    slots = torch.empty(0, dtype=torch.int32, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = int8_experts(x, slots, off, 2, codes_of(2, 64, 64), scales_of(2, 64), codes_of(2, 64, 32),
                       scales_of(2, 64))
    assert out.shape == (0, 64)


def test_refusals():
    from moe_expert_layer_histogram_gb300 import (MoEError, int8_experts, int8_linear, int8_matmul,
                                                  int8_quantize)
    x, w, ws = randn(8, 64), codes_of(32, 64), scales_of(32)
    with pytest.raises(MoEError):
        int8_linear(x[:, :40].contiguous(), codes_of(32, 40), ws)     # (rows off 16 bytes)
    for bad in (lambda: int8_linear(x, w, ws[:31]), lambda: int8_linear(x.float(), w, ws),
                lambda: int8_linear(x[:, :48], w, ws), lambda: int8_linear(x, w.float(), ws),
                lambda: int8_linear(x, codes_of(2, 32, 64), scales_of(2, 32)),
                lambda: int8_matmul(x, ws, w, ws), lambda: int8_quantize(x.float()),
                lambda: int8_matmul(codes_of(8, 64), scales_of(7), w, ws),
                lambda: int8_matmul(codes_of(8, 64), scales_of(8), codes_of(2, 32, 64),
                                    scales_of(2, 32)),
                lambda: int8_linear(x, w, ws, out=torch.empty(8, 31, dtype=torch.bfloat16,
                                                              device="cuda")),
                lambda: int8_experts(x, torch.zeros(8, dtype=torch.int32, device="cuda"),
                                     torch.zeros(3, dtype=torch.int32, device="cuda"), 1,
                                     codes_of(2, 48, 64), scales_of(2, 48), codes_of(2, 64, 24),
                                     scales_of(2, 64))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("T,k,H,I", [(1, 8, 2048, 512), (3, 8, 272, 144), (24, 1, 7168, 16)])
def test_a_few_tokens_of_no_expert(T, k, H, I):
    # all of a decoding step's tokens masked: no kernel has a row, none leaves before the
    # one ahead of it is over, the result stays as it was, and so do the next calls'
    from moe_expert_layer_histogram_gb300 import int8_experts
    E = 64
    x = randn(T, H)
    w13, w2 = codes_of(E, 2 * I, H, seed=1), codes_of(E, H, I, seed=2)
    s13, s2 = scales_of(E, 2 * I) * 0.02, scales_of(E, H, seed=1)
    slots = torch.arange(T * k, dtype=torch.int32, device="cuda")
    some = torch.arange(E + 1, dtype=torch.int32, device="cuda").clamp(max=T * k)
    want = int8_experts(x, slots, some, k, w13, s13, w2, s2)
    for offsets in (torch.zeros_like(some), torch.full_like(some, T * k)):
        for _ in range(20):
            out = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
            int8_experts(x, slots, offsets, k, w13, s13, w2, s2, out=out)
            got = int8_experts(x, slots, some, k, w13, s13, w2, s2)
            assert bool((out == 7).all()) and torch.equal(got, want)


@pytest.mark.parametrize("rows", [4, 600, 40000])
def test_experts_of_an_empty_x(rows):
    # every slot lies outside: rows of zeros
    from moe_expert_layer_histogram_gb300 import int8_experts
    E, H, I = 4, 256, 128
    w13, w2 = codes_of(E, 2 * I, H, seed=1), codes_of(E, H, I, seed=2)
    slots = torch.arange(rows, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, rows // 4, rows // 2, rows // 2, rows], dtype=torch.int32, device="cuda")
    out = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
    int8_experts(randn(0, H), slots, off, 2, w13, scales_of(E, 2 * I), w2, scales_of(E, H), out=out)
    assert bool((out == 0).all())


def test_gathered_rows_have_the_bits_of_smaller_calls():
    # 8.6 M codes of tokens quantised once, and the same rows quantised for themselves in a
    # call for each expert: 512 products of codes stay below 2^24, so all sums are exact
    # and every kernel gives the same bits
    from moe_expert_layer_histogram_gb300 import int8_experts
    T, E, k, H, I = 4200, 4, 4, 512, 144
    x = randn(T, H)
    w13, w2 = codes_of(E, 2 * I, H, seed=1), codes_of(E, H, I, seed=2)
    s13, s2 = scales_of(E, 2 * I) * 0.02, scales_of(E, H, seed=1)
    _, o = route(T, E, k, masked=0.1)
    slots = o.slots.clone()
    slots[3], slots[7], slots[-1] = -1, T * k, 2 ** 31 - 1
    out = int8_experts(x, slots, o.offsets, k, w13, s13, w2, s2)
    off = o.offsets.tolist()
    for e in range(E):
        for a in range(off[e], off[e + 1], 1000):
            part = slots[a:min(a + 1000, off[e + 1])]
            own = torch.full((E + 1,), len(part), dtype=torch.int32, device="cuda")
            own[:e + 1] = 0
            got = int8_experts(x, part, own, k, w13, s13, w2, s2)
            assert torch.equal(got, out[a:a + len(part)])


@pytest.mark.parametrize("T,E,k", [(2, 16, 8), (20, 1, 1), (100, 4, 2), (9800, 1, 1), (5000, 4, 4)])
def test_codes_of_h(T, E, k):
    # With the unit matrix for w2 an output is a code of h times its row's scale; in bf16
    # it is off by at most 127 2^-8 < 1/2 of that scale, so the code can be told.  Sums of
    # 1024 products of codes are exact.  Gate and up are off by 2 u of themselves (their
    # scales), the power by (4 + |g|) u, the quotient by 4 u, the product by u: h by
    # (13 + 3 |g|) u, at most 34 u with |g| <= 7, its scale by 2 u more.  So a quotient is
    # off by 127 * 70 u, and codes are those of 64 bits unless it lies as near to a half.
    from moe_expert_layer_histogram_gb300 import int8_experts
    H, I, clamp = 1024, 256, 7.0
    x = randn(T, H)
    w13 = codes_of(E, 2 * I, H, seed=1)
    s13 = scales_of(E, 2 * I) * 0.2
    w2 = torch.zeros(E, H, I, dtype=torch.int8, device="cuda")
    w2[:, torch.arange(I), torch.arange(I)] = 1
    _, o = route(T, E, k)
    out = int8_experts(x, o.slots, o.offsets, k, w13, s13, w2, torch.ones(E, H, device="cuda"),
                       clamp=clamp)
    assert bool((out[:, I:] == 0).all())
    q, s = quantized(x)
    off, rows = o.offsets.tolist(), o.slots.long() // k
    for e in range(E):
        r = rows[off[e]:off[e + 1]]
        gu, _ = matmul_reference(q[r], s[r], w13[e], s13[e])
        gate, up = gu[:, :I].clamp(-clamp, clamp), gu[:, I:].clamp(-clamp, clamp)
        h = gate * torch.sigmoid(gate) * up
        sh = h.abs().amax(1, keepdim=True) / 127
        quot = h / sh
        got = torch.round(out[off[e]:off[e + 1], :I].double() / sh)
        near = ((quot - torch.floor(quot)) - 0.5).abs() <= 127 * 70 * U
        assert bool((near | (got == torch.round(quot))).all())
        assert bool(((got - quot).abs() <= 0.5 + 127 * 70 * U).all())
        assert not near.numel() or float(near.double().mean()) < 0.01


@pytest.mark.parametrize("M,N,K", [(128, 2048, 8192), (100, 4096, 4096), (300, 4096, 7168), (69, 1995, 5756),
                                   (131, 2146, 4540), (1296, 23, 5388), (5236, 16, 1824), (64, 640, 8192),
                                   (33, 4096, 8192), (16, 4096, 7168), (2000, 2000, 5000), (6000, 3000, 2500)])
def test_many_blocks_of_reduction_give_the_same_bits_every_time(M, N, K):
    # codes of +-31: at most 8192 * 31^2 < 2^23, so every partial sum is exact in fp32.  The
    # rings go round several times in each CTA; a stage filled again too early shows as
    # wrong channels in some of the calls
    from moe_expert_layer_histogram_gb300 import int8_matmul
    g = torch.Generator(device="cuda").manual_seed(K)
    ld = (K + 15) // 16 * 16
    a = torch.randint(-31, 32, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-31, 32, (N, ld), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    s, ws = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    want = (a.double() @ w.double().t()).float().bfloat16()
    bad = sum(not torch.equal(int8_matmul(a, s, w, ws), want) for _ in range(60))
    assert bad == 0


@pytest.mark.parametrize("T,H,I", [(128, 4096, 1024), (100, 4096, 528), (70, 2048, 1024)])
def test_one_expert_of_long_rows_has_the_bits_of_smaller_calls(T, H, I):
    # tokens' codes of +-127 and weights of +-31: 4096 * 127 * 31 < 2^24, exact sums
    from moe_expert_layer_histogram_gb300 import int8_experts
    g = torch.Generator(device="cuda").manual_seed(H)
    x = randn(T, H)
    w13 = torch.randint(-31, 32, (1, 2 * I, H), generator=g, device="cuda", dtype=torch.int8)
    w2 = torch.randint(-31, 32, (1, H, I), generator=g, device="cuda", dtype=torch.int8)
    s13, s2 = scales_of(1, 2 * I) * 0.02, scales_of(1, H, seed=1)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")

    def run(a, b):
        off = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        return int8_experts(x, slots[a:b].contiguous(), off, 1, w13, s13, w2, s2)
    want = torch.cat([run(a, min(a + 16, T)) for a in range(0, T, 16)])
    for _ in range(60):
        assert torch.equal(run(0, T), want)


@pytest.mark.parametrize("M", [1, 3, 40])
@pytest.mark.parametrize("K", [1, 33, 250])
def test_one_channel_of_any_width(M, K):
    from moe_expert_layer_histogram_gb300 import int8_linear, int8_matmul, int8_quantize
    flat = torch.cat([codes_of(K, seed=2), torch.full((64,), 127, dtype=torch.int8, device="cuda")])
    w, ws = flat[:K].view(1, K), scales_of(1)
    a, s = codes_of(M, K, seed=1), scales_of(M)
    close(int8_matmul(a, s, w, ws), *matmul_reference(a, s, w, ws), K)
    x = randn(M, K)
    assert torch.equal(int8_linear(x, w, ws), int8_matmul(*int8_quantize(x), w, ws))


@pytest.mark.parametrize("E,M,N,K,rows", [(16, 5552, 4269, 9304, 1), (8, 3500, 2100, 9000, 1),
                                          (8, 3500, 2100, 9000, 40), (4, 2900, 4100, 5000, 130)])
def test_pairs_of_few_rows_wait_for_their_weights(E, M, N, K, rows):
    # experts of few rows in a call of many: weights come out of HBM more slowly than they
    # are used, and not in order.  Codes of +-31: exact sums (9304 * 31^2 < 2^24)
    from moe_expert_layer_histogram_gb300 import int8_matmul
    g = torch.Generator(device="cuda").manual_seed(K)
    ld = (K + 15) // 16 * 16
    a = torch.randint(-31, 32, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-31, 32, (E, N, ld), generator=g, device="cuda", dtype=torch.int8)[:, :, :K]
    s, ws = torch.ones(M, device="cuda"), torch.ones(E, N, device="cuda")
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * rows
    want = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        part = a[e * rows:(e + 1) * rows].double() @ w[e].double().t()
        want[e * rows:(e + 1) * rows] = part.float().bfloat16()
    out = torch.full_like(want, 7.0)
    for _ in range(60):
        int8_matmul(a, s, w, ws, offsets=off, out=out)
        assert torch.equal(out, want)
        out[:E * rows] = 0
