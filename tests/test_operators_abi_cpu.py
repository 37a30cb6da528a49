"""Argument checks of the router-balance and block-scaled FP8 entry points:
every refusal is found on the host before any CUDA call, so these run without
a GPU."""
import pytest

GOOD = 1 << 20
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from moe_expert_layer_histogram_gb300 import _build
    _build.build()
    import moe_expert_layer_histogram_gb300 as m
    return m.lib()


def forward(lib, **over):
    a = dict(logits=GOOD, dtype=0, ld=64, mask=None, T=32, E=64, K=6, coef=0.1, ids=GOOD,
             weights=GOOD, counts=GOOD, mean=GOOD, loss=GOOD, ws=GOOD, nbytes=1 << 30)
    a.update(over)
    return lib.moe_balance_forward(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID),
    (dict(ld=63), INVALID), (dict(dtype=2), INVALID), (dict(logits=None), INVALID),
    (dict(logits=GOOD + 2), INVALID), (dict(dtype=1, logits=GOOD + 1), INVALID),
    (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(counts=None), INVALID),
    (dict(loss=None), INVALID), (dict(ws=None), INVALID), (dict(ids=GOOD + 2), INVALID),
    (dict(weights=GOOD + 1), INVALID), (dict(counts=GOOD + 3), INVALID),
    (dict(mean=GOOD + 2), INVALID), (dict(loss=GOOD + 2), INVALID), (dict(ws=GOOD + 8), INVALID),
    (dict(nbytes=15), INVALID), (dict(T=4096, nbytes=100), INVALID),
    (dict(E=513, ld=513), UNSUPPORTED), (dict(K=17), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED)])
def test_balance_forward_refusals(lib, over, code):
    assert forward(lib, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(ld_d=63), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(counts=None), INVALID), (dict(d_logits=None), INVALID), (dict(ids=GOOD + 1), INVALID),
    (dict(d_loss=GOOD + 2), INVALID), (dict(d_weights=GOOD + 2), INVALID),
    (dict(d_logits=GOOD + 2), INVALID), (dict(E=600, ld=600, ld_d=600), UNSUPPORTED),
    (dict(T=0, logits=None, ids=None), 0)])
def test_balance_backward_refusals(lib, over, code):
    a = dict(logits=GOOD, dtype=0, ld=64, T=32, E=64, K=6, coef=0.1, ids=GOOD, weights=GOOD,
             counts=GOOD, d_loss=GOOD, d_weights=GOOD, d_logits=GOOD, ld_d=64)
    a.update(over)
    assert lib.moe_balance_backward(*a.values(), None) == code


def test_balance_workspace(lib):
    assert lib.moe_balance_workspace(-1, 8) == 0 and lib.moe_balance_workspace(8, 0) == 0
    assert lib.moe_balance_workspace(8, 513) == 0
    small, large = lib.moe_balance_workspace(1, 8), lib.moe_balance_workspace(1 << 20, 512)
    assert 0 < small <= large <= 16 << 20


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(ldx=255), INVALID),
    (dict(ld_codes=255), INVALID), (dict(ld_scales=7), INVALID), (dict(x_rows=7), INVALID),
    (dict(x_rows=-1), INVALID), (dict(slots=GOOD, top_k=0), INVALID), (dict(x=None), INVALID),
    (dict(x=GOOD + 1), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(scales=GOOD + 2), INVALID), (dict(slots=GOOD + 1), INVALID),
    (dict(rows=0, x=None, codes=None), 0)])
def test_quantize_refusals(lib, over, code):
    a = dict(x=GOOD, ldx=256, x_rows=8, slots=None, top_k=1, rows=8, cols=256, codes=GOOD,
             ld_codes=256, scales=GOOD, ld_scales=8)
    a.update(over)
    assert lib.moe_blockscale_quantize(*a.values(), None) == code


PRODUCT = [(dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(E=0), INVALID),
           (dict(E=2, offsets=None), INVALID), (dict(lda=240), INVALID), (dict(lda=264), INVALID),
           (dict(ld_as=7), INVALID), (dict(ldw=240), INVALID), (dict(ldw=260), INVALID),
           (dict(a=None), INVALID), (dict(a=GOOD + 8), INVALID), (dict(a_scales=GOOD + 2), INVALID),
           (dict(w=None), INVALID), (dict(w=GOOD + 4), INVALID), (dict(w_scales=None), INVALID),
           (dict(w_scales=GOOD + 1), INVALID), (dict(offsets=GOOD + 2), INVALID),
           (dict(E=513), UNSUPPORTED), (dict(M=0, a=None, w=None), 0)]


@pytest.mark.parametrize("over,code", PRODUCT + [
    (dict(N=0), INVALID), (dict(ldo=511), INVALID), (dict(out=None), INVALID),
    (dict(out=GOOD + 1), INVALID), (dict(transpose_w=1, ldw=256), INVALID)])
def test_matmul_refusals(lib, over, code):
    a = dict(a=GOOD, lda=256, a_scales=GOOD, ld_as=8, w=GOOD, ldw=256, w_scales=GOOD, offsets=GOOD,
             E=4, M=8, N=512, K=256, transpose_w=0, out=GOOD, ldo=512)
    a.update(over)
    assert lib.moe_blockscale_matmul(*a.values(), None) == code


@pytest.mark.parametrize("over,code", PRODUCT + [
    (dict(I=0), INVALID), (dict(I=192), UNSUPPORTED), (dict(h=None), INVALID),
    (dict(h=GOOD + 8), INVALID), (dict(ldh=255), INVALID), (dict(ldh=264), INVALID),
    (dict(h_scales=None), INVALID), (dict(h_scales=GOOD + 2), INVALID), (dict(ld_hs=7), INVALID)])
def test_swiglu_refusals(lib, over, code):
    a = dict(a=GOOD, lda=256, a_scales=GOOD, ld_as=8, w13=GOOD, ldw=256, w_scales=GOOD,
             offsets=GOOD, E=4, M=8, I=256, K=256, clamp=0.0, h=GOOD, ldh=256, h_scales=GOOD,
             ld_hs=8)
    if "w" in over:
        over = {("w13" if k == "w" else k): v for k, v in over.items()}
    a.update(over)
    assert lib.moe_blockscale_swiglu(*a.values(), None) == code


# Sizes whose round-up to a tile would pass 32 bits.
LARGEST = 2 ** 31 - 256


@pytest.mark.parametrize("over", [dict(N=LARGEST + 1, ldo=1 << 31), dict(N=2 ** 31 - 1, ldo=1 << 31),
                                  dict(K=LARGEST + 1, lda=1 << 31, ldw=1 << 31, N=1),
                                  dict(M=LARGEST + 1, ld_as=1 << 31, N=1, E=1),
                                  dict(M=2 ** 31 - 1, ld_as=1 << 31, N=1, E=1),
                                  dict(N=2 ** 31 - 1, ldo=1 << 31, ldw=1 << 31, K=16,
                                       transpose_w=1)])
def test_matmul_sizes_near_32_bits(lib, over):
    a = dict(a=GOOD, lda=256, a_scales=GOOD, ld_as=8, w=GOOD, ldw=16, w_scales=GOOD, offsets=GOOD,
             E=1, M=8, N=512, K=16, transpose_w=0, out=GOOD, ldo=512)
    a.update(over)
    assert lib.moe_blockscale_matmul(*a.values(), None) == UNSUPPORTED


@pytest.mark.parametrize("over", [dict(M=2 ** 31 - 1), dict(N=2 ** 31 - 1), dict(K=2 ** 31 - 1)])
def test_linear_sizes_near_32_bits(lib, over):
    a = dict(x=GOOD, ldx=1 << 31, w=GOOD, ldw=1 << 31, w_scales=GOOD, M=8, N=1, K=16, transpose_w=0,
             out=GOOD, ldo=1 << 31, ws=GOOD, nbytes=1 << 60)
    if "N" in over:
        a["ldw"] = 16
    a.update(over)
    assert lib.moe_blockscale_linear_workspace(a["M"], a["N"], a["K"]) == 0
    assert lib.moe_blockscale_linear(*a.values(), None) == UNSUPPORTED


@pytest.mark.parametrize("over", [dict(rows=2 ** 31 - 1), dict(H=2 ** 31 - 16)])
def test_experts_sizes_near_32_bits(lib, over):
    a = dict(x=GOOD, ldx=1 << 31, T=8, slots=GOOD, top_k=1, rows=8, offsets=GOOD, E=1, w13=GOOD,
             s13=GOOD, w2=GOOD, s2=GOOD, H=16, I=128, clamp=0.0, out=GOOD, ldo=1 << 31, ws=GOOD,
             nbytes=1 << 62)
    a.update(over)
    assert lib.moe_blockscale_experts_workspace(a["rows"], a["H"], a["I"]) == 0
    assert lib.moe_blockscale_experts(*a.values(), None) == UNSUPPORTED


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 4865, 2 ** 31 - 65535])
def test_balance_tokens_near_32_bits(lib, T):
    # (the warps' stride over the tokens passes T)
    assert lib.moe_balance_workspace(T, 8) == 0
    assert forward(lib, T=T, E=8, K=1) == UNSUPPORTED
    a = dict(logits=GOOD, dtype=0, ld=8, T=T, E=8, K=1, coef=0.1, ids=GOOD, weights=GOOD,
             counts=GOOD, d_loss=GOOD, d_weights=GOOD, d_logits=GOOD, ld_d=8)
    assert lib.moe_balance_backward(*a.values(), None) == UNSUPPORTED
    assert lib.moe_balance_workspace(2 ** 31 - 65536, 8) > 0
