"""The host code of the router gate, the expert order, the block join and the 8-bit
products on several devices and with failing calls, against the stand-in for the
CUDA runtime; and the wrappers' checks on stand-ins for tensors (no GPU)."""
import ctypes

import pytest
import torch

from . import fake_cuda
from .test_operators_wrappers_cpu import BIG, Fake

P = 1 << 20
OK, INVALID, UNSUPPORTED, CUDA_ERROR = 0, 1, 2, 4


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    return fake_cuda.build(str(tmp_path_factory.mktemp("fake_cuda")))


@pytest.fixture
def lib(built, tmp_path):
    import moe_expert_layer_histogram_gb300 as m
    L = fake_cuda.load(built, str(tmp_path))
    real = m.lib()
    for name in ("moe_gate_forward", "moe_gate_backward", "moe_order", "moe_order_workspace",
                 "moe_join_forward", "moe_join_backward", "moe_join_workspace", "moe_int8_quantize",
                 "moe_int8_matmul", "moe_int8_linear", "moe_int8_experts",
                 "moe_int8_linear_workspace"):
        getattr(L, name).argtypes = getattr(real, name).argtypes
        getattr(L, name).restype = getattr(real, name).restype
    return L


def gate(L, T, E, groups=1, bias=P, dtype=0, score=1):
    import moe_expert_layer_histogram_gb300 as m
    c = m.MoEGateConfig(score, groups, groups, 1, 1, 1.0)
    return L.moe_gate_forward(P, dtype, E, bias, None, T, E, 2, c, P, P, P, None)


def gate_back(L):
    import moe_expert_layer_histogram_gb300 as m
    c = m.MoEGateConfig(1, 1, 1, 1, 1, 1.0)
    return L.moe_gate_backward(P, 0, 64, 100, 64, 2, c, P, P, P, 64, None)


def order(L, n, E):
    return L.moe_order(P, n, E, P, P, P, P, 1 << 40, None)


def join(L, T, H, K, x_type=0, back=False, ld=None):
    import moe_expert_layer_histogram_gb300 as m
    ld = ld or H
    j = m.MoEJoin(T=T, H=H, K=K, x_type=x_type, weight_type=0, gate_type=0, scale=1.0, eps=1e-6,
                  x=P, ld_x=ld, expert_rows=P, ld_rows=ld, rows=T * K, row_of_slot=P, weights=P,
                  shared=P, ld_shared=ld, gate=P, post_weight=P, norm_weight=P)
    if back:
        return L.moe_join_backward(j, P, ld, P, P, P, ld, P, ld, P, ld, P, ld, P, P, P, ld, P, P, P,
                                   P, 1 << 40, None)
    return L.moe_join_forward(j, P, ld, P, ld, P, H + 15 - (H + 15) % 16, P, P, P, None)


def linear(L, M, N, K):
    return L.moe_int8_linear(P, K, P, K, P, M, N, K, P, N, P, 1 << 40, None)


def matmul(L, E, M, N, K):
    return L.moe_int8_matmul(P, K, P, P, K, P, P if E > 1 else None, E, M, N, K, P, N, P, 1 << 40,
                             None)


def experts(L, T, rows, E, H=256, I=128):
    return L.moe_int8_experts(P, H, T, P, 1, rows, P, E, P, P, P, P, H, I, 0.0, P, H, P, 1 << 40,
                              None)


CALLS = {
    **{"gate %s" % (a,): (lambda L, a=a: gate(L, *a)) for a in
       ((8, 64), (100, 64), (100, 384, 8), (100, 510, 3), (100, 512, 1, None), (100, 48, 4, None, 1),
        (0, 16))},
    "gate backward": gate_back,
    **{"order %s" % (a,): (lambda L, a=a: order(L, *a)) for a in ((0, 8), (2048, 512), (300000, 512))},
    **{"join %s" % (a,): (lambda L, a=a: join(L, *a)) for a in
       ((1, 7168, 8), (333, 2001, 0), (40, 16384, 2, 1), (40, 16381, 2))},
    **{"join backward %s" % (a,): (lambda L, a=a: join(L, *a, back=True)) for a in
       ((1, 7168, 8), (333, 2001, 1), (5000, 2048, 6, 1), (40, 16384, 2, 1))},
    **{"linear %s" % (a,): (lambda L, a=a: linear(L, *a)) for a in
       ((1, 4096, 7168), (2, 300, 16384), (3, 4096, 2000), (16, 4096, 7168), (333, 1001, 2000),
        (8192, 4096, 7168), (16, 60000, 256))},
    **{"matmul %s" % (a,): (lambda L, a=a: matmul(L, *a)) for a in
       ((1, 1, 100, 64), (1, 4, 100, 131072), (8, 8, 256, 2048), (8, 700, 4096, 512),
        (8, 9000, 4096, 512))},
    **{"experts %s" % (a,): (lambda L, a=a: experts(L, *a)) for a in
       ((8, 8, 4), (8, 8, 16), (500, 500, 4), (40000, 80000, 4))},
    "quantize": lambda L: L.moe_int8_quantize(P, 256, 8, None, 1, 8, 256, P, 256, P, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_call_works_on_every_device(lib, name):
    for device in (0, 1, 3, 0, 1):
        lib.fake_set_device(device)
        before = lib.fake_launches()
        assert CALLS[name](lib) == OK, device
        assert lib.fake_launches() > before


def test_limits_are_set_once_per_device(lib):
    for device in (0, 1):
        lib.fake_set_device(device)
        for call in CALLS.values():
            assert call(lib) == OK
    so_far = lib.fake_attribute_calls()
    for device in (0, 1):
        lib.fake_set_device(device)
        for call in CALLS.values():
            assert call(lib) == OK
    assert lib.fake_attribute_calls() == so_far


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_leaves_no_error_behind(lib, name):
    assert CALLS[name](lib) == OK
    start = lib.fake_launches()
    assert CALLS[name](lib) == OK
    for nth in range(lib.fake_launches() - start):      # each of the call's launches in turn
        lib.fake_fail_launch(nth)
        assert CALLS[name](lib) == CUDA_ERROR
        assert lib.cudaPeekAtLastError() == 0
    assert CALLS[name](lib) == OK


@pytest.mark.parametrize("name", ["order (300000, 512)", "join backward (5000, 2048, 6, 1)",
                                  "matmul (8, 8, 256, 2048)", "linear (333, 1001, 2000)"])
def test_a_failure_does_not_last(lib, name):
    lib.fake_set_device(2)
    assert linear(lib, 1, 64, 64) == OK                 # (the device's own look-up)
    lib.fake_fail_calls(1)
    assert CALLS[name](lib) != OK
    assert CALLS[name](lib) == OK


def test_a_row_or_two_need_one_kernel_and_no_workspace(lib):
    for M, launches, ws in ((1, 1, False), (2, 1, False), (3, 2, True), (4, 2, True), (5, 2, True)):
        assert (lib.moe_int8_linear_workspace(M, 4096, 7168) > 0) == ws
        before = lib.fake_launches()
        assert linear(lib, M, 4096, 7168) == OK
        assert lib.fake_launches() - before == launches


PRODUCT = [(dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(E=0), INVALID),
           (dict(E=2, offsets=None), INVALID), (dict(lda=255), INVALID), (dict(ldw=240), INVALID),
           (dict(ldw=260), INVALID), (dict(a=None), INVALID), (dict(a_scales=None), INVALID),
           (dict(a_scales=P + 2), INVALID), (dict(w=None), INVALID), (dict(w=P + 8), INVALID),
           (dict(w_scales=None), INVALID), (dict(w_scales=P + 1), INVALID),
           (dict(offsets=P + 2), INVALID), (dict(out=None), INVALID), (dict(out=P + 1), INVALID),
           (dict(ldo=511), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID),
           (dict(nbytes=100), INVALID), (dict(E=513), UNSUPPORTED),
           (dict(M=2 ** 31 - 1, N=1), UNSUPPORTED), (dict(N=2 ** 31 - 1, ldo=1 << 31), UNSUPPORTED),
           (dict(K=2 ** 31 - 65791, lda=1 << 31, ldw=1 << 31), UNSUPPORTED),
           (dict(M=0, a=None, w=None), 0)]


@pytest.mark.parametrize("over,code", PRODUCT)
def test_matmul_refusals(lib, over, code):
    a = dict(a=P, lda=256, a_scales=P, w=P, ldw=256, w_scales=P, offsets=P, E=4, M=8, N=512, K=256,
             out=P, ldo=512, ws=P, nbytes=1 << 40)
    a.update(over)
    assert lib.moe_int8_matmul(*a.values(), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(ldx=255), INVALID),
    (dict(w=P + 4), INVALID), (dict(ldw=257), INVALID), (dict(out=P + 1), INVALID),
    (dict(M=9, ws=None), INVALID), (dict(M=9, nbytes=0), INVALID), (dict(M=9, ws=P + 4), INVALID),
    (dict(M=2 ** 31 - 1), UNSUPPORTED), (dict(M=0, x=None), 0)])
def test_linear_refusals(lib, over, code):
    a = dict(x=P, ldx=256, w=P, ldw=256, w_scales=P, M=1, N=512, K=256, out=P, ldo=512, ws=P,
             nbytes=1 << 40)
    a.update(over)
    assert lib.moe_int8_linear(*a.values(), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(top_k=0), INVALID), (dict(slots=None), INVALID),
    (dict(slots=P + 2), INVALID), (dict(offsets=None), INVALID), (dict(w13=P + 8), INVALID),
    (dict(s2=None), INVALID), (dict(I=0), INVALID), (dict(I=24), UNSUPPORTED),
    (dict(H=24, ldx=24, ldo=24), UNSUPPORTED), (dict(x=None), INVALID), (dict(ldo=255), INVALID),
    (dict(ws=None), INVALID), (dict(nbytes=1000), INVALID), (dict(I=1 << 30), UNSUPPORTED),
    (dict(rows=2 ** 31 - 1), UNSUPPORTED), (dict(rows=0, x=None, out=None, ws=None), 0)])
def test_experts_refusals(lib, over, code):
    a = dict(x=P, ldx=256, T=8, slots=P, top_k=2, rows=16, offsets=P, E=4, w13=P, s13=P, w2=P, s2=P,
             H=256, I=128, clamp=0.0, out=P, ldo=256, ws=P, nbytes=1 << 40)
    a.update(over)
    assert lib.moe_int8_experts(*a.values(), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(ldx=255), INVALID),
    (dict(ld_codes=255), INVALID), (dict(x_rows=7), INVALID), (dict(slots=P, top_k=0), INVALID),
    (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(codes=None), INVALID),
    (dict(scales=P + 2), INVALID), (dict(slots=P + 1), INVALID),
    (dict(cols=2 ** 31 - 65791, ldx=1 << 31, ld_codes=1 << 31), UNSUPPORTED),
    (dict(rows=0, x=None, codes=None), 0)])
def test_quantize_refusals(lib, over, code):
    a = dict(x=P, ldx=256, x_rows=8, slots=None, top_k=1, rows=8, cols=256, codes=P, ld_codes=256,
             scales=P)
    a.update(over)
    assert lib.moe_int8_quantize(*a.values(), None) == code


# ---- the torch wrappers
def weights(shape, strides=None):
    return Fake(torch.int8, shape, strides), Fake(torch.float32, shape[:-1])


@pytest.mark.parametrize("shape,strides,want", [
    ((256, 512), None, (1, 256, 512, 512)), ((1, 512), (0, 1), (1, 1, 512, 512)),
    ((3, 256, 500), (256 * 512, 512, 1), (3, 256, 500, 512)),
    ((3, 1, 500), (512, 7, 1), (3, 1, 500, 512))])
def test_weight_strides(shape, strides, want):
    from moe_expert_layer_histogram_gb300 import int8
    assert int8._weights(*weights(shape, strides)) == want


@pytest.mark.parametrize("shape,strides", [
    ((3, 1, 512), (0, 0, 1)), ((3, 1, 512), (16, 16, 1)), ((3, 256, 512), (0, 512, 1)),
    ((256, 512), (1, 256)), ((BIG, 16), None), ((2, 16, BIG), None)])
def test_weight_strides_refused(shape, strides):
    from moe_expert_layer_histogram_gb300 import int8
    with pytest.raises(ValueError):
        int8._weights(*weights(shape, strides))


def test_more_ids_than_32_bits_are_refused(monkeypatch):
    from moe_expert_layer_histogram_gb300 import gate as g
    monkeypatch.setattr(g, "stream_on", lambda device: 0)
    ids = Fake(torch.int32, (BIG,))
    ids.numel = lambda: BIG
    with pytest.raises(ValueError):
        g.router_order(ids, 8)
    for bad in (dict(top_k=BIG), dict(top_k=2, groups=BIG), dict(top_k=2, group_top=BIG)):
        with pytest.raises(ValueError):
            g.router_gate(Fake(torch.float32, (4, 8)), **bad)


def test_structure_sizes():
    import moe_expert_layer_histogram_gb300 as m
    from moe_expert_layer_histogram_gb300 import join as j
    assert len(j._pack(*range(6), 1.0, 2.0, *range(12))) == ctypes.sizeof(m.MoEJoin)
    s = m.MoEJoin.from_buffer_copy(j._pack(*range(1, 7), 1.0, 2.0, *range(7, 19)))
    assert [getattr(s, n) for n, _ in m.MoEJoin._fields_] == [1, 2, 3, 4, 5, 6, 1.0, 2.0,
                                                              *range(7, 19)]


@pytest.mark.parametrize("rows", [8, 500, 40000, 80000])
def test_experts_of_no_tokens(lib, rows):
    # slots outside an empty x: rows of zeros, whatever their number
    before = lib.fake_launches()
    assert experts(lib, 0, rows, 4) == OK
    assert lib.fake_launches() > before


LOW = -(2 ** 32) + 4                                  # 4, if cut to 32 bits


def test_numbers_below_32_bits_are_refused(monkeypatch):
    from moe_expert_layer_histogram_gb300 import _tensors, balance, blockscale, int8
    from moe_expert_layer_histogram_gb300 import gate as g
    for n in (LOW, -(2 ** 31) - 1):
        with pytest.raises(ValueError):
            _tensors.fits(n, "top_k")
    assert _tensors.fits(-1, "top_k") is None          # (the library's own refusal)
    for module in (g, balance, blockscale, int8):
        monkeypatch.setattr(module, "stream_on", lambda device: 0)
    ids = Fake(torch.int32, (16,))
    ids.numel = lambda: 16
    x = Fake(torch.float32, (4, 8))
    with pytest.raises(ValueError):
        g.router_order(ids, LOW)
    for bad in (dict(top_k=LOW), dict(top_k=2, groups=LOW), dict(top_k=2, groups=4, group_top=LOW)):
        with pytest.raises(ValueError):
            g.router_gate(x, **bad)
    with pytest.raises(ValueError):
        balance.router_balance(x, LOW)
    rows = Fake(torch.bfloat16, (4, 16))
    for quantize in (blockscale.blockscale_quantize, int8.int8_quantize):
        with pytest.raises(ValueError):
            quantize(rows, ids, LOW)


@pytest.mark.parametrize("strides", [(33, 1), (0, 1), (100, 1)])
def test_the_stride_of_a_single_row_says_nothing(strides):
    # (the library wants strides of 16 bytes; there is no second row to be reached by one)
    from moe_expert_layer_histogram_gb300 import int8
    assert int8._weights(*weights((1, 33), strides)) == (1, 1, 33, 48)
    assert int8._weights(*weights((1, 1, 33), (33,) + strides)) == (1, 1, 33, 48)
