"""The operators' host code on several devices and with failing calls, against
a stand-in for the CUDA runtime (no GPU): a kernel's shared-memory limit belongs
to the device it was set on, so each device needs its own."""
import ctypes

import pytest

from . import fake_cuda

P = 1 << 20
OK, CUDA_ERROR = 0, 4


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    return fake_cuda.build(str(tmp_path_factory.mktemp("fake_cuda")))


@pytest.fixture
def lib(built, tmp_path):
    L = fake_cuda.load(built, str(tmp_path))
    vp, ci, i64, cf, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                           ctypes.c_size_t)
    L.moe_balance_forward.argtypes = [vp, ci, i64, vp, ci, ci, ci, cf, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_balance_backward.argtypes = [vp, ci, i64, ci, ci, ci, cf, vp, vp, vp, vp, vp, vp, i64, vp]
    L.moe_blockscale_quantize.argtypes = [vp, i64, ci, vp, ci, ci, ci, vp, i64, vp, i64, vp]
    L.moe_blockscale_matmul.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, ci, ci, ci, ci, ci, vp, i64,
                                        vp]
    L.moe_blockscale_linear.argtypes = [vp, i64, vp, i64, vp, ci, ci, ci, ci, vp, i64, vp, sz, vp]
    L.moe_blockscale_experts.argtypes = [vp, i64, ci, vp, ci, ci, vp, ci, vp, vp, vp, vp, ci, ci, cf,
                                         vp, i64, vp, sz, vp]
    L.moe_blockscale_linear_workspace.argtypes = [ci, ci, ci]
    L.moe_blockscale_linear_workspace.restype = sz
    return L


def balance(L, T, E):
    return L.moe_balance_forward(P, 0, E, None, T, E, 1, 1.0, P, P, P, P, P, P, 1 << 40, None)


def linear(L, M, N, K, transpose=0):
    return L.moe_blockscale_linear(P, K, P, N if transpose else K, P, M, N, K, transpose, P, N, P,
                                   1 << 40, None)


def matmul(L, E, M, N, K, transpose=0):
    return L.moe_blockscale_matmul(P, K, P, M, P, N if transpose else K, P, P, E, M, N, K, transpose,
                                   P, N, None)


def experts(L, T, rows, E, H=256, I=128):
    return L.moe_blockscale_experts(P, H, T, P, 1, rows, P, E, P, P, P, P, H, I, 0.0, P, H, P,
                                    1 << 40, None)


CALLS = {  # every kernel of the products, and the router's with most shared memory
    **{"balance %d x %d" % te: (lambda L, te=te: balance(L, *te)) for te in
       ((8, 64), (8, 200), (8, 300), (8, 512), (4096, 64), (4096, 300), (4096, 512))},
    **{"linear %s" % (a,): (lambda L, a=a: linear(L, *a)) for a in
       ((1, 4096, 7168, 0), (1, 4096, 7168, 1), (16, 32768, 256, 0), (16, 32768, 256, 1),
        (300, 1024, 2048, 0), (300, 1024, 2048, 1), (4000, 4096, 1024, 0), (4000, 4096, 1024, 1),
        (600, 8192, 256, 0), (600, 8192, 256, 1), (600, 4096, 256, 0), (600, 4096, 256, 1))},
    **{"grouped %s" % (a,): (lambda L, a=a: matmul(L, *a)) for a in
       ((8, 8, 256, 2048, 0), (8, 8, 256, 2048, 1), (8, 400, 256, 2048, 0), (8, 400, 256, 2048, 1),
        (8, 8192, 4096, 512, 0), (8, 8192, 4096, 512, 1), (8, 3000, 4096, 512, 0),
        (8, 3000, 4096, 512, 1))},
    **{"experts %s" % (a,): (lambda L, a=a: experts(L, *a)) for a in
       ((8, 8, 4), (8, 8, 1), (500, 500, 4), (8000, 8000, 4), (40000, 80000, 4))},
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
    set_so_far = lib.fake_attribute_calls()
    for device in (0, 1):
        lib.fake_set_device(device)
        for call in CALLS.values():
            assert call(lib) == OK
    assert lib.fake_attribute_calls() == set_so_far


# (the linear call looks the device up twice)
@pytest.mark.parametrize("name,failures", [("balance 8 x 512", 1), ("balance 4096 x 300", 1),
                                           ("grouped (8, 8, 256, 2048, 0)", 1),
                                           ("linear (1, 4096, 7168, 0)", 2)])
def test_a_failure_does_not_last(lib, name, failures):
    lib.fake_set_device(2)
    lib.fake_fail_calls(failures)
    assert CALLS[name](lib) != OK
    assert CALLS[name](lib) == OK


@pytest.mark.parametrize("name", ["balance 8 x 64", "balance 4096 x 512",
                                  "linear (1, 4096, 7168, 0)", "linear (4000, 4096, 1024, 0)",
                                  "grouped (8, 8, 256, 2048, 0)", "experts (500, 500, 4)",
                                  "experts (40000, 80000, 4)", "backward", "quantize"])
def test_a_failed_launch_leaves_no_error_behind(lib, name):
    # (the next launch check of the program would take it for its own)
    call = dict(CALLS, backward=lambda L: L.moe_balance_backward(
        P, 0, 64, 32, 64, 6, 1.0, P, P, P, P, P, P, 64, None),
        quantize=lambda L: L.moe_blockscale_quantize(P, 256, 8, None, 1, 8, 256, P, 256, P, 8, None)
    )[name]
    assert call(lib) == OK
    start = lib.fake_launches()
    assert call(lib) == OK
    for nth in range(lib.fake_launches() - start):      # each of the call's launches in turn
        lib.fake_fail_launch(nth)
        assert call(lib) == CUDA_ERROR
        assert lib.cudaPeekAtLastError() == 0
    assert call(lib) == OK


def test_every_product_has_stages_to_load_ahead(lib):
    # products that quantise their own rows keep them in shared memory beside the
    # ring of weight tiles: two stages at least, one to load while one is used
    seen = 0
    for M in (1, 2, 5, 16, 17, 32, 48, 64, 65, 128, 333, 1000):
        for N in (64, 1000, 4096, 9728, 12000, 20000):
            for K in list(range(128, 13000, 384)) + [10880, 10896, 11008, 11392, 16384, 30000]:
                own_rows = lib.moe_blockscale_linear_workspace(M, N, K) == 0
                seen += own_rows
                assert linear(lib, M, N, K) == OK
                assert lib.fake_last_stages() >= 2, (M, N, K, own_rows)
    assert seen > 100


def test_experts_of_many_tokens_copy_the_codes(lib):
    # one launch more: the tokens' quantisation, the copy, two products
    from .test_gpu_blockscale_edges import COPIED
    for T, E, topk, H, I in COPIED:
        before = lib.fake_launches()
        assert lib.moe_blockscale_experts(P, H, T, P, topk, T * topk, P, E, P, P, P, P, H, I, 0.0, P,
                                          H, P, 1 << 40, None) == OK
        assert lib.fake_launches() - before == 4
    before = lib.fake_launches()
    assert experts(lib, 64, 128, 4) == OK
    assert lib.fake_launches() - before == 3


def test_rows_are_quantised_in_the_product_only_where_all_ctas_run_at_once(lib):
    for M in (1, 3, 16, 17, 48, 128, 130, 400, 512):
        for N in (1, 128, 1000, 4096, 9728, 9729, 19456, 19457, 40000, 128256, 1 << 20):
            for K in (16, 128, 2000, 4096, 7168, 11008):
                if lib.moe_blockscale_linear_workspace(M, N, K) == 0:
                    assert linear(lib, M, (N + 15) // 16 * 16, K) == OK
                    assert lib.fake_last_grid() <= 152, (M, N, K)
