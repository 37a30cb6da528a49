"""The end of a block (routed rows, shared expert, norms, gate, residual): its
values, 8-bit codes and all gradients against plain implementations in 64 bits.

Tolerances.  u = 2^-24.  A sum over the width is made of runs of at most 32 terms
in a thread, 5 + 5 steps of a tree, and the products' own roundings: it is off by
at most 50 u of the sum of its terms' magnitudes; 1 / sqrt(mean + eps) by half of
that and 3 u more.  y is off by (K + 3) u of its terms' magnitudes and sigmoid's
6 u.  So x' is within 100 u of the sum of its terms' magnitudes, h (of the stored
x', which the tests take as it is) within 50 u of itself; d x' passes through one
such sum more and d y through two: 200 u and 400 u of their terms' magnitudes (in
which a mean counts with the magnitudes of its terms).  Sums over T tokens add
T u.  Rounding to bf16 adds 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8
TINY = 1e-30


def randn(*shape, seed=0, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def make(T, H, K, shared=True, gate=True, post=True, norm=True, x_type=torch.float32,
         w_type=torch.float32, gate_type=torch.float32, dead=0.2, seed=0, extra_rows=5):
    from moe_expert_layer_histogram_gb300 import RouterOrder
    a = dict(x=randn(T, H, seed=seed, dtype=x_type, scale=2.0), scale=0.7, eps=1e-5)
    if K:
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        n = T * K
        place = torch.randperm(n, generator=g, device="cuda")
        gone = torch.rand(n, generator=g, device="cuda") < dead
        live = n - int(gone.sum())
        rows = torch.empty(n, dtype=torch.int32, device="cuda")
        rows[gone] = -1
        rows[~gone] = torch.argsort(place[~gone]).to(torch.int32)
        a["expert_rows"] = randn(n + extra_rows, H, seed=seed + 2, dtype=torch.bfloat16)
        a["weights"] = randn(T, K, seed=seed + 3)
        offsets = torch.tensor([0, live], dtype=torch.int32, device="cuda")
        a["order"] = RouterOrder(None, offsets, rows)
    if shared:
        a["shared"] = randn(T, H, seed=seed + 4, dtype=torch.bfloat16)
        if gate:
            a["gate"] = randn(T, seed=seed + 5, dtype=gate_type, scale=2.0)
    if post:
        a["post_weight"] = (1 + randn(H, seed=seed + 6, scale=0.3)).to(w_type)
    if norm:
        a["norm_weight"] = (1 + randn(H, seed=seed + 7, scale=0.3)).to(w_type)
    return a


def d(t):
    return None if t is None else t.double()


def terms(a):
    """(y, its terms' magnitudes, the slots' rows [T, K, H], sigmoid of the gate)."""
    x = a["x"]
    T, H = x.shape
    y, m = torch.zeros(T, H, dtype=torch.float64, device="cuda"), 0.0
    z = None
    if "expert_rows" in a:
        r = getattr(a["order"], "rows", a["order"]).long()
        R = a["expert_rows"].shape[0]
        ok = (r >= 0) & (r < R)
        z = torch.where(ok[:, None], d(a["expert_rows"])[r.clamp(0, R - 1)], 0.0)
        z = z.view(T, -1, H)
        w = torch.where(ok.view(T, -1), d(a["weights"]), 0.0)[:, :, None]
        y, m = (w * z).sum(1), (w * z).abs().sum(1)
    s = torch.ones(T, 1, dtype=torch.float64, device="cuda")
    if a.get("gate") is not None:
        s = torch.sigmoid(d(a["gate"]))[:, None]
    if a.get("shared") is not None:
        y, m = y + s * d(a["shared"]), m + (s * d(a["shared"])).abs()
    return y, m, z, s


def rstd(v, eps):
    return (v.square().mean(1, keepdim=True) + eps).rsqrt()


def close(got, want, tol, what):
    if got.dtype is torch.bfloat16:
        tol = tol + BF16 * (want.abs() + tol)
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all()), what
    assert bool((err <= tol + TINY).all()), (what, float((err - tol).max()), float(err.max()))


def check(a, quantize=False, d_x=True, d_h=True, out=None, backward=True, seed=50):
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    x, eps, scale = a["x"], a["eps"], a["scale"]
    T, H = x.shape
    j = block_join(**a, quantize=quantize, out=out)
    y, m, z, s = terms(a)
    joined = "expert_rows" in a or "shared" in a
    r1 = rstd(y, eps) if "post_weight" in a else torch.ones(T, 1, dtype=torch.float64, device="cuda")
    wp = d(a["post_weight"]) if "post_weight" in a else 1.0
    # r1's relative error, from y's: the magnitudes of y's terms over its norm
    bad = 1.0
    if "post_weight" in a:
        bad = (m * y.abs()).mean(1, keepdim=True) / (y.square().mean(1, keepdim=True) + eps) + 1.0
    if joined:
        want = d(x0 := a.get("x_before", x)) + scale * y * r1 * wp
        close(j.x, want, 100 * U * (d(x0).abs() + abs(scale) * r1 * (m + y.abs() * bad) * abs(wp)), "x")
    else:
        assert j.x is x
    v = d(j.x)
    if "norm_weight" in a:
        r2 = rstd(v, eps)
        h = v * r2 * d(a["norm_weight"])
        if quantize:
            check_codes(j.codes, j.code_scales, h)
        else:
            close(j.h, h, 50 * U * h.abs(), "h")
    if not backward:
        return j, None
    dx = randn(T, H, seed=seed, dtype=x.dtype) if d_x else None
    dh = randn(T, H, seed=seed + 1, dtype=torch.bfloat16) if d_h and "norm_weight" in a else None
    got = block_join_backward(j, d_x=dx, d_h=dh)
    g = torch.zeros(T, H, dtype=torch.float64, device="cuda") if dx is None else d(dx)
    gm = g.abs()
    if dh is not None:
        xh, w = v * r2, d(a["norm_weight"])
        k = d(dh) * w
        close(got.norm_weight, (d(dh) * xh).sum(0), (60 + T) * U * (d(dh) * xh).abs().sum(0), "d_norm")
        g = g + r2 * (k - xh * (k * xh).mean(1, keepdim=True))
        gm = gm + r2 * (k.abs() + xh.abs() * (k * xh).abs().mean(1, keepdim=True))
    else:
        assert got.norm_weight is None
    close(got.x, g, 200 * U * gm, "d_x")
    if not joined:
        return j, got
    g, gm = scale * g, abs(scale) * gm
    if "post_weight" in a:
        yh, ym = y * r1, r1 * (m + y.abs() * bad)
        close(got.post_weight, (g * yh).sum(0),
              ((60 + T) * U * (g * yh).abs() + 300 * U * (gm * yh.abs() + gm * ym)).sum(0), "d_post")
        k, km = g * wp, gm * abs(wp)
        g = r1 * (k - yh * (k * yh).mean(1, keepdim=True))
        gm = r1 * bad * (km + ym * (km * ym).mean(1, keepdim=True))
    tol = 400 * U * gm
    if z is not None:
        R = a["expert_rows"].shape[0]
        K = z.shape[1]
        r = getattr(a["order"], "rows", a["order"]).long()
        ok = ((r >= 0) & (r < R)).view(T, K)
        close(got.weights, (g[:, None] * z).sum(2) * ok,
              (tol[:, None] * z.abs()).sum(2) + 60 * U * (g[:, None] * z).abs().sum(2), "d_weights")
        w = torch.where(ok, d(a["weights"]), 0.0)[:, :, None]
        named = r[ok.view(-1)]
        close(got.expert_rows[named], (w * g[:, None]).reshape(-1, H)[ok.view(-1)],
              (w.abs() * tol[:, None]).reshape(-1, H)[ok.view(-1)], "d_rows")
        if hasattr(a["order"], "offsets"):
            assert bool((got.expert_rows[int(a["order"].offsets[-1]):] == 0).all())
    if "shared" in a:
        close(got.shared, s * g, s * tol + 8 * U * (s * g).abs(), "d_shared")
        if "gate" in a:
            u, q = d(a["shared"]), (s * (1 - s))[:, 0]
            close(got.gate, (g * u).sum(1) * q,
                  q * ((tol * u.abs()).sum(1) + 60 * U * (g * u).abs().sum(1)) + 2 * U, "d_gate")
    return j, got


def check_codes(codes, scales, h):
    """Codes of h (64 bits; fp32 h is within 50 u of it) and their scales."""
    amax = h.abs().amax(1)
    s = scales.double()
    assert bool(((s - amax / 127).abs() <= 54 * U * amax / 127).all())
    q = h / torch.where(s > 0, s, 1.0)[:, None]
    # at most half a step, and what the quotient may be off by
    assert bool(((codes.double() - q).abs() <= 0.5 + 128 * 110 * U).all())
    assert codes.dtype is torch.int8 and int(codes.abs().max() if codes.numel() else 0) <= 127


CASES = [
    (1, 7168, 8), (3, 64, 2), (2, 1, 1), (5, 7, 3), (37, 2001, 4), (200, 333, 16), (160, 2048, 6),
    (400, 520, 1), (9, 16384, 2), (153, 8200, 3), (7, 4104, 5), (1000, 40, 2),
]


@pytest.mark.parametrize("T,H,K", CASES)
@pytest.mark.parametrize("x_type", [torch.float32, torch.bfloat16])
def test_everything(T, H, K, x_type):
    check(make(T, H, K, x_type=x_type, w_type=x_type, gate_type=x_type))


@pytest.mark.parametrize("K", [0, 3])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_parts_left_out(K, shared, post, norm):
    from moe_expert_layer_histogram_gb300 import block_join
    a = make(20, 264, K, shared=shared, gate=shared and post, post=post and (K > 0 or shared),
             norm=norm, w_type=torch.bfloat16)
    if not K and not shared and not norm:
        with pytest.raises(ValueError):
            block_join(**a)
        return
    for dx, dh in ((True, True), (False, True), (True, False), (False, False)):
        check(a, d_x=dx, d_h=dh)


@pytest.mark.parametrize("T,H", [(1, 7168), (3, 1), (40, 2001), (300, 512), (9, 16384)])
@pytest.mark.parametrize("x_type", [torch.float32, torch.bfloat16])
def test_codes(T, H, x_type):
    j, _ = check(make(T, H, 2, x_type=x_type), quantize=True, backward=False)
    assert j.h is None and j.codes.shape == (T, H) and j.codes.stride(0) % 16 == 0


def test_codes_of_zero_and_infinite_rows():
    from moe_expert_layer_histogram_gb300 import block_join
    x = randn(4, 96)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 9] = float("nan")
    j = block_join(x, norm_weight=torch.ones(96, device="cuda"), quantize=True)
    assert float(j.code_scales[1]) == 0 and bool((j.codes[1] == 0).all())
    assert bool(torch.isnan(j.code_scales[2:]).all()) and bool((j.codes[2:] == 0).all())


def test_rows_of_no_expert_are_no_terms():
    # a NaN weight or row behind a slot of no expert changes nothing
    a = make(30, 128, 4, dead=0.5)
    j, got = check(a)
    b = dict(a, weights=a["weights"].clone(), expert_rows=a["expert_rows"].clone())
    gone = (a["order"].rows < 0).view(30, 4)
    b["weights"][gone] = float("nan")
    b["expert_rows"][int(a["order"].offsets[-1]):] = float("nan")
    j2, got2 = check(b)
    assert torch.equal(j.x, j2.x) and torch.equal(got.x, got2.x)
    assert torch.equal(got.weights, got2.weights) and bool((got.weights[gone] == 0).all())


def test_tokens_without_any_row():
    # y = 0 through a norm: 0, with finite gradients
    a = make(12, 200, 3, shared=False, dead=1.0)
    j, got = check(a)
    assert torch.equal(j.x, a["x"])


def test_plain_rows_and_rows_outside():
    a = make(16, 72, 2, dead=0.0)
    rows = a["order"].rows.clone()
    rows[3], rows[9] = 10 ** 6, -5
    a["order"] = rows
    check(a)


def test_in_place():
    a = make(50, 256, 4)
    a["x_before"] = None
    del a["x_before"]
    from moe_expert_layer_histogram_gb300 import block_join
    want = block_join(**a)
    x = a["x"].clone()
    j = block_join(**dict(a, x=x), out=x)
    assert j.x is x and torch.equal(x, want.x) and torch.equal(j.h, want.h)


@pytest.mark.parametrize("T", [7, 2000])
def test_without_d_h_the_new_x_is_not_read(T):
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    a, dx = make(T, 4104, 2), randn(T, 4104, seed=60)
    j = block_join(**a)
    want = block_join_backward(j, d_x=dx)
    j.x, j._ld_x = torch.full((T, 4104), float("nan"), device="cuda"), 1
    got = block_join_backward(j, d_x=dx)
    for name in ("x", "expert_rows", "weights", "shared", "gate", "post_weight"):
        one, two = getattr(want, name), getattr(got, name)
        assert torch.equal(one, two) and bool(torch.isfinite(one).all()), name


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (8, 3), (16, 16)])
def test_strided_arguments(offset, pad):
    T, H, K = 23, 160, 3
    a = make(T, H, K, x_type=torch.bfloat16)

    def strided(t):
        big = torch.full((t.shape[0] * (H + pad) + offset,), float("nan"), dtype=t.dtype,
                         device="cuda")
        v = torch.as_strided(big, t.shape, (H + pad, 1), offset)
        v.copy_(t)
        return v
    b = dict(a, x=strided(a["x"]), expert_rows=strided(a["expert_rows"]), shared=strided(a["shared"]))
    out = strided(torch.zeros_like(a["x"]))
    j, got = check(a)
    j2, got2 = check(b, out=out)
    assert j2.x is out
    if offset % 8 == 0 and pad % 8 == 0:
        assert torch.equal(j.x, j2.x) and torch.equal(got.expert_rows, got2.expert_rows)


def test_gradients_against_differences():
    a = make(3, 12, 2, x_type=torch.float32, dead=0.0)
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    gx, gh = randn(3, 12, seed=60), randn(3, 12, seed=61, dtype=torch.bfloat16)

    def value(b):
        y, _, _, _ = terms(b)
        n = y * rstd(y, b["eps"]) * d(b["post_weight"])
        x = d(b["x"]) + b["scale"] * n
        h = x * rstd(x, b["eps"]) * d(b["norm_weight"])
        return float((x * d(gx)).sum() + (h * d(gh)).sum())

    got = block_join_backward(block_join(**a), d_x=gx, d_h=gh)
    step = 1e-5
    for name in ("x", "expert_rows", "weights", "shared", "gate", "post_weight", "norm_weight"):
        grad = getattr(got, name).double().flatten()
        base = a[name].double()
        for i in range(0, base.numel(), 5):
            f = []
            for sign in (1, -1):
                v = base.clone()
                v.view(-1)[i] += sign * step
                f.append(value(dict(a, **{name: v})))
            want = (f[0] - f[1]) / (2 * step)
            tol = 1e-4 + (BF16 * abs(want) if getattr(got, name).dtype is torch.bfloat16 else 0)
            if name == "expert_rows" and i // 12 >= int(a["order"].offsets[-1]):
                continue
            assert abs(float(grad[i]) - want) <= tol, (name, i)


def test_no_tokens():
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    a = make(0, 64, 2)
    j = block_join(**a)
    got = block_join_backward(j, d_x=torch.empty(0, 64, device="cuda"),
                              d_h=torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert j.x.shape == (0, 64) and bool((got.norm_weight == 0).all())
    assert bool((got.post_weight == 0).all())


def test_same_bits_every_time_on_streams_and_in_a_graph():
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    a = make(700, 1024, 4, x_type=torch.bfloat16)
    dx, dh = randn(700, 1024, dtype=torch.bfloat16), randn(700, 1024, seed=1, dtype=torch.bfloat16)

    def once():
        j = block_join(**a)
        g = block_join_backward(j, dx, dh)
        return [j.x, j.h, g.x, g.expert_rows, g.weights, g.shared, g.gate, g.post_weight,
                g.norm_weight]
    want = once()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(once())
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_rows_past_32_bits():
    # 2^31 elements and more before the last rows
    H, R = 16384, 140000
    rows = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    rows[-1] = randn(H, dtype=torch.bfloat16)
    a = dict(x=randn(1, H, seed=2), expert_rows=rows, scale=1.0, eps=1e-6,
             order=torch.tensor([R - 1], dtype=torch.int32, device="cuda"),
             weights=torch.full((1, 1), 2.0, device="cuda"))
    from moe_expert_layer_histogram_gb300 import block_join
    assert torch.equal(block_join(**a).x, a["x"] + 2 * rows[-1].float())


def test_refusals():
    from moe_expert_layer_histogram_gb300 import MoEError, block_join, block_join_backward
    a = make(6, 32, 2)
    for bad in (dict(weights=None), dict(order=None), dict(expert_rows=None), dict(shared=None),
                dict(gate=a["gate"][:5]), dict(post_weight=a["post_weight"].bfloat16()),
                dict(norm_weight=None, quantize=True), dict(weights=a["weights"][:5]),
                dict(x=a["x"][:, ::2]), dict(shared=a["shared"][:, :30]),
                dict(expert_rows=a["expert_rows"].float()), dict(out=a["x"].bfloat16()),
                dict(order=a["order"].rows.long()), dict(weights=a["weights"][:, :0])):
        with pytest.raises((ValueError, TypeError)):
            block_join(**dict(a, **bad))
    for bad in (dict(eps=-1.0), dict(scale=float("inf"))):
        with pytest.raises(MoEError):
            block_join(**dict(a, **bad))
    with pytest.raises(MoEError):
        block_join(randn(2, 16385), norm_weight=torch.ones(16385, device="cuda"))
    j = block_join(**a)
    with pytest.raises(ValueError):
        block_join_backward(j, d_x=a["x"].bfloat16())
    with pytest.raises(ValueError):
        block_join_backward(j, d_h=a["x"])
    with pytest.raises(ValueError):
        block_join_backward(block_join(**dict(a, norm_weight=None)),
                            d_h=torch.zeros(6, 32, dtype=torch.bfloat16, device="cuda"))


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    from moe_expert_layer_histogram_gb300 import moe_join_status
    assert moe_join_status() == 0


@pytest.mark.parametrize("T,H,K", [(12500, 64, 2), (4000, 1032, 3), (1000, 4096, 16), (1000, 7936, 4),
                                   (400, 7944, 4), (2500, 8, 1)])
@pytest.mark.parametrize("x_type", [torch.float32, torch.bfloat16])
def test_many_tokens_for_each_block(T, H, K, x_type):
    check(make(T, H, K, x_type=x_type, w_type=x_type, post=K % 2 == 0))


@pytest.mark.parametrize("T,H", [(28, 264), (28, 2001), (4200, 1032), (420, 7168)])
@pytest.mark.parametrize("gate_type", [torch.float32, torch.bfloat16])
def test_gradient_of_saturated_gates(T, H, gate_type):
    # 1 - sigmoid(a) cancels where sigmoid(a) is near 1.  Without norms d y is scale d x'
    # to 2 u of itself (scale's rounding and the product's) and the dot product is off by
    # 62 u of its terms' magnitudes; sigmoid(a) and sigmoid(-a) by 6 u each, their
    # products by 2 u: no absolute term
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    a = make(T, H, 0, post=False, norm=False, gate_type=gate_type)
    size = torch.tensor([0.5, 4.0, 8.0, 12.0, 16.0, 20.0, 40.0], device="cuda")
    a["gate"] = torch.cat([size, -size]).repeat(T // 14).to(gate_type)
    dx = randn(T, H, seed=70)
    got = block_join_backward(block_join(**a), d_x=dx).gate
    s = torch.sigmoid(d(a["gate"])) * torch.sigmoid(-d(a["gate"]))
    parts = a["scale"] * d(dx) * d(a["shared"])
    want = s * parts.sum(1)
    tol = 62 * U * s * parts.abs().sum(1) + 14 * U * want.abs()
    if gate_type is torch.bfloat16:
        tol = tol + BF16 * (want.abs() + tol)
    assert bool(((got.double() - want).abs() <= tol + 2.0 ** -126).all())
    check(dict(a, norm_weight=1 + randn(H, seed=71, scale=0.3), post_weight=1 + randn(H, seed=72, scale=0.3)))


@pytest.mark.parametrize("H", [64, 61])
@pytest.mark.parametrize("live", [0, 3])
def test_no_tokens_leave_zeros_in_rows_of_no_expert(H, live):
    from moe_expert_layer_histogram_gb300 import MoEJoin, moe_join_backward
    rows = torch.zeros(2000, H, dtype=torch.bfloat16, device="cuda")
    j = MoEJoin(T=0, H=H, K=2, scale=1.0, eps=1e-6, expert_rows=rows.data_ptr(), ld_rows=H, rows=2000)
    got = torch.full((2001, H), 7.0, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([live], dtype=torch.int32, device="cuda")
    moe_join_backward(j, None, H, None, None, None, H, None, H, None, H, got, H, n, None, None, H,
                      None, None, None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert bool((got[live:2000] == 0).all()) and bool((got[:live] == 7).all())
    assert bool((got[2000] == 7).all())


def test_gradients_of_a_padded_buffer_without_tokens():
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward, router_order
    H = 96
    order = router_order(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    n = torch.ones(H, device="cuda")
    j = block_join(torch.empty(0, H, device="cuda"), randn(50, H, dtype=torch.bfloat16), order,
                   torch.empty(0, 2, device="cuda"), post_weight=n, norm_weight=n)
    torch.full((50, H), 7.0, dtype=torch.bfloat16, device="cuda")   # (what the allocator gives next)
    got = block_join_backward(j, d_x=torch.empty(0, H, device="cuda"),
                              d_h=torch.empty(0, H, dtype=torch.bfloat16, device="cuda"))
    assert got.expert_rows.shape == (50, H) and bool((got.expert_rows == 0).all())
    assert bool((got.norm_weight == 0).all()) and bool((got.post_weight == 0).all())


@pytest.mark.parametrize("T,H,K,x_type", [(2000, 7168, 8, torch.bfloat16), (1600, 4104, 3, torch.float32),
                                          (1000, 7936, 5, torch.bfloat16), (6000, 2048, 6, torch.bfloat16)])
def test_a_ring_gives_the_bits_of_small_calls_every_time(T, H, K, x_type):
    # many tokens to a block, whose rows come through a ring of stages, against calls of
    # few tokens, whose rows do not: x' is summed in the same order
    from moe_expert_layer_histogram_gb300 import block_join, block_join_backward
    a = make(T, H, K, x_type=x_type, w_type=x_type, post=False)
    want = []
    for t in range(0, T, 100):
        few = slice(t, min(t + 100, T))
        b = dict(a, order=a["order"].rows.view(T, K)[few].contiguous(),
                 **{n: a[n][few].contiguous() for n in ("x", "weights", "shared", "gate")})
        want.append(block_join(**b).x)
    want = torch.cat(want)
    dx, dh = randn(T, H, seed=80, dtype=x_type), randn(T, H, seed=81, dtype=torch.bfloat16)
    first = None
    for _ in range(30):
        j = block_join(**a)
        g = block_join_backward(j, dx, dh)
        assert torch.equal(j.x, want)
        now = [j.h, g.x, g.expert_rows, g.weights, g.shared, g.gate, g.norm_weight]
        first = first or now
        assert all(torch.equal(p, q) for p, q in zip(now, first))
