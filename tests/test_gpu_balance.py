"""Router balance: top-k ids, weights, counts, mean probabilities, the loss and
the gradient of the logits, against a plain 64-bit implementation.

Tolerances.  With u = 2^-24 (fp32 rounding) and logits within R of their row's
maximum, exp(x - m) is off by at most (R + 2) u of itself (the rounding of
x - m, then expf's two ulp), a sum of E such terms by E u more, the quotient by
two roundings: every probability and weight is within
eps = (2 R + E + 8) u of itself.  Sums over T tokens add T u.  A gradient
p (g - dot) + w (dw - wdot) is off by at most 3 eps of the sum of its terms'
magnitudes; bf16 gradients add half an ulp, 2^-8, of the result.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def reference(x, K, coef, mask=None, d_loss=None, dw=None):
    """Plain 64-bit forward and gradient; x float64 [T, E]."""
    T, E = x.shape
    live = np.isfinite(np.max(np.where(np.isneginf(x), -np.inf, x), axis=1)) if T else np.zeros(0, bool)
    live = live & (np.ones(T, bool) if mask is None else mask.astype(bool))
    ids = np.argsort(-x, axis=1, kind="stable")[:, :K].astype(np.int32)
    w, p = np.zeros((T, K)), np.zeros((T, E))
    for t in range(T):
        if not live[t]:
            ids[t] = -1
            continue
        m = x[t].max()
        p[t] = np.exp(x[t] - m)
        p[t] /= p[t].sum()
        w[t] = np.exp(x[t, ids[t]] - m)
        w[t] /= w[t].sum()
    n = int(live.sum())
    counts = np.bincount(ids[ids >= 0].reshape(-1), minlength=E)
    out = dict(ids=ids, weights=w, counts=counts, live=live, p=p)
    out["mean"] = p.sum(0) / max(n, 1)
    f = counts * E / (K * max(n, 1))
    out["loss"] = coef * float(f @ out["mean"])
    g = (d_loss or 0.0) * coef * f / max(n, 1)
    dot = p @ g
    d = p * (g[None] - dot[:, None])
    mag = p * (np.abs(g)[None] + np.abs(dot)[:, None])
    if dw is not None:
        wdot = (w * dw).sum(1, keepdims=True)
        for t in np.nonzero(live)[0]:
            d[t, ids[t]] += w[t] * (dw[t] - wdot[t])
            mag[t, ids[t]] += w[t] * (np.abs(dw[t]) + (w[t] * np.abs(dw[t])).sum())
    out["d"], out["mag"] = d, mag
    return out


def run(logits, K, coef, mask=None, d_loss=None, dw=None, out=None):
    from moe_expert_layer_histogram_gb300 import router_balance, router_balance_backward
    r = router_balance(logits, K, coef, mask=mask)
    dl = None if d_loss is None else torch.tensor(d_loss, dtype=torch.float32, device="cuda")
    d = router_balance_backward(logits, r, d_loss=dl, d_weights=dw, out=out)
    torch.cuda.synchronize()
    return r, d


def check(logits, K, coef=0.01, mask=None, d_loss=1.5, dw=None):
    x = logits.double().cpu().numpy()
    T, E = x.shape
    npm = None if mask is None else mask.cpu().numpy()
    ref = reference(x, K, coef, npm, d_loss, None if dw is None else dw.double().cpu().numpy())
    r, d = run(logits, K, coef, mask, d_loss, dw)
    finite = x[np.isfinite(x)]
    R = float(finite.max() - finite.min()) if finite.size else 0.0
    eps = (2 * R + E + 8) * U
    assert np.array_equal(r.ids.cpu().numpy(), ref["ids"])
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    assert np.all(np.abs(r.weights.double().cpu().numpy() - ref["weights"]) <= eps * ref["weights"])
    sums = eps + (T + 8) * U
    assert np.all(np.abs(r.mean_probs.double().cpu().numpy() - ref["mean"]) <= sums * ref["mean"])
    assert abs(float(r.loss) - ref["loss"]) <= (sums + E * U) * abs(ref["loss"])
    tol = 3 * eps * ref["mag"]
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref["d"])
    assert d.dtype == logits.dtype
    err = np.abs(d.double().cpu().numpy() - ref["d"])
    assert np.all(err <= tol + 1e-38), float(np.max(err - tol))
    return r, d, ref


def draw(T, E, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * scale).to(dtype).cuda()


def draw_dw(T, K, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    return torch.randn(T, K, generator=g).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (2, 3, 3), (7, 31, 4), (8, 32, 6),
                                   (9, 33, 1), (16, 8, 2), (63, 96, 6), (64, 128, 8),
                                   (65, 129, 8), (200, 256, 16), (300, 257, 5), (333, 384, 8),
                                   (100, 385, 7), (70, 511, 16), (129, 512, 16), (2500, 64, 6),
                                   (5000, 40, 3)])
def test_matches_64_bits(T, E, K, dtype):
    check(draw(T, E, T + E, dtype), K, dw=draw_dw(T, K, T))


@pytest.mark.parametrize("T", [1, 5, 40, 333, 3000])
def test_masks(T):
    logits = draw(T, 48, T, scale=3.0)
    g = torch.Generator().manual_seed(T)
    mask = torch.rand(T, generator=g) < 0.5
    check(logits, 4, mask=mask.cuda(), dw=draw_dw(T, 4, T))
    # uint8 masks, any value but 0 is live
    check(logits, 4, mask=(mask.to(torch.uint8) * 7).cuda(), dw=draw_dw(T, 4, T))


def test_no_live_token():
    logits = draw(37, 20, 3)
    r, d = run(logits, 3, 0.5, mask=torch.zeros(37, dtype=torch.bool, device="cuda"), d_loss=1.0,
               dw=draw_dw(37, 3, 0))
    assert float(r.loss) == 0.0 and int(r.counts.sum()) == 0 and float(r.mean_probs.sum()) == 0.0
    assert bool((r.ids == -1).all()) and not bool(r.weights.any()) and not bool(d.any())


def test_no_token():
    from moe_expert_layer_histogram_gb300 import router_balance, router_balance_backward
    logits = torch.empty(0, 16, device="cuda")
    r = router_balance(logits, 2, 1.0)
    assert float(r.loss) == 0.0 and not bool(r.counts.any()) and r.ids.shape == (0, 2)
    assert router_balance_backward(logits, r, d_loss=torch.ones((), device="cuda")).shape == (0, 16)


def test_infinite_and_lowest_logits():
    lowest = torch.finfo(torch.float32).min
    x = draw(12, 24, 9)
    x[0] = -float("inf")                       # leaves nothing: not live
    x[1, 3:] = -float("inf")                   # fewer finite logits than K
    x[2] = lowest                              # every expert at the type's lowest value: live
    x[3, :20] = lowest
    x[4] = 0.0                                 # all tied
    x[5, 7] = 80.0                             # one expert takes all
    ref = reference(x.double().cpu().numpy(), 4, 0.01, None, 1.0, None)
    r, d = run(x, 4, 0.01, d_loss=1.0)
    assert np.array_equal(r.ids.cpu().numpy(), ref["ids"])
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    assert bool((r.ids[0] == -1).all()) and not bool(d[0].any())
    assert np.allclose(r.weights.cpu().numpy(), ref["weights"], rtol=2e-5, atol=0)
    assert np.isclose(float(r.loss), ref["loss"], rtol=2e-5)
    assert bool(torch.isfinite(d).all())
    assert np.all(np.abs(d.double().cpu().numpy() - ref["d"]) <= 2e-5 * ref["mag"] + 1e-38)


def test_nan_stays_in_its_token():
    x = draw(20, 40, 5)
    x[6, 11] = float("nan")
    x[7] = float("nan")
    r, d = run(x, 4, 0.01, d_loss=1.0, dw=draw_dw(20, 4, 1))
    ids = r.ids.cpu().numpy()
    assert ids.min() >= 0 and ids.max() < 40 and np.isnan(float(r.loss))
    assert bool(torch.isnan(d[6]).all()) and bool(torch.isnan(d[7]).all())
    rest = [t for t in range(20) if t not in (6, 7)]
    assert bool(torch.isfinite(r.weights[rest]).all()) and bool(torch.isfinite(d[rest]).all())


def test_ties_take_the_lower_index():
    x = torch.zeros(40, 70, device="cuda")
    x[1::2] = torch.round(draw(20, 70, 2) * 2) / 2
    x[3, 5], x[3, 6] = -0.0, 0.0
    check(x, 6, dw=draw_dw(40, 6, 2))
    check(x.bfloat16(), 6, dw=draw_dw(40, 6, 2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_and_unaligned_starts(dtype):
    big = draw(50, 101, 4, dtype)
    view = big[:, 3:68]                        # 65 experts, odd row stride, odd start
    outbig = torch.full((50, 90), 7.0, dtype=dtype, device="cuda")
    out = outbig[:, 5:70]
    dw = draw_dw(50, 6, 4)
    _, want, ref = check(view, 6, dw=dw)
    run(view, 6, 0.01, d_loss=1.5, dw=dw, out=out)
    assert torch.equal(out, want)
    assert bool((outbig[:, :5] == 7).all()) and bool((outbig[:, 70:] == 7).all())


def test_gradient_parts_add_up():
    x, dw = draw(90, 60, 8), draw_dw(90, 5, 8)
    check(x, 5, d_loss=2.0, dw=None)
    check(x, 5, d_loss=None, dw=dw)
    _, d = run(x, 5, 0.01, d_loss=None, dw=None)
    assert not bool(d.any())


def test_gradient_against_differences():
    # central differences of the 64-bit forward along random directions; the
    # step 1e-5 leaves the top-k alone, the error of the difference is of the
    # order of its square
    T, E, K, coef, d_loss = 30, 24, 4, 3.0, 0.7
    x, dw = draw(T, E, 11), draw_dw(T, K, 11)
    _, d = run(x, K, coef, d_loss=d_loss, dw=dw)
    base, dwn = x.double().cpu().numpy(), dw.double().cpu().numpy()
    rng = np.random.default_rng(0)
    for _ in range(4):
        v = rng.standard_normal((T, E))
        h = 1e-5
        vals = []
        for s in (h, -h):
            r = reference(base + s * v, K, coef)
            vals.append(d_loss * r["loss"] + float((r["weights"] * dwn).sum()))
        num = (vals[0] - vals[1]) / (2 * h)
        got = float((d.double().cpu().numpy() * v).sum())
        assert abs(num - got) <= 1e-5 * max(1.0, float(np.abs(d.double().cpu().numpy() * v).sum()))


def test_same_bits_every_time_and_on_another_stream():
    x, dw = draw(4000, 96, 6), draw_dw(4000, 6, 6)
    r0, d0 = run(x, 6, 0.1, d_loss=1.0, dw=dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r1, d1 = run(x, 6, 0.1, d_loss=1.0, dw=dw)
    assert torch.equal(r0.loss, r1.loss) and torch.equal(r0.mean_probs, r1.mean_probs)
    assert torch.equal(d0, d1) and torch.equal(r0.weights, r1.weights)


def test_routes_as_the_layer_does():
    from moe_expert_layer_histogram_gb300 import moe_route_permute_static, router_balance
    T, E, K = 500, 384, 8
    x = draw(T, E, 12)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * K, dtype=torch.int32, device="cuda")
    moe_route_permute_static(x, T, E, K, ids, w, off, perm, torch.cuda.current_stream().cuda_stream)
    r = router_balance(x, K)
    assert torch.equal(r.ids, ids) and torch.equal(r.counts, off[1:] - off[:-1])
    assert float((r.weights - w).abs().max()) <= 1e-6


def test_graph_capture():
    from moe_expert_layer_histogram_gb300 import router_balance, router_balance_backward
    x, dw = draw(700, 64, 1), draw_dw(700, 6, 1)
    one = torch.ones((), device="cuda")
    run(x, 6, 0.1, d_loss=1.0, dw=dw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = router_balance(x, 6, 0.1)
        d = router_balance_backward(x, r, d_loss=one, d_weights=dw)
    x.copy_(draw(700, 64, 2))
    g.replay()
    torch.cuda.synchronize()
    r2, d2 = run(x, 6, 0.1, d_loss=1.0, dw=dw)
    assert torch.equal(r.ids, r2.ids) and torch.equal(r.loss, r2.loss) and torch.equal(d, d2)


def test_wrapper_refusals():
    from moe_expert_layer_histogram_gb300 import MoEError, router_balance, router_balance_backward
    x = draw(8, 16, 0)
    with pytest.raises(TypeError):
        router_balance(x.half(), 2)
    with pytest.raises(ValueError):
        router_balance(x.t(), 2)
    with pytest.raises(ValueError):
        router_balance(x.cpu(), 2)
    with pytest.raises(ValueError):
        router_balance(x, 2, mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(MoEError) as e:
        router_balance(x, 17)
    assert e.value.code == 1
    with pytest.raises(MoEError) as e:
        router_balance(torch.zeros(2, 513, device="cuda"), 2)
    assert e.value.code == 2
    with pytest.raises(MoEError) as e:                    # rows that overlap
        router_balance(x[:1].expand(8, 16), 2)
    assert e.value.code == 1
    r = router_balance(x, 2)
    with pytest.raises(ValueError):
        router_balance_backward(x[:4], r)
    with pytest.raises(ValueError):
        router_balance_backward(x, r, d_weights=torch.zeros(8, 3, device="cuda"))
    with pytest.raises(ValueError):
        router_balance_backward(x, r, d_loss=torch.zeros(2, device="cuda"))
