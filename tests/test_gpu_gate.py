"""The router's gate: chosen experts, weights, counts and the gradient of the
logits, and the expert order of slots, against plain implementations in 64 bits.

Tolerances.  u = 2^-24.  A sigmoid or power of e is within 6 u of itself (expf's
two ulp, a sum, a quotient) plus, for powers of differences, |d| u for the
difference's rounding; with logits within R of their largest, and sums of n terms
n u more, every weight is within eps = (2 R + n + 16) u of itself, n = K
(normalised) or E.  A gradient is off by at most 3 eps of the sum of its terms'
magnitudes; bf16 gradients add half an ulp, 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def sort_key(c):
    """Sorting key, ascending: NaN first, then by falling value."""
    return np.where(np.isnan(c), -np.inf, -c), ~np.isnan(c)


def order_of(c):
    k, real = sort_key(c)
    return np.lexsort((np.arange(c.size), k, real))


def reference(x, K, score="softmax", bias=None, groups=1, group_top=None, group_score="top2",
              normalize=True, scale=1.0, mask=None, dw=None):
    """x float64 [T, E], one token at a time."""
    T, E = x.shape
    group_top = group_top or groups
    size = E // groups
    ids = np.full((T, K), -1, np.int32)
    w, d, mag = np.zeros((T, K)), np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        l = x[t]
        if (mask is not None and not mask[t]) or np.all(np.isneginf(l)):
            continue
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max())
            s = s / s.sum()
        c = l.copy() if bias is None else s + bias
        c[np.isneginf(l)] = -np.inf
        kept = np.ones(E, bool)
        if group_top < groups:
            per = c.reshape(groups, size)
            value = np.empty(groups)
            for g in range(groups):
                best = per[g][order_of(per[g])][:2]
                if group_score == "max" or size == 1:
                    value[g] = best[0]
                elif bias is None:
                    at = order_of(per[g])[:2] + g * size
                    value[g] = sum(-np.inf if np.isneginf(l[i]) else s[i] for i in at)
                else:
                    value[g] = best.sum()
            kept[:] = False
            for g in order_of(value)[:group_top]:
                kept[g * size:(g + 1) * size] = True
        among = np.nonzero(kept)[0]
        ids[t] = among[order_of(c[among])][:K]
        sk = s[ids[t]]
        total = sk.sum()
        u = np.zeros(K) if total == 0 else sk / total
        w[t] = scale * (u if normalize else sk)
        if dw is None:
            continue
        if normalize:
            ds = scale * (dw[t] - (u * dw[t]).sum()) * u          # times s_k
            m = abs(scale) * (np.abs(dw[t]) + (u * np.abs(dw[t])).sum()) * u
        else:
            ds, m = scale * dw[t] * sk, abs(scale * dw[t]) * sk
        if score == "sigmoid":
            d[t, ids[t]], mag[t, ids[t]] = ds * (1 - sk), m * (1 - sk)
        else:
            d[t], mag[t] = -s * ds.sum(), s * m.sum()
            d[t, ids[t]] += ds
            mag[t, ids[t]] += m
            if normalize:
                d[t, np.setdiff1d(np.arange(E), ids[t])] = 0.0     # (the sum of ds is 0)
    counts = np.bincount(ids[ids >= 0].reshape(-1), minlength=E)
    return dict(ids=ids, weights=w, counts=counts, d=d, mag=mag)


def run(logits, K, dw=None, out=None, **kw):
    from moe_expert_layer_histogram_gb300 import router_gate, router_gate_backward
    r = router_gate(logits, K, **kw)
    d = None if dw is None else router_gate_backward(logits, r, dw, out=out)
    torch.cuda.synchronize()
    return r, d


def check(logits, K, dw=True, out=None, **kw):
    x = logits.double().cpu().numpy()
    T, E = x.shape
    g = torch.Generator(device="cuda").manual_seed(5)
    dw = torch.randn(T, K, generator=g, device="cuda") if dw else None
    np_kw = {k: v.double().cpu().numpy() if k == "bias" and v is not None
             else v.cpu().numpy() if torch.is_tensor(v) else v for k, v in kw.items()}
    ref = reference(x, K, dw=None if dw is None else dw.double().cpu().numpy(), **np_kw)
    r, d = run(logits, K, dw, out, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ref["ids"])
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    finite = x[np.isfinite(x)]
    R = float(finite.max() - finite.min()) if finite.size else 0.0
    eps = (2 * R + (K if kw.get("normalize", True) else E) + 16) * U
    err = np.abs(r.weights.double().cpu().numpy() - ref["weights"])
    assert np.all(err <= eps * np.abs(ref["weights"]) + 2.0 ** -140), err.max()
    if d is not None:
        tol = 3 * eps * ref["mag"] + 2.0 ** -140
        if logits.dtype is torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref["d"])
        err = np.abs(d.double().cpu().numpy() - ref["d"])
        assert np.all(err <= tol), (err - tol).max()
    return r, d, ref


def logits_of(T, E, dtype=torch.float32, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * spread).to(dtype)


def bias_of(E, size=0.05, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(E, generator=g, device="cuda") * size


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,K,groups,group_top,group_score,dtype", [
    (1, 1, 1, 1, 1, "max", torch.float32),
    (16, 64, 6, 1, 1, "max", torch.float32),
    (33, 8, 2, 4, 2, "top2", torch.float32),
    (70, 384, 8, 8, 4, "top2", torch.bfloat16),
    (40, 510, 16, 3, 1, "max", torch.float32),
    (50, 512, 16, 32, 9, "top2", torch.float32),
    (37, 505, 5, 5, 3, "top2", torch.bfloat16),
    (31, 28 * 17, 7, 17, 17, "max", torch.float32),
    (64, 7, 7, 7, 7, "top2", torch.float32),
    (64, 7, 3, 7, 3, "top2", torch.bfloat16),
])
def test_gate(score, normalize, with_bias, T, E, K, groups, group_top, group_score, dtype):
    check(logits_of(T, E, dtype), K, score=score, normalize=normalize,
          bias=bias_of(E, 0.05 if score == "sigmoid" else 0.3 / E) if with_bias else None,
          groups=groups, group_top=group_top, group_score=group_score, scale=2.5)


def test_many_tokens_and_a_mask():
    T, E, K = 5000, 384, 8
    mask = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(3),
                      device="cuda") > 0.3
    check(logits_of(T, E, torch.bfloat16), K, score="sigmoid", bias=bias_of(E), groups=8,
          group_top=4, mask=mask)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(score):
    # few distinct logits and biases: most choices are ties, also of groups
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(0, 3, (200, 96), generator=g, device="cuda").float()
    for bias in (None, torch.zeros(96, device="cuda"),
                 torch.randint(0, 2, (96,), generator=g, device="cuda").float()):
        check(x, 8, score=score, bias=bias, groups=12, group_top=5)


@pytest.mark.parametrize("gap", [0.0, 2.0 ** -24, 2.0 ** -30, -2.0 ** -30, 2.0 ** -45])
def test_choices_that_fp32_cannot_tell_apart(gap):
    # bias_e = 1 - sigmoid(l_e) + tiny steps: all choices near 1.  The biases are
    # fp32 numbers, so the 64-bit choices differ by their roundings (about 2^-25)
    T, E, K = 64, 64, 8
    x = logits_of(1, E, seed=4).repeat(T, 1)
    b = (1.0 - torch.sigmoid(x[0].double()) + gap * torch.arange(E, device="cuda").double()).float()
    r, _, ref = check(x, K, score="sigmoid", bias=b)
    assert len(np.unique(ref["ids"][0])) == K
    check(x, K, score="sigmoid", bias=b, groups=16, group_top=3)


@pytest.mark.parametrize("score,b", [("sigmoid", 100.0), ("softmax", 100.0), ("softmax", 1e-4)])
def test_large_and_small_biases(score, b):
    check(logits_of(100, 256), 8, score=score, bias=bias_of(256, b), groups=4, group_top=2)


def test_wide_logits():
    # saturated sigmoids, sums that underflow
    x = logits_of(200, 64, spread=60.0)
    check(x, 6, score="softmax", dw=False)
    for normalize in (True, False):
        check(x.clamp(-80, 80), 6, score="sigmoid", normalize=normalize, dw=False)
    # the chosen experts' scores all underflow in fp32: still weights of sum 1
    r, _ = run(logits_of(50, 64) - 150.0, 6, score="sigmoid")
    assert torch.all((r.weights.sum(1) - 1).abs() < 1e-6)


def test_dead_tokens_and_disabled_experts():
    x = logits_of(60, 48)
    x[3] = float("-inf")
    x[7, 5:] = float("-inf")            # fewer experts than K
    x[:, 20:24] = float("-inf")         # a whole group
    x[9, :44] = float("-inf")
    for bias in (None, bias_of(48)):
        for score in ("softmax", "sigmoid"):
            r, d, _ = check(x, 8, score=score, bias=bias, groups=12, group_top=6, dw=score == "sigmoid")
            assert torch.all(r.ids[3] == -1) and torch.all(r.weights[3] == 0)
            if d is not None:
                assert torch.all(d[3] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 2)])
def test_biases_as_far_apart_as_fp32_has_them(score, groups, group_top):
    bias = torch.full((64,), 3e38, device="cuda")
    bias[::3] = -3e38
    bias[5::7] = 0.0
    check(logits_of(40, 64), 8, score=score, bias=bias, groups=groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("E", [6, 64, 384])
def test_gradient_in_place(score, normalize, E):
    x = logits_of(300, E)
    dw = torch.randn(300, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    r, want = run(x, 4, dw, score=score, normalize=normalize)
    _, got = run(x, 4, dw, out=x, score=score, normalize=normalize)
    assert got is x and torch.equal(got, want)


def test_settings_go_by_their_values():
    # (a scale in a tensor that is changed between two calls)
    x, scale = logits_of(8, 16), torch.ones(())
    one = run(x, 2, scale=scale)[0].weights
    scale.fill_(3.0)
    assert torch.equal(run(x, 2, scale=scale)[0].weights, run(x, 2, scale=3.0)[0].weights)
    assert not torch.equal(run(x, 2, scale=scale)[0].weights, one)


def test_infinite_biases():
    b = bias_of(64)
    b[7] = float("inf")
    b[50] = float("inf")
    b[10] = float("-inf")
    r, _, _ = check(logits_of(40, 64), 6, score="sigmoid", bias=b)
    assert torch.all(r.ids[:, 0] == 7) and torch.all(r.ids[:, 1] == 50)


def test_nan_logits_come_first():
    x = logits_of(40, 64)
    x[5, 33] = float("nan")
    x[5, 40] = -float("nan")
    r, d = run(x, 6, torch.ones(40, 6, device="cuda"), score="sigmoid", bias=bias_of(64), groups=4,
               group_top=2)
    assert r.ids[5, :2].tolist() == [33, 40]
    assert torch.all(torch.isnan(r.weights[5]))
    others = [t for t in range(40) if t != 5]
    assert torch.all(torch.isfinite(r.weights[others])) and torch.all(torch.isfinite(d[others]))


def test_every_token_masked_and_no_tokens():
    mask = torch.zeros(10, dtype=torch.uint8, device="cuda")
    r, d, _ = check(logits_of(10, 16), 4, mask=mask)
    assert torch.all(d == 0) and torch.all(r.counts == 0)
    r, d = run(torch.empty(0, 16, device="cuda"), 4, torch.empty(0, 4, device="cuda"))
    assert r.ids.shape == (0, 4) and torch.all(r.counts == 0) and d.shape == (0, 16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,ld", [(0, 75), (1, 72), (3, 76), (4, 72)])
def test_strided_rows(dtype, offset, ld):
    big = logits_of(50, ld + 8, dtype)
    x = torch.as_strided(big, (50, 64), (ld, 1), offset)
    out = torch.full((50 * ld + 8,), 7.0, device="cuda", dtype=dtype)
    view = torch.as_strided(out, (50, 64), (ld, 1), offset)
    keep = torch.ones_like(out, dtype=torch.bool)
    torch.as_strided(keep, (50, 64), (ld, 1), offset).fill_(False)
    check(x, 6, out=view, score="sigmoid", groups=4, group_top=2)
    assert torch.all(out[keep] == 7)


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False),
                                             ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, normalize):
    T, E, K = 6, 24, 4
    x = logits_of(T, E, seed=8)
    dw = logits_of(T, K, seed=9)
    kw = dict(score=score, normalize=normalize, scale=1.5, bias=bias_of(E), groups=4, group_top=3)
    _, d = run(x, K, dw, **kw)
    base, npdw = x.double().cpu().numpy(), dw.double().cpu().numpy()
    np_kw = dict(kw, bias=kw["bias"].double().cpu().numpy())
    h = 1e-6
    for e in range(E):
        plus, minus = base.copy(), base.copy()
        plus[:, e] += h
        minus[:, e] -= h
        f = [(reference(v, K, **np_kw)["weights"] * npdw).sum(1) for v in (plus, minus)]
        # (differences of 64-bit values: 1e-9; the gradient itself 1e-5 of terms of order 4)
        assert np.all(np.abs((f[0] - f[1]) / (2 * h) - d[:, e].double().cpu().numpy()) < 5e-5)


def test_same_bits_every_time_and_in_a_graph():
    x, dw = logits_of(3000, 384, torch.bfloat16), logits_of(3000, 8, seed=3)
    kw = dict(score="sigmoid", bias=bias_of(384), groups=8, group_top=4)
    first, d = run(x, 8, dw, **kw)
    from moe_expert_layer_histogram_gb300 import router_gate, router_gate_backward, router_order
    o = router_order(first.ids, 384)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        router_gate(x, 8, **kw)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            r2 = router_gate(x, 8, **kw)
            d2 = router_gate_backward(x, r2, dw)
            o2 = router_order(r2.ids, 384)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in ((first.ids, r2.ids), (first.weights, r2.weights), (first.counts, r2.counts),
                 (d, d2), (o.slots, o2.slots), (o.offsets, o2.offsets), (o.rows, o2.rows)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,E", [(0, 5), (1, 1), (31, 4), (33, 512), (2048, 384), (2049, 384),
                                 (8192, 7), (24577, 64), (262144, 384), (300000, 512)])
@pytest.mark.parametrize("dead", [0.0, 0.3, 1.0])
def test_order(n, E, dead):
    from moe_expert_layer_histogram_gb300 import router_order
    rng = np.random.default_rng(n + E)
    ids = rng.integers(0, E, n).astype(np.int32)
    ids[rng.random(n) < dead] = -1
    if n > 10:
        ids[5], ids[6] = E, 2 ** 31 - 1                       # of no expert either
    o = router_order(torch.from_numpy(ids).cuda(), E)
    torch.cuda.synchronize()
    key = np.where((ids >= 0) & (ids < E), ids, E)
    slots = np.argsort(key, kind="stable").astype(np.int32)
    rows = np.empty(n, np.int32)
    rows[slots] = np.arange(n, dtype=np.int32)
    rows[key == E] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    assert np.array_equal(o.slots.cpu().numpy(), slots)
    assert np.array_equal(o.offsets.cpu().numpy(), offsets)
    assert np.array_equal(o.rows.cpu().numpy(), rows)


def test_order_agrees_with_the_allocation_free_routing():
    from moe_expert_layer_histogram_gb300 import (moe_route_permute_static, router_gate,
                                                  router_order)
    T, E, K = 700, 64, 6
    x = logits_of(T, E)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * K, dtype=torch.int32, device="cuda")
    moe_route_permute_static(x, T, E, K, ids, w, off, perm,
                             torch.cuda.current_stream().cuda_stream)
    r = router_gate(x, K)
    o = router_order(r.ids, E)
    assert torch.equal(r.ids, ids) and torch.equal(o.slots, perm) and torch.equal(o.offsets, off)
    assert torch.all((r.weights - w).abs() <= 64 * U * w)


def test_two_streams_at_once():
    from moe_expert_layer_histogram_gb300 import router_gate, router_order
    xs = [logits_of(4000, 384, seed=i) for i in range(2)]
    kw = dict(score="sigmoid", bias=bias_of(384), groups=8, group_top=4)
    want = [run(x, 8, **kw)[0] for x in xs]
    orders = [router_order(r.ids, 384) for r in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                r = router_gate(x, 8, **kw)
                got.append((r, router_order(r.ids, 384)))
        torch.cuda.synchronize()
        for (r, o), w, wo in zip(got, want, orders):
            assert torch.equal(r.ids, w.ids) and torch.equal(r.counts, w.counts)
            assert torch.equal(o.slots, wo.slots)


def test_refusals():
    from moe_expert_layer_histogram_gb300 import (MoEError, router_gate, router_gate_backward,
                                                  router_order)
    x = logits_of(8, 24)
    for kw in (dict(groups=5), dict(groups=4, group_top=5), dict(groups=0), dict(scale=float("nan")),
               dict(groups=12, group_top=1)):                 # (two experts for four places)
        with pytest.raises(MoEError):
            router_gate(x, 4, **kw)
    for kw in (dict(score="tanh"), dict(group_score="mean"), dict(bias=bias_of(23)),
               dict(bias=bias_of(24).double()), dict(mask=torch.ones(7, device="cuda") > 0)):
        with pytest.raises(ValueError):
            router_gate(x, 4, **kw)
    with pytest.raises(TypeError):
        router_gate(x.half(), 4)
    with pytest.raises(MoEError):
        router_gate(x, 25)
    r = router_gate(x, 4)
    with pytest.raises(ValueError):
        router_gate_backward(x[:7], r, torch.zeros(7, 4, device="cuda"))
    with pytest.raises(ValueError):
        router_gate_backward(x, r, torch.zeros(8, 3, device="cuda"))
    with pytest.raises(ValueError):
        router_order(r.ids.long(), 24)
    with pytest.raises(MoEError):
        router_order(r.ids, 513)


@pytest.mark.parametrize("groups,group_top,group_score,dtype", [
    (6, 3, "top2", torch.float32), (3, 1, "max", torch.float32), (12, 5, "max", torch.float32),
    (6, 3, "top2", torch.bfloat16), (24, 9, "top2", torch.bfloat16)])
def test_groups_that_are_no_power_of_two_take_the_same_way(groups, group_top, group_score, dtype):
    # lanes without a group once sent every token through the choice in 64 bits, forty times
    # the work of all the rest: no more than four times what 8 groups take says that few
    # tokens go there
    from moe_expert_layer_histogram_gb300 import router_gate
    x = logits_of(32768, 384, dtype)

    def time(groups, group_top):
        best = float("inf")
        for _ in range(12):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(4):
                router_gate(x, 8, groups=groups, group_top=group_top, group_score=group_score)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        return best
    time(8, 4)
    few, many = time(groups, group_top), time(8, 4)
    assert few <= 4.0 * many, (few / 4, many / 4)
    y = x[:300]
    for score in ("softmax", "sigmoid"):
        check(y, 8, score=score, groups=groups, group_top=group_top, group_score=group_score)
