"""Cases and plain forms of the router-balance and block-scaled FP8 operators.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and through the package's entry points:

  balance  the router's step in training: top-k, routing weights, per-expert
           counts, the balance loss, and the gradient of the logits from the
           loss and from the routing weights (router_balance,
           router_balance_backward);
  linear   y = x W^T with W in e4m3 and one fp32 scale per 128 x 128 block,
           x quantised per row and 128 columns within the call
           (blockscale_linear);
  dx       its input gradient dx = dy W from the same stored W
           (blockscale_linear_dx);
  experts  the experts' products of one layer on routed rows: gather and
           quantise, gate/up product, SwiGLU, re-quantise, down product
           (blockscale_experts).

Definitions.  Quantisation of a row's block of 128 columns: s = amax / 448
rounded to fp32, codes e4m3(x / s) of the quotient rounded to fp32 (both
roundings are the format's own); an all-zero block has s = 0 and zero codes.  Balance
loss over the n unmasked tokens, with p the softmax over all experts:
coef * sum_e f_e P_e, f_e = counts_e E / (K n), P_e = sum_t p_te / n.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a smoke-sized router step: latency is all that counts
        dict(name="balance_t16", op="balance", T=16, E=8, K=2, dtype="f32", masked=0.0, zipf=0.0),
        # a micro-batch of the 64-expert layer, a tenth of it padding
        dict(name="balance_t512", op="balance", T=512, E=64, K=6, dtype="f32", masked=0.1,
             zipf=0.0),
        # an 8K-token batch with skewed popularity, logits of a bf16 gate
        dict(name="balance_t8192", op="balance", T=8192, E=384, K=8, dtype="bf16", masked=0.05,
             zipf=1.1),
        # the 32K-token batch
        dict(name="balance_t32768", op="balance", T=32768, E=384, K=8, dtype="f32", masked=0.0,
             zipf=0.0),
        # one token through a gate/up projection every token takes
        dict(name="linear_t1", op="linear", T=1, K=7168, N=4096),
        # odd sizes: ragged tokens, a last block of 80 columns, an odd width
        dict(name="linear_t333_odd", op="linear", T=333, K=2000, N=1001),
        # prefill through the same projection as linear_t1
        dict(name="linear_t8192", op="linear", T=8192, K=7168, N=4096),
        # input gradient of a few sequences' last tokens
        dict(name="dx_t48", op="dx", T=48, K=7168, N=2048),
        # input gradient of a training micro-batch
        dict(name="dx_t4096", op="dx", T=4096, K=7168, N=4096),
        # decode: 64 tokens, about eight rows for each of 64 experts
        dict(name="experts_t64", op="experts", T=64, E=64, topk=8, H=7168, I=2048, clamp=0.0),
        # a 512-token batch of the smaller layer, gate and up clamped
        dict(name="experts_t512", op="experts", T=512, E=64, topk=6, H=2048, I=1024, clamp=7.0),
        # prefill: about a thousand rows for each of 64 experts
        dict(name="experts_t8192", op="experts", T=8192, E=64, topk=8, H=7168, I=2048, clamp=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "linear", "dx", "experts"])
    if op == "balance":
        E = _log_int(rng, 4, 384)
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, K=rng.randint(1, min(E, 8)),
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.0, 0.1, 0.5]),
                    zipf=rng.choice([0.0, 1.1]))
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 1, 8192), K=16 * _log_int(rng, 8, 448),
                    N=_log_int(rng, 100, 4096))
    if op == "dx":
        return dict(op=op, T=_log_int(rng, 1, 4096), K=16 * _log_int(rng, 8, 448),
                    N=_log_int(rng, 100, 4096))
    E = _log_int(rng, 4, 64)
    return dict(op=op, T=_log_int(rng, 1, 8192), E=E, topk=rng.randint(1, min(E, 8)),
                H=16 * _log_int(rng, 16, 448), I=128 * _log_int(rng, 2, 16),
                clamp=rng.choice([0.0, 7.0]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _draw_weights(g, E, N, K, std=0.02):
    """e4m3 codes [E, N, K] and fp32 scales [E, ceil(N/128), ceil(K/128)] of N(0, std)
    weights, quantised as a checkpoint's writer does it."""
    nb, kb = _blocks(N), _blocks(K)
    codes = torch.empty(E, N, K, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(E, nb, kb, device="cuda", dtype=torch.float32)
    for e in range(E):
        w = torch.zeros(nb * BLOCK, kb * BLOCK, device="cuda")
        w[:N, :K] = _randn(g, N, K) * std
        v = w.view(nb, BLOCK, kb, BLOCK)
        s = v.abs().amax(dim=(1, 3)) / E4M3_MAX
        codes[e] = (v / s[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:N, :K].to(
            torch.float8_e4m3fn)
        scales[e] = s
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    if op == "balance":
        E, K = case["E"], case["K"]
        logits = _randn(g, T, E)
        if case["zipf"]:
            rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
            logits = logits - case["zipf"] * torch.log(rank)
        logits = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        mask = None
        if case["masked"]:
            mask = torch.rand(T, generator=g, device="cuda") >= case["masked"]
        return dict(case=case, logits=logits, mask=mask, d_weights=_randn(g, T, K) * 0.01,
                    d_loss=torch.ones((), device="cuda") + 0.1 * _randn(g, 1)[0], coef=0.01)
    if op in ("linear", "dx"):
        w, ws = _draw_weights(g, 1, case["N"], case["K"])
        x = _randn(g, T, case["K"] if op == "linear" else case["N"])
        if op == "dx":
            x = x * 0.01
        return dict(case=case, x=x.to(torch.bfloat16), w=w[0], ws=ws[0])
    E, k, H, I = case["E"], case["topk"], case["H"], case["I"]
    w13, s13 = _draw_weights(g, E, 2 * I, H)
    w2, s2 = _draw_weights(g, E, H, I)
    # routed rows in expert order, as the permutation leaves them: slot t*k+j of each row
    ids = _randn(g, T, E).topk(k, dim=1).indices.reshape(-1)
    slots = torch.sort(ids, stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    return dict(case=case, x=_randn(g, T, H).to(torch.bfloat16), w13=w13, s13=s13, w2=w2, s2=s2,
                slots=slots, offsets=offsets, expert=torch.sort(ids, stable=True).values,
                capacity=int(counts.max()))


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if op == "balance":
        return _balance_own(state) if own else _balance_plain(state)
    if op == "linear":
        if own:
            from moe_expert_layer_histogram_gb300 import blockscale_linear
            return blockscale_linear(state["x"], state["w"], state["ws"])
        return (_quantized(state["x"]) @ _weight(state["w"], state["ws"]).t()).to(torch.bfloat16)
    if op == "dx":
        if own:
            from moe_expert_layer_histogram_gb300 import blockscale_linear_dx
            return blockscale_linear_dx(state["x"], state["w"], state["ws"])
        return (_quantized(state["x"]) @ _weight(state["w"], state["ws"])).to(torch.bfloat16)
    if own:
        from moe_expert_layer_histogram_gb300 import blockscale_experts
        return blockscale_experts(state["x"], state["slots"], state["offsets"],
                                  state["case"]["topk"], state["w13"], state["s13"], state["w2"],
                                  state["s2"], clamp=state["case"]["clamp"])
    return _experts_plain(state)


def _balance_own(st):
    from moe_expert_layer_histogram_gb300 import router_balance, router_balance_backward
    K = st["case"]["K"]
    r = router_balance(st["logits"], K, st["coef"], mask=st["mask"])
    d = router_balance_backward(st["logits"], r, d_loss=st["d_loss"], d_weights=st["d_weights"])
    return dict(ids=r.ids, weights=r.weights, counts=r.counts, loss=r.loss, d_logits=d)


def _balance_plain(st):
    E, K, coef = st["case"]["E"], st["case"]["K"], st["coef"]
    x = st["logits"].float()
    T = x.shape[0]
    live = torch.ones(T, device=x.device, dtype=torch.bool) if st["mask"] is None else st["mask"]
    p = torch.exp(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * live[:, None]
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)
    v, ids = v[:, :K], ids[:, :K]
    w = torch.exp(v - v[:, :1])
    w = w / w.sum(1, keepdim=True) * live[:, None]
    n = live.sum().clamp(min=1)
    hit = torch.zeros(T, E, device=x.device).scatter_(1, ids, 1.0) * live[:, None]
    counts = hit.sum(0)
    f = counts * E / (K * n)
    loss = coef * (f * (p.sum(0) / n)).sum()
    g = st["d_loss"] * coef * f / n
    d = p * (g - (p * g).sum(1, keepdim=True))
    dw = st["d_weights"]
    d = d.scatter_add(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    return dict(ids=torch.where(live[:, None], ids, -1).to(torch.int32), weights=w,
                counts=counts.to(torch.int32), loss=loss, d_logits=d.to(st["logits"].dtype))


def _quantized(x):
    """The values that x's block-quantised codes stand for, fp32."""
    rows, cols = x.shape
    kb = _blocks(cols)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - cols)).view(rows, kb, BLOCK)
    s = v.abs().amax(2, keepdim=True)
    s = s / torch.full_like(s, E4M3_MAX)  # (a Python divisor would become a multiplication)
    q = torch.where(s > 0, v / s, torch.zeros_like(v)).to(torch.float8_e4m3fn)
    return (q.float() * s).view(rows, kb * BLOCK)[:, :cols]


def _weight(codes, scales):
    """Dequantised weights [..., N, K], fp32."""
    N, K = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return codes.float() * s


def _experts_plain(st):
    c = st["case"]
    E, I = c["E"], c["I"]
    x = _quantized(st["x"])[st["slots"].long() // c["topk"]]
    e = st["expert"]
    pos = torch.arange(e.numel(), device=e.device) - st["offsets"].long()[e]
    rows = torch.zeros(E, st["capacity"], c["H"], device=e.device)
    rows[e, pos] = x
    gu = torch.bmm(rows, _weight(st["w13"], st["s13"]).transpose(1, 2))[e, pos]
    gate, up = gu[:, :I], gu[:, I:]
    if c["clamp"]:
        gate, up = gate.clamp(-c["clamp"], c["clamp"]), up.clamp(-c["clamp"], c["clamp"])
    h = _quantized(gate / (1.0 + torch.exp(-gate)) * up)
    rows = torch.zeros(E, st["capacity"], I, device=e.device)
    rows[e, pos] = h
    return torch.bmm(rows, _weight(st["w2"], st["s2"]).transpose(1, 2))[e, pos].to(torch.bfloat16)


# ---------------------------------------------------------------- work
def work(case):
    T = case["T"]
    if case["op"] == "balance":
        E, K = case["E"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * T * E * size + 12 * T * K + (T if case["masked"] else 0) + 4 * E + 8,
                "flops": 12 * T * E}
    if case["op"] in ("linear", "dx"):
        K, N = case["K"], case["N"]
        return {"bytes": 2 * T * (K + N) + N * K + 4 * _blocks(N) * _blocks(K),
                "flops": 2 * T * N * K}
    E, k, H, I = case["E"], case["topk"], case["H"], case["I"]
    rows = T * k
    touched = E * (1.0 - (1.0 - k / E) ** T)
    per = 3 * H * I + 4 * (_blocks(2 * I) * _blocks(H) + _blocks(H) * _blocks(I))
    return {"bytes": 2 * T * H + 4 * rows + 4 * (E + 1) + touched * per + 2 * rows * H,
            "flops": 6 * rows * H * I}


# ---------------------------------------------------------------- 64 bits
def _round_e4m3(q):
    """Nearest e4m3 value (ties to even) of |q| <= 448, in 64 bits."""
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(x):
    """x (64 bits) as its codes and 32-bit scales give it back, 64 bits.  The scale and the
    quotient that is coded are rounded to fp32, as the format says."""
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], BLOCK):
        b = x[:, j:j + BLOCK]
        s = (b.abs().max(dim=1, keepdim=True).values / E4M3_MAX).float().double()
        q = (b / torch.where(s == 0, torch.ones_like(s), s)).float().double()
        out[:, j:j + BLOCK] = _round_e4m3(q) * s
    return out


def _exact_weight(codes, scales):
    w = codes.to(torch.float64)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scales[i, j].double()
    return w


def exact(case, seed):
    if work(case)["flops"] > 1.2e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_rows(st["x"].double()) @ _exact_weight(st["w"], st["ws"]).T
    if case["op"] == "dx":
        return _exact_rows(st["x"].double()) @ _exact_weight(st["w"], st["ws"])
    if case["op"] == "experts":
        I, k = case["I"], case["topk"]
        y = torch.zeros(case["T"] * k, case["H"], device="cuda", dtype=torch.float64)
        off = st["offsets"].tolist()
        x = st["x"].double()
        for e in range(case["E"]):
            if off[e] == off[e + 1]:
                continue
            src = st["slots"][off[e]:off[e + 1]].long().div(k, rounding_mode="floor")
            gu = _exact_rows(x[src]) @ _exact_weight(st["w13"][e], st["s13"][e]).T
            if case["clamp"]:
                gu = gu.clamp(-case["clamp"], case["clamp"])
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            y[off[e]:off[e + 1]] = _exact_rows(h) @ _exact_weight(st["w2"][e], st["s2"][e]).T
        return y
    E, K = case["E"], case["K"]
    x = st["logits"].double()
    if st["mask"] is not None:
        x = x[st["mask"]]
    n = x.shape[0]
    live = torch.arange(case["T"], device="cuda") if st["mask"] is None else st["mask"].nonzero()[:, 0]
    dw = st["d_weights"].double()[live]
    p = torch.softmax(x, 1)
    ids = torch.argsort(x, dim=1, descending=True, stable=True)[:, :K]
    counts = torch.bincount(ids.reshape(-1), minlength=E).double()
    w = torch.softmax(x.gather(1, ids), 1)
    f = counts * E / (K * max(n, 1))
    loss = st["coef"] * torch.dot(f, p.sum(0)) / max(n, 1)
    g = st["d_loss"].double() * st["coef"] * f / max(n, 1)
    d = p * (g - p @ g[:, None])
    d.scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    weights = torch.zeros(case["T"], K, device="cuda", dtype=torch.float64)
    d_logits = torch.zeros(case["T"], E, device="cuda", dtype=torch.float64)
    weights[live], d_logits[live] = w, d
    return dict(ids=None, weights=weights, counts=None, loss=loss, d_logits=d_logits)
