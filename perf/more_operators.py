"""Cases and plain forms of the grouped router gate, the block join with its norms, and the INT8
operators.

Five kinds of pass, each in a plain form (elementary torch operations) and through the package's
entry points:

  gate     the router's gate: sigmoid or softmax scores, a bias that only the choice sees, the best
           groups of experts, top-k within them, weights (router_gate); the routed slots in expert
           order (router_order); in training the gradient of the logits (router_gate_backward);
  join     the end of a block: the experts' rows added up by their weights, a shared expert behind
           its sigmoid gate, a norm after the block, the scaled sum with the residual, the norm
           before the next block (block_join); in training all its gradients (block_join_backward);
  chain    a serving step between two blocks: the join, its last norm quantised to 8 bits, and the
           next projection from those codes (block_join, int8_matmul);
  linear   y = x W^T with W in 8 bits and one scale per output channel, x quantised per token within
           the call (int8_linear);
  experts  the experts' products on routed rows from 8-bit weights: gather and quantise, gate/up
           product, SwiGLU, quantise again, down product (int8_experts).

Definitions.
  Gate: s = sigmoid(l) or softmax(l); the choice goes by c = s + b, ties to the lower index.  A
  group's score is its largest c ("max") or the sum of its two largest ("top2").  Weights are the
  chosen experts' s, divided by their sum where `normalize`, times `scale`.
  Join: y = sum_k w_k rows[row_of_slot_k] + sigmoid(gate) shared; x' = x + scale N(y; post_weight),
  stored in x's type; h = N(x'; norm_weight) of the stored x'.  N(v; w) = w v / sqrt(mean(v^2) +
  eps).
  8 bits: per row s = amax / 127 rounded to fp32, codes round(v / s) to even within +-127, the
  quotient rounded to fp32; a zero row has s = 0 and zero codes.
"""
import math

import torch

own = False

I8_MAX = 127.0
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's gate: 16 tokens, one group; latency is all that counts
        dict(name="gate_t16", op="gate", T=16, E=64, K=6, score="softmax", bias=False, groups=1,
             group_top=1, group_score="max", normalize=True, dtype="f32", masked=0.0, train=False),
        # a training micro-batch of bf16 logits, a twentieth of it padding
        dict(name="gate_t4096", op="gate", T=4096, E=384, K=8, score="sigmoid", bias=True, groups=8,
             group_top=4, group_score="top2", normalize=True, dtype="bf16", masked=0.05,
             train=True),
        # the 32K-token batch
        dict(name="gate_t32768", op="gate", T=32768, E=384, K=8, score="sigmoid", bias=True,
             groups=8, group_top=4, group_score="top2", normalize=True, dtype="f32", masked=0.0,
             train=True),
        # odd sizes behind a dense block: no experts, ragged tokens, rows off 16 bytes
        dict(name="join_t333_odd", op="join", T=333, H=2001, K=0, shared=True, gate=False,
             post=True, dtype="bf16", masked=0.0, train=True),
        # a micro-batch of the 64-expert layer with an fp32 residual stream
        dict(name="join_t512", op="join", T=512, H=2048, K=6, shared=True, gate=True, post=True,
             dtype="f32", masked=0.1, train=True),
        # a training micro-batch of the large layer
        dict(name="join_t4096", op="join", T=4096, H=7168, K=8, shared=True, gate=True, post=False,
             dtype="bf16", masked=0.0, train=True),
        # one decoded token between two blocks
        dict(name="chain_t1", op="chain", T=1, H=7168, K=8, N=4096, shared=True, gate=True,
             post=False, dtype="bf16"),
        # one token through a projection every token takes
        dict(name="linear_t1", op="linear", T=1, K=7168, N=4096),
        # odd sizes: ragged tokens, an odd width
        dict(name="linear_t333_odd", op="linear", T=333, K=2000, N=1001),
        # prefill through the same projection as linear_t1
        dict(name="linear_t8192", op="linear", T=8192, K=7168, N=4096),
        # decode: 64 tokens, about eight rows for each of 64 experts
        dict(name="experts_t64", op="experts", T=64, E=64, topk=8, H=7168, I=2048, clamp=0.0),
        # a prefill batch of the smaller layer, gate and up clamped
        dict(name="experts_t4096", op="experts", T=4096, E=64, topk=6, H=2048, I=1024, clamp=7.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "join", "chain", "linear", "experts"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 3, 4, 8, 16])
        size = _log_int(rng, 4, 384 // groups)
        group_top = rng.randint(max(1, groups // 4), groups)
        return dict(op=op, T=_log_int(rng, 1, 32768), E=groups * size,
                    K=rng.randint(1, min(group_top * size, 8)),
                    score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.7,
                    groups=groups, group_top=group_top, group_score=rng.choice(["top2", "max"]),
                    normalize=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.choice([0.0, 0.0, 0.1, 0.5]), train=rng.random() < 0.7)
    if op == "join":
        K = rng.choice([0, 1, 2, 4, 6, 8])
        shared = K == 0 or rng.random() < 0.6
        return dict(op=op, T=_log_int(rng, 1, 4096), H=_log_int(rng, 64, 7168), K=K, shared=shared,
                    gate=shared and rng.random() < 0.6, post=rng.random() < 0.5,
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.1]),
                    train=rng.random() < 0.6)
    if op == "chain":
        return dict(op=op, T=_log_int(rng, 1, 256), H=16 * _log_int(rng, 8, 448),
                    K=rng.randint(1, 8), N=_log_int(rng, 100, 4096), shared=rng.random() < 0.6,
                    gate=False, post=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]))
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 1, 8192), K=16 * _log_int(rng, 8, 448),
                    N=_log_int(rng, 100, 4096))
    E = _log_int(rng, 4, 64)
    H, I = 16 * _log_int(rng, 16, 448), 128 * _log_int(rng, 2, 16)
    topk = rng.randint(1, min(E, 8))
    # (at most the work of the largest listed case)
    T = _log_int(rng, 1, max(2, min(8192, int(9e10 / (topk * H * I)))))
    return dict(op=op, T=T, E=E, topk=topk, H=H, I=I, clamp=rng.choice([0.0, 7.0]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _weights_8bit(g, E, N, K, std=0.02):
    """int8 codes [E, N, K] and fp32 scales [E, N] of N(0, std) weights."""
    codes = torch.empty(E, N, K, device="cuda", dtype=torch.int8)
    scales = torch.empty(E, N, device="cuda", dtype=torch.float32)
    for e in range(E):
        w = _randn(g, N, K) * std
        s = w.abs().amax(1) / I8_MAX
        codes[e] = torch.round(w / s[:, None]).to(torch.int8)
        scales[e] = s
    return codes, scales


def _routing(g, T, E, k, masked):
    """A routed batch as router_order leaves it: row_of_slot int32 [T * k], live rows."""
    ids = _randn(g, T, E).topk(k, dim=1).indices
    live = torch.rand(T, generator=g, device="cuda") >= masked
    key = torch.where(live[:, None], ids, E).reshape(-1)
    slots = torch.sort(key, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(T * k, device="cuda")
    rows = torch.where(live.repeat_interleave(k), rows, -1)
    offsets = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    return slots.to(torch.int32), offsets, rows.to(torch.int32), live


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    if op == "gate":
        E, K = case["E"], case["K"]
        st = dict(case=case, logits=_randn(g, T, E).to(_dtype(case["dtype"])), bias=None, mask=None,
                  d_weights=_randn(g, T, K) * 0.01, scale=2.5)
        if case["bias"]:
            st["bias"] = _randn(g, E) * (0.05 if case["score"] == "sigmoid" else 0.2 / E)
        if case["masked"]:
            st["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"]
        return st
    if op in ("join", "chain"):
        H, K, t = case["H"], case["K"], _dtype(case["dtype"])
        st = dict(case=case, x=(_randn(g, T, H) * 2).to(t), rows=None, slots=None, offsets=None,
                  row_of_slot=None, weights=None, shared=None, gate=None, post=None, scale=0.5,
                  norm=(1.0 + 0.1 * _randn(g, H)).to(t))
        if K:
            st["slots"], st["offsets"], st["row_of_slot"], live = _routing(
                g, T, max(16, 2 * K), K, case.get("masked", 0.0))
            w = torch.rand(T, K, generator=g, device="cuda") + 0.1
            st["weights"] = w / w.sum(1, keepdim=True) * live[:, None]
            st["rows"] = _randn(g, T * K, H).to(torch.bfloat16)
        if case["shared"]:
            st["shared"] = _randn(g, T, H).to(torch.bfloat16)
        if case["gate"]:
            st["gate"] = _randn(g, T)
        if case["post"]:
            st["post"] = (1.0 + 0.1 * _randn(g, H)).to(t)
        if op == "join":
            st["d_x"] = (_randn(g, T, H) * 0.01).to(t)
            st["d_h"] = (_randn(g, T, H) * 0.01).to(torch.bfloat16)
        else:
            w, ws = _weights_8bit(g, 1, case["N"], H)
            st["w"], st["ws"] = w[0], ws[0]
        return st
    if op == "linear":
        w, ws = _weights_8bit(g, 1, case["N"], case["K"])
        return dict(case=case, x=_randn(g, T, case["K"]).to(torch.bfloat16), w=w[0], ws=ws[0])
    E, k, H, I = case["E"], case["topk"], case["H"], case["I"]
    w13, s13 = _weights_8bit(g, E, 2 * I, H)
    w2, s2 = _weights_8bit(g, E, H, I)
    slots, offsets, _, _ = _routing(g, T, E, k, 0.0)
    counts = (offsets[1:] - offsets[:-1]).long()
    return dict(case=case, x=_randn(g, T, H).to(torch.bfloat16), w13=w13, s13=s13, w2=w2, s2=s2,
                slots=slots, offsets=offsets,
                expert=torch.repeat_interleave(torch.arange(E, device="cuda"), counts),
                capacity=int(counts.max()))


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"gate": _gate_own, "join": _join_own, "chain": _chain_own, "linear": _linear_own,
                "experts": _experts_own}[op](state)
    if op == "gate":
        return _gate_plain(state)
    if op == "join":
        return _join_plain(state)
    if op == "chain":
        x, h, _, _, _ = _join_values(state)
        y = _quantized(h) @ (state["w"].float() * state["ws"][:, None]).t()
        return dict(x=x.to(state["x"].dtype), y=y.to(torch.bfloat16))
    if op == "linear":
        w = state["w"].float() * state["ws"][:, None]
        return (_quantized(state["x"].float()) @ w.t()).to(torch.bfloat16)
    return _experts_plain(state)


def _gate_own(st):
    from moe_expert_layer_histogram_gb300 import (router_gate, router_gate_backward, router_order)
    c = st["case"]
    r = router_gate(st["logits"], c["K"], score=c["score"], bias=st["bias"], groups=c["groups"],
                    group_top=c["group_top"], group_score=c["group_score"],
                    normalize=c["normalize"], scale=st["scale"], mask=st["mask"])
    o = router_order(r.ids, c["E"])
    out = dict(ids=r.ids, weights=r.weights, counts=r.counts, slots=o.slots, offsets=o.offsets,
               rows=o.rows)
    if c["train"]:
        out["d_logits"] = router_gate_backward(st["logits"], r, st["d_weights"])
    return out


def _gate_plain(st):
    c = st["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    # (64 bits: experts whose choices differ by less than 32 bits tell apart)
    x = st["logits"].double()
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        s = torch.exp(x - x.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    choice = s if st["bias"] is None else s + st["bias"].double()
    if c["group_top"] < G:
        per = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        best = per[:, :, :2].sum(2) if c["group_score"] == "top2" else per[:, :, 0]
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["group_top"]]
        kept = torch.zeros(T, G, device=x.device, dtype=torch.bool).scatter_(1, order, True)
        choice = torch.where(kept.repeat_interleave(E // G, 1), choice, float("-inf"))
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :K]
    sk = s.gather(1, ids)
    total = sk.sum(1, keepdim=True)
    w = st["scale"] * (sk / total if c["normalize"] else sk)
    live = torch.ones(T, device=x.device, dtype=torch.bool) if st["mask"] is None else st["mask"]
    key = torch.where(live[:, None], ids, E).reshape(-1)
    slots = torch.sort(key, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(T * K, device=x.device)
    counts = torch.zeros(E + 1, device=x.device, dtype=torch.int64).scatter_add_(
        0, key, torch.ones_like(key))[:E]
    offsets = torch.zeros(E + 1, device=x.device, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    out = dict(ids=torch.where(live[:, None], ids, -1).to(torch.int32),
               weights=(w * live[:, None]).float(), counts=counts.to(torch.int32),
               slots=slots.to(torch.int32), offsets=offsets,
               rows=torch.where(live.repeat_interleave(K), rows, -1).to(torch.int32))
    if c["train"]:
        dw = st["d_weights"].double()
        if c["normalize"]:
            ds = st["scale"] / total * (dw - (dw * sk / total).sum(1, keepdim=True))
        else:
            ds = st["scale"] * dw
        if c["score"] == "sigmoid":
            d = torch.zeros_like(x).scatter_(1, ids, ds * sk * (1.0 - sk))
        else:
            d = -s * (ds * sk).sum(1, keepdim=True)
            d = d.scatter_add(1, ids, ds * sk)
        out["d_logits"] = (d * live[:, None]).to(st["logits"].dtype)
    return out


def _join_own(st):
    from moe_expert_layer_histogram_gb300 import (RouterOrder, block_join, block_join_backward)
    order = None
    if st["case"]["K"]:
        order = RouterOrder(st["slots"], st["offsets"], st["row_of_slot"])
    j = block_join(st["x"], expert_rows=st["rows"], order=order, weights=st["weights"],
                   shared=st["shared"], gate=st["gate"], post_weight=st["post"], scale=st["scale"],
                   norm_weight=st["norm"], eps=EPS)
    out = dict(x=j.x, h=j.h)
    if st["case"]["train"]:
        d = block_join_backward(j, d_x=st["d_x"], d_h=st["d_h"])
        out.update(d_x=d.x, d_rows=d.expert_rows, d_weights=d.weights, d_shared=d.shared,
                   d_gate=d.gate, d_post=d.post_weight, d_norm=d.norm_weight)
    return out


def _join_values(st):
    """x' (in fp32, of the stored values), h (fp32), and the block's sum, gate and rows."""
    c = st["case"]
    T, H, K = c["T"], c["H"], c["K"]
    y = torch.zeros(T, H, device=st["x"].device)
    z = sig = None
    if K:
        r = st["row_of_slot"].long()
        z = st["rows"].float()[r.clamp(min=0)] * (r >= 0)[:, None]
        z = z.view(T, K, H)
        y = y + (st["weights"][:, :, None] * z).sum(1)
    if st["shared"] is not None:
        if st["gate"] is not None:
            sig = (1.0 / (1.0 + torch.exp(-st["gate"])))[:, None]
            y = y + sig * st["shared"].float()
        else:
            y = y + st["shared"].float()
    n = y
    if st["post"] is not None:
        n = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * st["post"].float()
    x = (st["x"].float() + st["scale"] * n).to(st["x"].dtype).float()
    h = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * st["norm"].float()
    return x, h, y, sig, z


def _norm_back(v, w, d):
    """Gradients of N(v; w) for d: of v, and of w."""
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    u = v * r
    dw = (d * u).sum(0)
    d = d * w
    return r * (d - u * (d * u).mean(1, keepdim=True)), dw


def _join_plain(st):
    c = st["case"]
    x, h, y, sig, z = _join_values(st)
    out = dict(x=x.to(st["x"].dtype), h=h.to(torch.bfloat16))
    if not c["train"]:
        return out
    T, K, H = c["T"], c["K"], c["H"]
    d, d_norm = _norm_back(x, st["norm"].float(), st["d_h"].float())
    d = d + st["d_x"].float()
    out.update(d_x=d.to(st["x"].dtype), d_rows=None, d_weights=None, d_shared=None, d_gate=None,
               d_post=None, d_norm=d_norm.to(st["norm"].dtype))
    d = st["scale"] * d
    if st["post"] is not None:
        d, d_post = _norm_back(y, st["post"].float(), d)
        out["d_post"] = d_post.to(st["post"].dtype)
    if K:
        out["d_weights"] = (d[:, None, :] * z).sum(2)
        r = st["row_of_slot"].long()
        d_rows = torch.zeros(T * K + 1, H, device=d.device, dtype=torch.bfloat16)
        d_rows[torch.where(r < 0, T * K, r)] = (st["weights"][:, :, None] * d[:, None, :]).to(
            torch.bfloat16).view(T * K, H)
        d_rows[T * K] = 0
        out["d_rows"] = d_rows[:T * K]
    if st["shared"] is not None:
        out["d_shared"] = (d if sig is None else sig * d).to(torch.bfloat16)
        if sig is not None:
            out["d_gate"] = (d * st["shared"].float()).sum(1) * (sig * (1.0 - sig))[:, 0]
    return out


def _chain_own(st):
    from moe_expert_layer_histogram_gb300 import RouterOrder, block_join, int8_matmul
    j = block_join(st["x"], expert_rows=st["rows"],
                   order=RouterOrder(st["slots"], st["offsets"], st["row_of_slot"]),
                   weights=st["weights"], shared=st["shared"], gate=st["gate"],
                   post_weight=st["post"], scale=st["scale"], norm_weight=st["norm"], eps=EPS,
                   quantize=True)
    return dict(x=j.x, y=int8_matmul(j.codes, j.code_scales, st["w"], st["ws"]))


def _linear_own(st):
    from moe_expert_layer_histogram_gb300 import int8_linear
    return int8_linear(st["x"], st["w"], st["ws"])


def _experts_own(st):
    from moe_expert_layer_histogram_gb300 import int8_experts
    c = st["case"]
    return int8_experts(st["x"], st["slots"], st["offsets"], c["topk"], st["w13"], st["s13"],
                        st["w2"], st["s2"], clamp=c["clamp"])


def _quantized(v):
    """The values that v's rows in 8 bits stand for, fp32."""
    s = v.abs().amax(1, keepdim=True)
    s = s / torch.full_like(s, I8_MAX)  # (a Python divisor would become a multiplication)
    q = torch.where(s > 0, v / s, torch.zeros_like(v))
    return torch.round(q).clamp(-I8_MAX, I8_MAX) * s


def _experts_plain(st):
    c = st["case"]
    E, I = c["E"], c["I"]
    x = _quantized(st["x"].float())[st["slots"].long() // c["topk"]]
    e = st["expert"]
    pos = torch.arange(e.numel(), device=e.device) - st["offsets"].long()[e]
    rows = torch.zeros(E, st["capacity"], c["H"], device=e.device)
    rows[e, pos] = x
    gu = torch.bmm(rows, (st["w13"].float() * st["s13"][:, :, None]).transpose(1, 2))[e, pos]
    gate, up = gu[:, :I], gu[:, I:]
    if c["clamp"]:
        gate, up = gate.clamp(-c["clamp"], c["clamp"]), up.clamp(-c["clamp"], c["clamp"])
    h = _quantized(gate / (1.0 + torch.exp(-gate)) * up)
    rows = torch.zeros(E, st["capacity"], I, device=e.device)
    rows[e, pos] = h
    return torch.bmm(rows, (st["w2"].float() * st["s2"][:, :, None]).transpose(1, 2))[e, pos].to(
        torch.bfloat16)


# ---------------------------------------------------------------- work
def work(case):
    op, T = case["op"], case["T"]
    if op == "gate":
        E, K = case["E"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        n = T * E * size + 8 * T * K + 8 * T * K + 8 * E + (T if case["masked"] else 0)
        if case["train"]:
            n += T * E * size + 4 * T * K
        return {"bytes": n, "flops": 10 * T * E}
    if op in ("join", "chain"):
        H, K = case["H"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        live = T * K * (1.0 - case.get("masked", 0.0))
        # x, x', the experts' rows, the shared expert, h; the norms' weights
        n = 2 * T * H * size + 2 * live * H + 8 * T * K + size * H * (1 + case["post"])
        n += 2 * T * H * case["shared"] + 4 * T * case["gate"]
        flops = T * H * (2 * K + 12)
        if op == "chain":
            return {"bytes": n + case["N"] * (H + 4) + 2 * T * case["N"],
                    "flops": flops + 2 * T * H * case["N"]}
        n += 2 * T * H
        if case["train"]:
            # d_x', d_h, x' again, d_x; the rows' gradients, the shared expert's
            n += T * H * (3 * size + 2) + 2 * T * K * H + 4 * T * K
            n += 2 * T * H * case["shared"] + 4 * T * case["gate"] + size * H * (1 + case["post"])
            flops += T * H * (4 * K + 20)
        return {"bytes": n, "flops": flops}
    if op == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * T * (K + N) + N * K + 4 * N, "flops": 2 * T * N * K}
    E, k, H, I = case["E"], case["topk"], case["H"], case["I"]
    rows = T * k
    touched = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": 2 * T * H + 4 * rows + 4 * (E + 1) + touched * (3 * H * I + 4 * (2 * I + H))
            + 2 * rows * H, "flops": 6 * rows * H * I}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    if work(case)["flops"] > 1.2e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(st)
    if op == "linear":
        return _exact_rows(st["x"].double()) @ (st["w"].double() * st["ws"].double()[:, None]).T
    if op == "experts":
        return _exact_experts(st)
    if op == "chain":
        x, h = _exact_join_forward(st)[:2]
        w = st["w"].double() * st["ws"].double()[:, None]
        return dict(x=x, y=_exact_rows(h) @ w.T)
    return _exact_join(st)


def _exact_rows(v):
    """Rows of v (64 bits) as their codes and 32-bit scales give them back.  The scale and the
    quotient that is coded are rounded to fp32, as the format says."""
    s = (v.abs().max(dim=1, keepdim=True).values / I8_MAX).float().double()
    q = (v / torch.where(s == 0, torch.ones_like(s), s)).float().double()
    return torch.round(q).clamp(-I8_MAX, I8_MAX) * s


def _exact_gate(st):
    c = st["case"]
    T, E, K = c["T"], c["E"], c["K"]
    live = list(range(T)) if st["mask"] is None else st["mask"].nonzero()[:, 0].tolist()
    at = torch.tensor(live, device="cuda", dtype=torch.long)
    x = st["logits"].double()[at]
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    choice = s + (0.0 if st["bias"] is None else st["bias"].double())
    size = E // c["groups"]
    allowed = torch.zeros_like(choice, dtype=torch.bool)
    grouped = choice.unflatten(1, (c["groups"], size))
    if c["group_score"] == "max":
        value = grouped.amax(2)
    else:
        value = torch.topk(grouped, min(2, size), dim=2).values.sum(2)
    chosen = torch.argsort(-value, dim=1, stable=True)[:, :c["group_top"]]
    for j in range(c["group_top"]):
        for i in range(size):
            allowed.scatter_(1, chosen[:, j:j + 1] * size + i, True)
    ids = torch.argsort(-choice.masked_fill(~allowed, -math.inf), dim=1, stable=True)[:, :K]
    picked = torch.gather(s, 1, ids)
    w = picked
    if c["normalize"]:
        w = w / picked.sum(1, keepdim=True)
    w = st["scale"] * w
    weights = torch.zeros(T, K, device="cuda", dtype=torch.float64)
    weights[at] = w
    out = dict(ids=None, weights=weights, counts=None, slots=None, offsets=None, rows=None)
    if c["train"]:
        # the weights' Jacobian by the chosen scores, then the scores' by the logits
        dw = st["d_weights"].double()[at]
        if c["normalize"]:
            total = picked.sum(1, keepdim=True)
            g = (st["scale"] * dw - (w * dw).sum(1, keepdim=True)) / total
        else:
            g = st["scale"] * dw
        ds = torch.zeros_like(s).scatter_(1, ids, g)
        if c["score"] == "sigmoid":
            d = ds * s * (1 - s)
        else:
            d = s * (ds - (s * ds).sum(1, keepdim=True))
        out["d_logits"] = torch.zeros(T, E, device="cuda", dtype=torch.float64)
        out["d_logits"][at] = d
    return out


def _exact_join_forward(st):
    c = st["case"]
    T, H, K = c["T"], c["H"], c["K"]
    y = torch.zeros(T, H, device="cuda", dtype=torch.float64)
    for k in range(K):
        r = st["row_of_slot"].view(T, K)[:, k].long()
        t = (r >= 0).nonzero()[:, 0]
        y[t] += st["weights"][t, k].double()[:, None] * st["rows"][r[t]].double()
    gate = torch.ones(T, 1, device="cuda", dtype=torch.float64)
    if st["gate"] is not None:
        gate = torch.sigmoid(st["gate"].double())[:, None]
    if st["shared"] is not None:
        y += gate * st["shared"].double()
    n = y
    if st["post"] is not None:
        n = st["post"].double() * y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    x = st["x"].double() + st["scale"] * n
    x = x.to(st["x"].dtype).double()  # (as it is stored)
    h = st["norm"].double() * x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    return x, h, y, gate


def _exact_norm_back(v, w, d):
    """d N(v; w) / dv by the quotient rule, with q = mean(v^2) + eps."""
    q = v.square().mean(1, keepdim=True) + EPS
    dv = (d * w) * q.rsqrt() - v * (d * w * v).mean(1, keepdim=True) * q.pow(-1.5)
    return dv, torch.einsum("th,th->h", d, v * q.rsqrt())


def _exact_join(st):
    c = st["case"]
    T, H, K = c["T"], c["H"], c["K"]
    x, h, y, gate = _exact_join_forward(st)
    out = dict(x=x, h=h)
    if not c["train"]:
        return out
    d, d_norm = _exact_norm_back(x, st["norm"].double(), st["d_h"].double())
    d = d + st["d_x"].double()
    out.update(d_x=d, d_rows=None, d_weights=None, d_shared=None, d_gate=None, d_post=None,
               d_norm=d_norm)
    d = d * st["scale"]
    if st["post"] is not None:
        d, out["d_post"] = _exact_norm_back(y, st["post"].double(), d)
    if K:
        out["d_rows"] = torch.zeros(T * K, H, device="cuda", dtype=torch.float64)
        out["d_weights"] = torch.zeros(T, K, device="cuda", dtype=torch.float64)
        for k in range(K):
            r = st["row_of_slot"].view(T, K)[:, k].long()
            t = (r >= 0).nonzero()[:, 0]
            out["d_rows"][r[t]] = st["weights"][t, k].double()[:, None] * d[t]
            out["d_weights"][t, k] = torch.einsum("th,th->t", d[t], st["rows"][r[t]].double())
    if st["shared"] is not None:
        out["d_shared"] = gate * d
        if st["gate"] is not None:
            dot = torch.einsum("th,th->t", d, st["shared"].double())
            out["d_gate"] = dot * (gate * (1 - gate))[:, 0]
    return out


def _exact_experts(st):
    c = st["case"]
    I, k = c["I"], c["topk"]
    y = torch.zeros(c["T"] * k, c["H"], device="cuda", dtype=torch.float64)
    off = st["offsets"].tolist()
    x = _exact_rows(st["x"].double())
    for e in range(c["E"]):
        if off[e] == off[e + 1]:
            continue
        src = st["slots"][off[e]:off[e + 1]].long().div(k, rounding_mode="floor")
        gu = x[src] @ (st["w13"][e].double() * st["s13"][e].double()[:, None]).T
        if c["clamp"]:
            gu = gu.clamp(-c["clamp"], c["clamp"])
        h = _exact_rows(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
        y[off[e]:off[e + 1]] = h @ (st["w2"][e].double() * st["s2"][e].double()[:, None]).T
    return y
