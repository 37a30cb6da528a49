"""Argument checks of the router gate, the expert order and the block join: every
refusal is found on the host before any CUDA call, so these run without a GPU."""
import ctypes

import pytest

GOOD = 1 << 20
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def m():
    from moe_expert_layer_histogram_gb300 import _build
    _build.build()
    import moe_expert_layer_histogram_gb300 as m
    m.lib()
    return m


GATE = dict(score=1, groups=8, group_top=4, group_score=1, normalize=1, scale=1.0)
BAD_GATE = [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID),
    (dict(ld=63), INVALID), (dict(dtype=2), INVALID), (dict(logits=None), INVALID),
    (dict(logits=GOOD + 2), INVALID), (dict(dtype=1, logits=GOOD + 1), INVALID),
    (dict(config=None), INVALID), (dict(score=2), INVALID), (dict(group_score=-1), INVALID),
    (dict(groups=0), INVALID), (dict(groups=7), INVALID), (dict(group_top=0), INVALID),
    (dict(group_top=9), INVALID), (dict(group_top=1, K=9), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ids=None), INVALID), (dict(ids=GOOD + 2), INVALID),
    (dict(E=513, ld=513, groups=1, group_top=1), UNSUPPORTED), (dict(K=17), UNSUPPORTED),
    (dict(groups=64, group_top=64), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(T=2 ** 31 - 1, K=1), UNSUPPORTED), (dict(T=2 ** 31 - 65535, K=1), UNSUPPORTED)]


def split(m, over):
    config = dict(GATE)
    rest = {}
    for k, v in over.items():
        (config if k in config else rest)[k] = v
    if "config" not in rest:
        rest["config"] = m.MoEGateConfig(**config)
    return rest


@pytest.mark.parametrize("over,code", BAD_GATE + [
    (dict(weights=None), INVALID), (dict(weights=GOOD + 1), INVALID), (dict(counts=None), INVALID),
    (dict(counts=GOOD + 2), INVALID), (dict(bias=GOOD + 2), INVALID)])
def test_gate_forward_refusals(m, over, code):
    a = dict(logits=GOOD, dtype=0, ld=64, bias=None, mask=None, T=32, E=64, K=6, config=None,
             ids=GOOD, weights=GOOD, counts=GOOD)
    a.update(split(m, over))
    assert m.lib().moe_gate_forward(*a.values(), None) == code


@pytest.mark.parametrize("over,code", BAD_GATE + [
    (dict(ld_d=63), INVALID), (dict(d_weights=None), INVALID), (dict(d_weights=GOOD + 2), INVALID),
    (dict(d_logits=None), INVALID), (dict(d_logits=GOOD + 2), INVALID),
    (dict(T=0, logits=None, ids=None), 0)])
def test_gate_backward_refusals(m, over, code):
    a = dict(logits=GOOD, dtype=0, ld=64, T=32, E=64, K=6, config=None, ids=GOOD, d_weights=GOOD,
             d_logits=GOOD, ld_d=64)
    over = dict(over)
    if over.get("E") == 513:
        over["ld_d"] = 513
    a.update(split(m, over))
    assert m.lib().moe_gate_backward(*a.values(), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), INVALID), (dict(E=0), INVALID), (dict(E=513), UNSUPPORTED), (dict(ids=None), INVALID),
    (dict(slots=None), INVALID), (dict(offsets=None), INVALID), (dict(ids=GOOD + 2), INVALID),
    (dict(slots=GOOD + 1), INVALID), (dict(offsets=GOOD + 2), INVALID), (dict(rows=GOOD + 2), INVALID),
    (dict(ws=None), INVALID), (dict(ws=GOOD + 2), INVALID), (dict(nbytes=100), INVALID)])
def test_order_refusals(m, over, code):
    a = dict(ids=GOOD, n=100000, E=64, slots=GOOD, offsets=GOOD, rows=GOOD, ws=GOOD, nbytes=1 << 30)
    a.update(over)
    assert m.lib().moe_order(*a.values(), None) == code


def test_order_workspace(m):
    ws = m.moe_order_workspace
    assert ws(-1, 8) == 0 and ws(8, 0) == 0 and ws(8, 513) == 0 and ws(2048, 64) == 0
    assert 0 < ws(2049, 64) <= ws(2 ** 31 - 1, 512) <= 129 * 513 * 4


JOIN = dict(T=8, H=64, K=2, x_type=0, weight_type=1, gate_type=0, scale=1.0, eps=1e-6, x=GOOD,
            ld_x=64, expert_rows=GOOD, ld_rows=64, rows=16, row_of_slot=GOOD, weights=GOOD,
            shared=GOOD, ld_shared=64, gate=GOOD, post_weight=GOOD, norm_weight=GOOD)
BAD_JOIN = [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(K=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(x_type=2), INVALID), (dict(weight_type=-1), INVALID), (dict(gate_type=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(K=17), UNSUPPORTED), (dict(H=16385), UNSUPPORTED), (dict(shared=None), INVALID),
    (dict(K=0, shared=None, gate=None), INVALID), (dict(row_of_slot=None), INVALID),
    (dict(weights=None), INVALID), (dict(expert_rows=None), INVALID),
    (dict(expert_rows=GOOD + 1), INVALID), (dict(ld_rows=63), INVALID),
    (dict(row_of_slot=GOOD + 2), INVALID), (dict(weights=GOOD + 2), INVALID),
    (dict(shared=GOOD + 1), INVALID), (dict(ld_shared=63), INVALID), (dict(gate=GOOD + 2), INVALID),
    (dict(post_weight=GOOD + 1), INVALID), (dict(norm_weight=GOOD + 1), INVALID),
    (dict(join=None), INVALID)]


def joined(m, a, over):
    join = dict(JOIN)
    for k, v in over.items():
        if k in join:
            join[k] = v
        else:
            a[k] = v
    if "join" not in over:
        a["join"] = m.MoEJoin(**join)
    return a.values()


@pytest.mark.parametrize("over,code", BAD_JOIN + [
    (dict(x=None), INVALID), (dict(x=GOOD + 2), INVALID), (dict(ld_x=63), INVALID),
    (dict(x_out=None), INVALID), (dict(x_out=GOOD + 2), INVALID), (dict(ld_out=63), INVALID),
    (dict(h=None), INVALID), (dict(norm_weight=None), INVALID), (dict(ld_h=63), INVALID),
    (dict(h=GOOD + 1), INVALID), (dict(codes=GOOD, ld_codes=63), INVALID),
    (dict(codes=GOOD, code_scales=None), INVALID), (dict(post_rstd=GOOD + 2), INVALID),
    (dict(norm_rstd=GOOD + 1), INVALID), (dict(T=0, x=None, h=None, x_out=None), 0)])
def test_join_forward_refusals(m, over, code):
    a = dict(join=None, x_out=GOOD, ld_out=64, h=GOOD, ld_h=64, codes=None, ld_codes=64,
             code_scales=GOOD, post_rstd=GOOD, norm_rstd=GOOD)
    assert m.lib().moe_join_forward(*joined(m, a, over), None) == code


@pytest.mark.parametrize("over,code", BAD_JOIN + [
    (dict(norm_weight=None), INVALID), (dict(x_out=None), INVALID), (dict(norm_rstd=None), INVALID),
    (dict(post_rstd=None), INVALID), (dict(d_h=None), INVALID), (dict(post_weight=None), INVALID),
    (dict(gate=None), INVALID), (dict(ld_out=63), INVALID), (dict(ld_dxo=63), INVALID),
    (dict(ld_dh=63), INVALID), (dict(ld_dx=63), INVALID), (dict(ld_drows=63), INVALID),
    (dict(ld_dshared=63), INVALID), (dict(d_x=GOOD + 2), INVALID), (dict(d_h=GOOD + 1), INVALID),
    (dict(d_rows=GOOD + 1), INVALID), (dict(live_rows=GOOD + 1), INVALID),
    (dict(d_weights=GOOD + 2), INVALID), (dict(d_shared=GOOD + 1), INVALID),
    (dict(d_gate=GOOD + 2), INVALID), (dict(d_post=GOOD + 1), INVALID),
    (dict(d_norm=GOOD + 1), INVALID), (dict(ws=None), INVALID), (dict(ws=GOOD + 8), INVALID),
    (dict(nbytes=64), INVALID), (dict(K=0), INVALID)])
def test_join_backward_refusals(m, over, code):
    a = dict(join=None, x_out=GOOD, ld_out=64, post_rstd=GOOD, norm_rstd=GOOD, d_xo=GOOD, ld_dxo=64,
             d_h=GOOD, ld_dh=64, d_x=GOOD, ld_dx=64, d_rows=GOOD, ld_drows=64, live_rows=GOOD,
             d_weights=GOOD, d_shared=GOOD, ld_dshared=64, d_gate=GOOD, d_post=GOOD, d_norm=GOOD,
             ws=GOOD, nbytes=1 << 30)
    assert m.lib().moe_join_backward(*joined(m, a, over), None) == code


def test_join_workspace(m):
    ws = m.moe_join_workspace
    assert ws(0, 64) == 0 and ws(8, 0) == 0 and ws(8, 16385) == 0
    assert 0 < ws(1, 1) <= ws(2 ** 31 - 1, 16384) <= 64 << 20


def test_structures_have_the_header_s_sizes(m):
    # (moe_gate_config: six words; moe_join: eight words, nine 8-byte members and
    # an int32 with its padding)
    assert ctypes.sizeof(m.MoEGateConfig) == 24
    assert ctypes.sizeof(m.MoEJoin) == 32 + 8 * 12
