"""The router's gate on torch tensors: scores with groups and a bias for
balance, the gradient of the logits, and the routed slots in expert order.

Thin wrappers of ``moe_gate_forward``, ``moe_gate_backward`` and ``moe_order``
(``include/moe.h`` states the formulas); work goes on torch's current stream.
"""
import functools
from operator import index

import torch

from . import MOE_GROUP, MOE_SCORE, MoEError, MoEGateConfig, lib
from ._tensors import check, fits, row_stride, stream_on

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


class RouterGate:
    """What the gate chose: ids int32 [T, K] and weights f32 [T, K] (-1 and 0 for
    tokens that are not live), counts int32 [E], and the settings."""
    __slots__ = ("ids", "weights", "counts", "top_k", "config")

    def __init__(self, ids, weights, counts, top_k, config):
        self.ids, self.weights, self.counts = ids, weights, counts
        self.top_k, self.config = top_k, config


class RouterOrder:
    """Routed slots in expert order: slots int32 [n] (those of no expert last),
    offsets int32 [E + 1], rows int32 [n] (the place of each slot, -1 for one of
    no expert)."""
    __slots__ = ("slots", "offsets", "rows")

    def __init__(self, slots, offsets, rows):
        self.slots, self.offsets, self.rows = slots, offsets, rows


@functools.lru_cache(maxsize=64)
def _config(score, groups, group_top, group_score, normalize, scale):
    if score not in MOE_SCORE or group_score not in MOE_GROUP:
        raise ValueError("score: one of %s, group_score: one of %s"
                         % (sorted(MOE_SCORE), sorted(MOE_GROUP)))
    return MoEGateConfig(MOE_SCORE[score], groups, group_top, MOE_GROUP[group_score], normalize,
                         scale)


def _logits(t, name):
    """(element type code, row stride) of logits or their gradient."""
    if t.dtype is _F32:
        return 0, row_stride(t, _F32, name)
    if t.dtype is _BF16:
        return 1, row_stride(t, _BF16, name)
    raise TypeError("%s: float32 or bfloat16, got %s" % (name, t.dtype))


def router_gate(logits, top_k, score="softmax", bias=None, groups=1, group_top=None,
                group_score="top2", normalize=True, scale=1.0, mask=None):
    """logits [T, E] f32 or bf16 (rows may be strided) -> RouterGate.  score
    "softmax" or "sigmoid"; bias f32 [E], added to the scores for the choice
    alone; the experts in `groups` equal runs, of which the best `group_top` (all
    if None) by their largest choice ("max") or their two largest ("top2") stay;
    weights divided by their sum if `normalize`, times `scale`; mask bool or
    uint8 [T] (0: padding)."""
    dtype, ld = _logits(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    stream = stream_on(dev)
    if bias is not None:
        check(bias, _F32, (E,), dev, "bias")
    if mask is not None:
        check(mask, torch.bool if mask.dtype is torch.bool else torch.uint8, (T,), dev, "mask")
    fits(top_k, "top_k")
    if group_top is None:
        group_top = groups
    fits(groups, "groups")
    fits(group_top, "group_top")
    config = _config(score, index(groups), index(group_top),
                     group_score, bool(normalize), float(scale))
    k = max(top_k, 0)
    ids = torch.empty(T, k, dtype=_I32, device=dev)
    weights = torch.empty(T, k, dtype=_F32, device=dev)
    counts = torch.empty(E, dtype=_I32, device=dev)
    code = lib().moe_gate_forward(
        logits.data_ptr(), dtype, ld, None if bias is None else bias.data_ptr(),
        None if mask is None else mask.data_ptr(), T, E, top_k, config, ids.data_ptr(),
        weights.data_ptr(), counts.data_ptr(), stream)
    if code:
        raise MoEError(code, "moe_gate_forward")
    return RouterGate(ids, weights, counts, top_k, config)


def router_gate_backward(logits, fwd, d_weights, out=None):
    """Gradient of `logits` (same type) from d_weights f32 [T, K].  `fwd` is
    router_gate's result for the same logits."""
    dtype, ld = _logits(logits, "logits")
    T, E = shape = logits.shape
    dev = logits.device
    stream = stream_on(dev)
    K = fwd.top_k
    if fwd.ids.shape != (T, K) or fwd.counts.shape != (E,) or fwd.ids.device != dev:
        raise ValueError("fwd: router_gate's result for logits of this shape")
    check(d_weights, _F32, (T, K), dev, "d_weights")
    if out is None:
        out, ld_d = torch.empty(shape, dtype=logits.dtype, device=dev), E
    else:
        out_dtype, ld_d = _logits(out, "out")
        if out_dtype != dtype or out.shape != shape or out.device != dev:
            raise ValueError("out: the logits' type and shape")
    code = lib().moe_gate_backward(
        logits.data_ptr(), dtype, ld, T, E, K, fwd.config, fwd.ids.data_ptr(),
        d_weights.data_ptr(), out.data_ptr(), ld_d, stream)
    if code:
        raise MoEError(code, "moe_gate_backward")
    return out


def router_order(ids, num_experts):
    """The slots of int32 ids (of any shape, as router_gate and router_balance
    give them) in expert order -> RouterOrder, whose slots and offsets
    blockscale_experts and int8_experts take."""
    n, dev = ids.numel(), ids.device
    stream = stream_on(dev)
    fits(n, "ids")
    fits(num_experts, "num_experts")
    if ids.dtype is not _I32 or not ids.is_contiguous():
        raise ValueError("ids: contiguous int32")
    L = lib()
    nbytes = L.moe_order_workspace(n, num_experts)
    slots, rows = torch.empty(n, dtype=_I32, device=dev), torch.empty(n, dtype=_I32, device=dev)
    offsets = torch.empty(max(num_experts, 0) + 1, dtype=_I32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    code = L.moe_order(ids.data_ptr(), n, num_experts, slots.data_ptr(), offsets.data_ptr(),
                       rows.data_ptr(), ws.data_ptr() if nbytes else None, nbytes, stream)
    if code:
        raise MoEError(code, "moe_order")
    return RouterOrder(slots, offsets, rows)
