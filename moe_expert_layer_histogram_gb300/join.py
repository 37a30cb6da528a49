"""The end of a block on torch tensors: the experts' rows added up by their
routing weights, a shared expert behind its gate, a norm after the block, the
scaled sum with the residual, the norm before the next block; and all of its
gradients.

Thin wrappers of ``moe_join_forward`` and ``moe_join_backward``
(``include/moe.h`` states the formulas); work goes on torch's current stream.
"""
import struct

import torch

from . import MoEError, MoEJoin, lib
from ._tensors import check, row_stride, stream_on
from .gate import RouterOrder

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_TYPE = {_F32: 0, _BF16: 1}


class BlockJoin:
    """What the join gave: x [T, H] (x's type; x itself where nothing was
    joined), h bf16 [T, H] or None, or in 8 bits codes int8 [T, H] and code_scales
    f32 [T]; and what its backward pass takes."""
    __slots__ = ("x", "h", "codes", "code_scales", "_join", "_ld_x", "_stats", "_live", "_inputs")

    def __init__(self, x, h, codes, code_scales, join, ld_x, stats, live, inputs):
        self.x, self.h, self.codes, self.code_scales = x, h, codes, code_scales
        self._join, self._ld_x, self._stats = join, ld_x, stats
        self._live, self._inputs = live, inputs


class JoinGradients:
    """Gradients of block_join's arguments, under their names; None for those
    that it did not have, and for norm_weight without d_h."""
    __slots__ = ("x", "expert_rows", "weights", "shared", "gate", "post_weight", "norm_weight")

    def __init__(self, x, expert_rows, weights, shared, gate, post_weight, norm_weight):
        self.x, self.expert_rows, self.weights = x, expert_rows, weights
        self.shared, self.gate = shared, gate
        self.post_weight, self.norm_weight = post_weight, norm_weight


# moe_join's members, in order
_pack = struct.Struct("6i2fQqQqi4xQQQqQQQ").pack
_empty = torch.empty


def _type(t, name):
    if t.dtype not in _TYPE:
        raise TypeError("%s: float32 or bfloat16, got %s" % (name, t.dtype))
    return _TYPE[t.dtype]


def _rows(t, dtype, shape, device, name):
    """Row stride of a [T, H] argument."""
    ld = row_stride(t, dtype, name)
    if t.shape != shape or t.device != device:
        raise ValueError("%s: %s on %s" % (name, tuple(shape), device))
    return ld


def _vector(t, dtype, n, device, name):
    """Address of a contiguous vector of n elements."""
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError("%s: contiguous %s [%d] on %s" % (name, dtype, n, device))
    return t.data_ptr()


def block_join(x, expert_rows=None, order=None, weights=None, shared=None, gate=None,
               post_weight=None, scale=1.0, norm_weight=None, eps=1e-6, quantize=False, out=None):
    """x [T, H] f32 or bf16; expert_rows bf16 [R, H] with order (router_order's
    RouterOrder, or int32 rows [T * K]: the row of each slot, anything outside
    [0, R) for none) and weights f32 [T, K]; shared bf16 [T, H] with gate [T]
    (logits, f32 or bf16) or without; post_weight and norm_weight [H], both f32 or
    both bf16 -> BlockJoin.  h comes in 8 bits if `quantize`; out: where the new x
    goes (x itself, say)."""
    x_type = _type(x, "x")
    dtype = x.dtype
    ld_x = row_stride(x, dtype, "x")
    T, H = shape = x.shape
    dev = x.device
    stream = stream_on(dev)
    K = ld_rows = rows = rows_ptr = slots_ptr = weights_ptr = 0
    row_of_slot = live = None
    if expert_rows is not None:
        if order is None or weights is None or weights.dim() != 2 or not weights.shape[1]:
            raise ValueError("expert_rows: wanted with order and weights [T, K], K >= 1")
        K = weights.shape[1]
        row_of_slot = order
        if isinstance(order, RouterOrder):
            row_of_slot, live = order.rows, order.offsets
        check(weights, _F32, (T, K), dev, "weights")
        if (row_of_slot.dtype is not _I32 or row_of_slot.numel() != T * K
                or row_of_slot.device != dev or not row_of_slot.is_contiguous()):
            raise ValueError("order: int32 rows of %d slots on %s" % (T * K, dev))
        ld_rows = row_stride(expert_rows, _BF16, "expert_rows")
        rows, width = expert_rows.shape
        if width != H or expert_rows.device != dev:
            raise ValueError("expert_rows: [R, %d] on %s" % (H, dev))
        if live is not None and (live.dtype is not _I32 or live.dim() != 1 or live.device != dev
                                 or not live.numel() or not live.is_contiguous()):
            raise ValueError("order: contiguous int32 offsets on %s" % dev)
        rows_ptr, slots_ptr = expert_rows.data_ptr(), row_of_slot.data_ptr()
        weights_ptr = weights.data_ptr()
    elif order is not None or weights is not None:
        raise ValueError("order and weights: wanted with expert_rows")
    ld_shared = shared_ptr = gate_ptr = gate_type = 0
    if shared is not None:
        ld_shared = _rows(shared, _BF16, shape, dev, "shared")
        shared_ptr = shared.data_ptr()
    if gate is not None:
        gate_type = _type(gate, "gate")
        if shared is None:
            raise ValueError("gate: wanted with shared")
        gate_ptr = _vector(gate, gate.dtype, T, dev, "gate")
    post_ptr = norm_ptr = weight_type = 0
    if post_weight is not None:
        weight_type = _type(post_weight, "post_weight")
        post_ptr = _vector(post_weight, post_weight.dtype, H, dev, "post_weight")
    if norm_weight is not None:
        weight_type = _type(norm_weight, "norm_weight")
        norm_ptr = _vector(norm_weight, norm_weight.dtype if post_weight is None
                           else post_weight.dtype, H, dev, "norm_weight")
    elif quantize:
        raise ValueError("quantize: wanted with norm_weight")
    joined = K > 0 or shared is not None
    if not joined and norm_weight is None:
        raise ValueError("nothing to join and no norm_weight")
    ld_out, x_out, out_ptr = H, x, None
    if not joined:
        if out is not None:
            raise ValueError("out: there is nothing to join")
    elif out is None:
        x_out = _empty(shape, dtype=dtype, device=dev)
        out_ptr = x_out.data_ptr()
    else:
        ld_out, x_out = _rows(out, dtype, shape, dev, "out"), out
        out_ptr = out.data_ptr()
    # (the norms' statistics and the codes' scales: a row each)
    stats = _empty((3, T), dtype=_F32, device=dev)
    base = stats.data_ptr()
    h = codes = code_scales = h_ptr = codes_ptr = scales_ptr = None
    ld_codes = (H + 15) // 16 * 16
    if norm_ptr and quantize:
        codes = _empty((T, ld_codes), dtype=torch.int8, device=dev)
        codes_ptr, scales_ptr, code_scales = codes.data_ptr(), base + 8 * T, stats[2]
    elif norm_weight is not None:
        h = _empty(shape, dtype=_BF16, device=dev)
        h_ptr = h.data_ptr()
    join = MoEJoin.from_buffer_copy(_pack(
        T, H, K, x_type, weight_type, gate_type, scale, eps, x.data_ptr(), ld_x, rows_ptr, ld_rows,
        rows, slots_ptr, weights_ptr, shared_ptr, ld_shared, gate_ptr, post_ptr, norm_ptr))
    code = lib().moe_join_forward(join, out_ptr, ld_out, h_ptr, H, codes_ptr, ld_codes, scales_ptr,
                                  base + 4 * T, base, stream)
    if code:
        raise MoEError(code, "moe_join_forward")
    if codes is not None and ld_codes != H:
        codes = codes[:, :H]
    return BlockJoin(x_out, h, codes, code_scales, join, ld_out if joined else ld_x, stats, live,
                     (expert_rows, row_of_slot, weights, shared, gate, post_weight, norm_weight))


def block_join_backward(fwd, d_x=None, d_h=None):
    """Gradients of block_join's arguments -> JoinGradients, from d_x (the new
    x's, of its type) and d_h bf16 [T, H]; either may be None.  `fwd` is
    block_join's result, whose x, and the arguments it was given, are as they
    were.  The gradient of expert_rows is zero for rows of no expert, where fwd
    was given a RouterOrder; with plain rows it has whatever was in memory in
    rows that no slot names, and a row may be named by one slot at most (the
    gradients of several are not added up)."""
    x = fwd.x
    expert_rows, _, weights, shared, gate, post_weight, norm_weight = fwd._inputs
    live = fwd._live
    T, H = shape = x.shape
    dev = x.device
    stream = stream_on(dev)
    ld_dxo = ld_dh = H
    dx_ptr = dh_ptr = rows_ptr = live_ptr = weights_ptr = shared_ptr = gate_ptr = None
    post_ptr = norm_ptr = None
    if d_x is not None:
        ld_dxo = _rows(d_x, x.dtype, shape, dev, "d_x")
        dx_ptr = d_x.data_ptr()
    if d_h is not None:
        if norm_weight is None:
            raise ValueError("d_h: the join had no norm_weight")
        ld_dh = _rows(d_h, _BF16, shape, dev, "d_h")
        dh_ptr = d_h.data_ptr()
    out_x = _empty(shape, dtype=x.dtype, device=dev)
    d_rows = d_weights = d_shared = d_gate = d_post = d_norm = None
    if expert_rows is not None:
        d_rows = _empty((expert_rows.shape[0], H), dtype=_BF16, device=dev)
        d_weights = torch.empty_like(weights)
        rows_ptr, weights_ptr = d_rows.data_ptr(), d_weights.data_ptr()
        if live is not None:
            live_ptr = live.data_ptr() + 4 * (live.numel() - 1)
    if shared is not None:
        d_shared = _empty(shape, dtype=_BF16, device=dev)
        shared_ptr = d_shared.data_ptr()
    if gate is not None:
        d_gate = torch.empty_like(gate)
        gate_ptr = d_gate.data_ptr()
    if post_weight is not None:
        d_post = torch.empty_like(post_weight)
        post_ptr = d_post.data_ptr()
    if d_h is not None:
        d_norm = torch.empty_like(norm_weight)
        norm_ptr = d_norm.data_ptr()
    L = lib()
    nbytes, ws_ptr = 0, None
    if post_ptr or norm_ptr:
        nbytes = L.moe_join_workspace(T, H)
        ws = _empty(nbytes, dtype=torch.uint8, device=dev)
        ws_ptr = ws.data_ptr()
    base = fwd._stats.data_ptr()
    code = L.moe_join_backward(
        fwd._join, x.data_ptr(), fwd._ld_x, base + 4 * T, base, dx_ptr, ld_dxo, dh_ptr, ld_dh,
        out_x.data_ptr(), H, rows_ptr, H, live_ptr, weights_ptr, shared_ptr, H, gate_ptr, post_ptr,
        norm_ptr, ws_ptr, nbytes, stream)
    if code:
        raise MoEError(code, "moe_join_backward")
    return JoinGradients(out_x, d_rows, d_weights, d_shared, d_gate, d_post, d_norm)
