"""The end of a block on torch tensors: the experts' rows added up by their
routing weights, a shared expert behind its gate, a norm after the block, the
scaled sum with the residual, the norm before the next block; and all of its
gradients.

Thin wrappers of ``moe_join_forward`` and ``moe_join_backward``
(``include/moe.h`` states the formulas); work goes on torch's current stream.
"""
import torch

from . import MoEError, MoEJoin, lib
from ._tensors import check, row_stride, stream_on

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_TYPE = {_F32: 0, _BF16: 1}


class BlockJoin:
    """What the join gave: x [T, H] (x's type; x itself where nothing was
    joined), h bf16 [T, H] or None, or in 8 bits codes int8 [T, H] and code_scales
    f32 [T]; and what its backward pass takes."""
    __slots__ = ("x", "h", "codes", "code_scales", "_join", "_inputs", "_post_rstd", "_norm_rstd")

    def __init__(self, x, h, codes, code_scales, join, inputs, post_rstd, norm_rstd):
        self.x, self.h, self.codes, self.code_scales = x, h, codes, code_scales
        self._join, self._inputs = join, inputs
        self._post_rstd, self._norm_rstd = post_rstd, norm_rstd


class JoinGradients:
    """Gradients of block_join's arguments, under their names; None for those
    that it did not have."""
    __slots__ = ("x", "expert_rows", "weights", "shared", "gate", "post_weight", "norm_weight")

    def __init__(self, x, expert_rows, weights, shared, gate, post_weight, norm_weight):
        self.x, self.expert_rows, self.weights = x, expert_rows, weights
        self.shared, self.gate = shared, gate
        self.post_weight, self.norm_weight = post_weight, norm_weight


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


def _ptr(t):
    return None if t is None else t.data_ptr()


def block_join(x, expert_rows=None, order=None, weights=None, shared=None, gate=None,
               post_weight=None, scale=1.0, norm_weight=None, eps=1e-6, quantize=False, out=None):
    """x [T, H] f32 or bf16; expert_rows bf16 [R, H] with order (router_order's
    RouterOrder, or int32 rows [T * K]: the row of each slot, anything outside
    [0, R) for none) and weights f32 [T, K]; shared bf16 [T, H] with gate [T]
    (logits, f32 or bf16) or without; post_weight and norm_weight [H], f32 or
    bf16 -> BlockJoin.  h comes in 8 bits if `quantize`; out: where the new x
    goes (x itself, say)."""
    x_type = _type(x, "x")
    ld_x = row_stride(x, x.dtype, "x")
    T, H = shape = x.shape
    dev = x.device
    stream = stream_on(dev)
    join = MoEJoin(T=T, H=H, x_type=x_type, scale=scale, eps=eps, x=x.data_ptr(), ld_x=ld_x)
    row_of_slot = live = None
    if expert_rows is not None:
        if order is None or weights is None or weights.dim() != 2:
            raise ValueError("expert_rows: wanted with order and weights [T, K]")
        K = join.K = weights.shape[1]
        row_of_slot = getattr(order, "rows", order)
        if row_of_slot is not order:
            live = order.offsets[-1:]
        check(weights, _F32, (T, K), dev, "weights")
        if (row_of_slot.dtype is not _I32 or row_of_slot.numel() != T * K
                or row_of_slot.device != dev or not row_of_slot.is_contiguous()):
            raise ValueError("order: int32 rows of %d slots on %s" % (T * K, dev))
        join.ld_rows = row_stride(expert_rows, _BF16, "expert_rows")
        join.rows = expert_rows.shape[0]
        if expert_rows.shape[1] != H or expert_rows.device != dev:
            raise ValueError("expert_rows: [R, %d] on %s" % (H, dev))
        join.expert_rows, join.row_of_slot = expert_rows.data_ptr(), row_of_slot.data_ptr()
        join.weights = weights.data_ptr()
    elif order is not None or weights is not None:
        raise ValueError("order and weights: wanted with expert_rows")
    if shared is not None:
        join.ld_shared = _rows(shared, _BF16, shape, dev, "shared")
        join.shared = shared.data_ptr()
    if gate is not None:
        join.gate_type = _type(gate, "gate")
        check(gate, gate.dtype, (T,), dev, "gate")
        if shared is None:
            raise ValueError("gate: wanted with shared")
        join.gate = gate.data_ptr()
    norms = [w for w in (post_weight, norm_weight) if w is not None]
    for w, name in ((post_weight, "post_weight"), (norm_weight, "norm_weight")):
        if w is not None:
            join.weight_type = _type(w, name)
            check(w, norms[0].dtype, (H,), dev, name)
    join.post_weight, join.norm_weight = _ptr(post_weight), _ptr(norm_weight)
    joined = join.K > 0 or shared is not None
    if not joined and norm_weight is None:
        raise ValueError("nothing to join and no norm_weight")
    if quantize and norm_weight is None:
        raise ValueError("quantize: wanted with norm_weight")
    ld_out, x_out = H, None
    if joined:
        x_out = torch.empty(T, H, dtype=x.dtype, device=dev) if out is None else out
        if out is not None:
            ld_out = _rows(out, x.dtype, shape, dev, "out")
    elif out is not None:
        raise ValueError("out: there is nothing to join")
    h = codes = code_scales = norm_rstd = post_rstd = None
    ld_codes = (H + 15) // 16 * 16
    # (one allocation for the norms' statistics and the codes' scales)
    stats = torch.empty(3, T, dtype=_F32, device=dev)
    if norm_weight is not None:
        norm_rstd = stats[0]
        if quantize:
            codes = torch.empty(T, ld_codes, dtype=torch.int8, device=dev)
            code_scales = stats[2]
        else:
            h = torch.empty(T, H, dtype=_BF16, device=dev)
    if post_weight is not None:
        post_rstd = stats[1]
    code = lib().moe_join_forward(join, _ptr(x_out), ld_out, _ptr(h), H, _ptr(codes), ld_codes,
                                  _ptr(code_scales), _ptr(post_rstd), _ptr(norm_rstd), stream)
    if code:
        raise MoEError(code, "moe_join_forward")
    if codes is not None and ld_codes != H:
        codes = codes[:, :H]
    if x_out is None:
        x_out, ld_out = x, ld_x
    return BlockJoin(x_out, h, codes, code_scales, join,
                     (ld_out, row_of_slot, live, expert_rows, weights, shared, gate, post_weight,
                      norm_weight), post_rstd, norm_rstd)


def block_join_backward(fwd, d_x=None, d_h=None):
    """Gradients of block_join's arguments -> JoinGradients, from d_x (the new
    x's, of its type) and d_h bf16 [T, H]; either may be None.  `fwd` is
    block_join's result, whose x, and the arguments it was given, are as they
    were.  The gradient of expert_rows is zero for rows of no expert, where fwd
    was given a RouterOrder; with plain rows it has whatever was in memory in
    rows that no slot names."""
    join, x = fwd._join, fwd.x
    (ld_out, row_of_slot, live, expert_rows, weights, shared, gate, post_weight,
     norm_weight) = fwd._inputs
    T, H = shape = x.shape
    dev = x.device
    stream = stream_on(dev)
    ld_dxo = H if d_x is None else _rows(d_x, x.dtype, shape, dev, "d_x")
    ld_dh = H
    if d_h is not None:
        if norm_weight is None:
            raise ValueError("d_h: the join had no norm_weight")
        ld_dh = _rows(d_h, _BF16, shape, dev, "d_h")
    out_x = torch.empty(T, H, dtype=x.dtype, device=dev)
    d_rows = d_weights = d_shared = d_gate = d_post = d_norm = None
    if row_of_slot is not None:
        d_rows = torch.empty(expert_rows.shape[0], H, dtype=_BF16, device=dev)
        d_weights = torch.empty_like(weights)
    if shared is not None:
        d_shared = torch.empty(T, H, dtype=_BF16, device=dev)
    if gate is not None:
        d_gate = torch.empty_like(gate)
    if post_weight is not None:
        d_post = torch.empty_like(post_weight)
    if d_h is not None:
        d_norm = torch.empty_like(norm_weight)
    L = lib()
    nbytes, ws = 0, None
    if d_post is not None or d_norm is not None:
        nbytes = L.moe_join_workspace(T, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    code = L.moe_join_backward(
        join, x.data_ptr(), ld_out, _ptr(fwd._post_rstd), _ptr(fwd._norm_rstd), _ptr(d_x), ld_dxo,
        _ptr(d_h), ld_dh, out_x.data_ptr(), H, _ptr(d_rows), H, _ptr(live), _ptr(d_weights),
        _ptr(d_shared), H, _ptr(d_gate), _ptr(d_post), _ptr(d_norm), _ptr(ws), nbytes, stream)
    if code:
        raise MoEError(code, "moe_join_backward")
    return JoinGradients(out_x, d_rows, d_weights, d_shared, d_gate, d_post, d_norm)
