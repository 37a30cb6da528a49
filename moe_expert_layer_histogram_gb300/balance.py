"""The router in training, on torch tensors: top-k routing with the
load-balance loss, and the gradient of the logits.

Thin wrappers of ``moe_balance_forward`` and ``moe_balance_backward``
(``include/moe.h`` states the formulas); work goes on torch's current stream.
"""
import torch

from . import MoEError, lib
from ._tensors import check, fits, row_stride, stream_on

_F32, _BF16 = torch.float32, torch.bfloat16


class RouterBalance:
    """What the forward computed: ids int32 [T, K] and weights f32 [T, K] (-1
    and 0 for tokens that are not live), counts int32 [E], mean_probs f32 [E],
    loss f32 (a scalar tensor), and the K and coef it was computed for."""
    __slots__ = ("ids", "weights", "counts", "loss", "top_k", "coef", "_stats")

    def __init__(self, ids, weights, counts, stats, top_k, coef):
        self.ids, self.weights, self.counts = ids, weights, counts
        self.loss, self.top_k, self.coef, self._stats = stats[0], top_k, coef, stats

    @property
    def mean_probs(self):
        return self._stats[4:4 + self.counts.numel()]


def _logits(t, name):
    """(element type code, row stride) of logits or their gradient."""
    if t.dtype is _F32:
        return 0, row_stride(t, _F32, name)
    if t.dtype is _BF16:
        return 1, row_stride(t, _BF16, name)
    raise TypeError("%s: float32 or bfloat16, got %s" % (name, t.dtype))


def router_balance(logits, top_k, coef=1.0, mask=None):
    """logits [T, E] f32 or bf16 (rows may be strided), mask bool or uint8 [T]
    (0: padding) or None -> RouterBalance."""
    dtype, ld = _logits(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    stream = stream_on(dev)
    if mask is not None:
        check(mask, torch.bool if mask.dtype is torch.bool else torch.uint8, (T,), dev, "mask")
    L = lib()
    nbytes = L.moe_balance_workspace(T, E)
    fits(top_k, "top_k")
    k = max(top_k, 0)
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    weights = torch.empty(T, k, dtype=_F32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    # loss and mean_probs (from word 4); a small workspace behind them (16-byte
    # aligned), a large one apart, so that a loss that is kept keeps none of it
    words = 4 + (E + 3) // 4 * 4
    large = nbytes > 16
    stats = torch.empty(words if large else words + 4, dtype=_F32, device=dev)
    base = stats.data_ptr()
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev) if large else None
    code = L.moe_balance_forward(
        logits.data_ptr(), dtype, ld, None if mask is None else mask.data_ptr(), T, E, top_k, coef,
        ids.data_ptr(), weights.data_ptr(), counts.data_ptr(), base + 16, base,
        work.data_ptr() if large else base + 4 * words, nbytes, stream)
    if code:
        raise MoEError(code, "moe_balance_forward")
    return RouterBalance(ids, weights, counts, stats, top_k, coef)


def router_balance_backward(logits, fwd, d_loss=None, d_weights=None, out=None):
    """Gradient of `logits` (same type) from d_loss (f32 scalar tensor) and
    d_weights (f32 [T, K]); either may be None.  `fwd` is router_balance's
    result for the same logits."""
    dtype, ld = _logits(logits, "logits")
    T, E = shape = logits.shape
    dev = logits.device
    stream = stream_on(dev)
    K = fwd.top_k
    if fwd.ids.shape != (T, K) or fwd.counts.shape != (E,) or fwd.ids.device != dev:
        raise ValueError("fwd: router_balance's result for logits of this shape")
    if d_loss is not None and (d_loss.numel() != 1 or d_loss.dtype is not _F32
                               or d_loss.device != dev):
        raise ValueError("d_loss: one float32 on %s" % dev)
    if d_weights is not None:
        check(d_weights, _F32, (T, K), dev, "d_weights")
    if out is None:
        out, ld_d = torch.empty(shape, dtype=logits.dtype, device=dev), E
    else:
        out_dtype, ld_d = _logits(out, "out")
        if out_dtype != dtype or out.shape != shape or out.device != dev:
            raise ValueError("out: the logits' type and shape")
    code = lib().moe_balance_backward(
        logits.data_ptr(), dtype, ld, T, E, K, fwd.coef, fwd.ids.data_ptr(),
        fwd.weights.data_ptr(), fwd.counts.data_ptr(),
        None if d_loss is None else d_loss.data_ptr(),
        None if d_weights is None else d_weights.data_ptr(), out.data_ptr(), ld_d, stream)
    if code:
        raise MoEError(code, "moe_balance_backward")
    return out
