"""The router in training, on torch tensors: top-k routing with the
load-balance loss, and the gradient of the logits.

Thin wrappers of ``moe_balance_forward`` and ``moe_balance_backward``
(``include/moe.h`` states the formulas); work goes on torch's current stream.
"""


class RouterBalance:
    """What the forward computed: ids int32 [T, K] and weights f32 [T, K] (-1
    and 0 for tokens that are not live), counts int32 [E], mean_probs f32 [E],
    loss f32 (a scalar tensor), and the K and coef it was computed for."""
    __slots__ = ("ids", "weights", "counts", "mean_probs", "loss", "top_k", "coef")

    def __init__(self, ids, weights, counts, mean_probs, loss, top_k, coef):
        self.ids, self.weights, self.counts = ids, weights, counts
        self.mean_probs, self.loss, self.top_k, self.coef = mean_probs, loss, top_k, coef


def _dtype(torch, t, name):
    if t.dtype == torch.float32:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    raise TypeError("%s: float32 or bfloat16, got %s" % (name, t.dtype))


def _logits(torch, logits, name="logits"):
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("%s: a CUDA tensor [T, E] with contiguous rows" % name)
    return _dtype(torch, logits, name), logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]


def _side(t, shape, dtype, device, name):
    if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or t.device != device
                          or not t.is_contiguous()):
        raise ValueError("%s: a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, shape, device))
    return t


def router_balance(logits, top_k, coef=1.0, mask=None):
    """logits [T, E] f32 or bf16 (rows may be strided), mask bool or uint8 [T]
    (0: padding) or None -> RouterBalance."""
    import torch

    from . import lib, moe_balance_forward
    dtype, ld = _logits(torch, logits)
    T, E = logits.shape
    dev = logits.device
    if mask is not None:
        _side(mask, (T,), torch.bool if mask.dtype == torch.bool else torch.uint8, dev, "mask")
    ids = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    weights = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    mean_probs = torch.empty(E, dtype=torch.float32, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    nbytes = lib().moe_balance_workspace(T, E)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    moe_balance_forward(logits, dtype, ld, mask, T, E, top_k, coef, ids, weights, counts,
                        mean_probs, loss, ws, nbytes,
                        torch.cuda.current_stream(dev).cuda_stream)
    return RouterBalance(ids, weights, counts, mean_probs, loss, top_k, coef)


def router_balance_backward(logits, fwd, d_loss=None, d_weights=None, out=None):
    """Gradient of `logits` (same type) from d_loss (f32 scalar tensor) and
    d_weights (f32 [T, K]); either may be None.  `fwd` is router_balance's
    result for the same logits."""
    import torch

    from . import moe_balance_backward
    dtype, ld = _logits(torch, logits)
    T, E = logits.shape
    dev = logits.device
    if tuple(fwd.ids.shape) != (T, fwd.top_k) or tuple(fwd.counts.shape) != (E,):
        raise ValueError("fwd: router_balance's result for logits of this shape")
    if d_loss is not None and (d_loss.numel() != 1 or d_loss.dtype != torch.float32
                               or d_loss.device != dev):
        raise ValueError("d_loss: one float32 on %s" % dev)
    _side(d_weights, (T, fwd.top_k), torch.float32, dev, "d_weights")
    if out is None:
        out = torch.empty(T, E, dtype=logits.dtype, device=dev)
    out_dtype, ld_d = _logits(torch, out, "out")
    if out_dtype != dtype or out.shape != logits.shape:
        raise ValueError("out: the logits' type and shape")
    moe_balance_backward(logits, dtype, ld, T, E, fwd.top_k, fwd.coef, fwd.ids, fwd.weights,
                         fwd.counts, d_loss, d_weights, out, ld_d,
                         torch.cuda.current_stream(dev).cuda_stream)
    return out
