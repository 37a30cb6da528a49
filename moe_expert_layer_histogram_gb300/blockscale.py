"""FP8 products with one fp32 scale per block of 128, on torch tensors.

Weights are float8_e4m3fn codes [N, K] (or [E, N, K]) with fp32 scales
[ceil(N/128), ceil(K/128)] ([E, ...]); activations come in bf16 and are
quantised per row and 128 columns on the way in.  Thin wrappers of the
``moe_blockscale_*`` calls (``include/moe.h`` states the formulas); work goes
on torch's current stream, and the quantised activations live in torch's
allocator for the length of the call.
"""
import torch

from . import MoEError, lib
from ._tensors import check, fits, row_stride, stream_on

_F32, _BF16, _E4M3, _I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32


def _weights(w, w_scales):
    """(E, N, K, row stride) of [N, K] or [E, N, K] weights; checks the scales."""
    if w.dtype is not _E4M3 or not w.is_cuda:
        raise ValueError("w: CUDA float8_e4m3fn codes")
    shape, strides = w.shape, w.stride()
    if len(shape) == 2:
        E, (N, K), (ldw, one) = 1, shape, strides
        blocks = ((N + 127) // 128, (K + 127) // 128)
    elif len(shape) == 3:
        (E, N, K), (ld_e, ldw, one) = shape, strides
        blocks = (E, (N + 127) // 128, (K + 127) // 128)
        if E > 1:
            if N == 1:  # (the stride of a single row says nothing)
                ldw = ld_e
            if ld_e != N * ldw or ldw < K:
                raise ValueError("w: experts at a stride of N rows of at least K codes")
    else:
        raise ValueError("w: [N, K] or [E, N, K]")
    if one != 1 and K > 1:
        raise ValueError("w: contiguous rows")
    fits(max(E, N, K), "w")
    if N == 1 and ldw < K:  # (one expert)
        ldw = K
    check(w_scales, _F32, blocks, w.device, "w_scales")
    return E, N, K, ldw


def _result(out, M, N, device):
    """(bf16 [M, N], its row stride): the caller's or a new one."""
    if out is None:
        return torch.empty(M, N, dtype=_BF16, device=device), N
    ldo = row_stride(out, _BF16, "out")
    if out.shape != (M, N) or out.device != device:
        raise ValueError("out: [%d, %d] on %s" % (M, N, device))
    return out, ldo


def blockscale_quantize(x, slots=None, top_k=1):
    """bf16 rows -> (codes float8_e4m3fn [R, C], scales f32 [ceil(C/128), R]).
    With int32 `slots` [R], row r is x's row slots[r] // top_k (zero where that
    is outside x).  The codes' rows are 16-byte aligned."""
    ldx = row_stride(x, _BF16, "x")
    (T, C), dev = x.shape, x.device
    stream = stream_on(dev)
    R = T
    fits(top_k, "top_k")
    if slots is not None:
        R = slots.numel()
        check(slots, _I32, (R,), dev, "slots")
    ld = (C + 15) // 16 * 16
    codes = torch.empty(R, ld, dtype=_E4M3, device=dev)
    scales = torch.empty((C + 127) // 128, R, dtype=_F32, device=dev)
    code = lib().moe_blockscale_quantize(
        x.data_ptr(), ldx, T, None if slots is None else slots.data_ptr(), top_k, R, C,
        codes.data_ptr(), ld, scales.data_ptr(), R, stream)
    if code:
        raise MoEError(code, "moe_blockscale_quantize")
    return (codes if ld == C else codes[:, :C]), scales


def blockscale_matmul(codes, scales, w, w_scales, offsets=None, transpose_w=False, out=None):
    """Quantised rows [M, K] (from blockscale_quantize) times w^T -> bf16
    [M, N]; transpose_w: w is [K, N] (the input gradient of a product with
    w).  offsets int32 [E+1]: the rows of each expert of w [E, ...]; rows of
    no expert are left as they are."""
    lda = row_stride(codes, _E4M3, "codes")
    E, wr, wc, ldw = _weights(w, w_scales)
    N, K = (wc, wr) if transpose_w else (wr, wc)
    M, dev = codes.shape[0], w.device
    stream = stream_on(dev)
    if codes.shape[1] != K or codes.device != dev:
        raise ValueError("codes: [M, %d] on %s" % (K, dev))
    ld_as = row_stride(scales, _F32, "scales")
    if scales.shape != ((K + 127) // 128, M) or scales.device != dev:
        raise ValueError("scales: [%d, %d] on %s" % ((K + 127) // 128, M, dev))
    if offsets is not None:
        check(offsets, _I32, (E + 1,), dev, "offsets")
    elif E != 1:
        raise ValueError("offsets: wanted for weights of several experts")
    out, ldo = _result(out, M, N, dev)
    code = lib().moe_blockscale_matmul(
        codes.data_ptr(), lda, scales.data_ptr(), ld_as, w.data_ptr(), ldw, w_scales.data_ptr(),
        None if offsets is None else offsets.data_ptr(), E, M, N, K, 1 if transpose_w else 0,
        out.data_ptr(), ldo, stream)
    if code:
        raise MoEError(code, "moe_blockscale_matmul")
    return out


def _linear(x, w, w_scales, transpose_w, out):
    ldx = row_stride(x, _BF16, "x")
    if w.dim() != 2:
        raise ValueError("w: one weight matrix")
    _, wr, wc, ldw = _weights(w, w_scales)
    N, K = (wc, wr) if transpose_w else (wr, wc)
    M, dev = x.shape[0], w.device
    stream = stream_on(dev)
    if x.shape[1] != K or x.device != dev:
        raise ValueError("x: [M, %d] on %s" % (K, dev))
    out, ldo = _result(out, M, N, dev)
    L = lib()
    nbytes = L.moe_blockscale_linear_workspace(M, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    code = L.moe_blockscale_linear(x.data_ptr(), ldx, w.data_ptr(), ldw, w_scales.data_ptr(), M, N,
                                   K, transpose_w, out.data_ptr(), ldo,
                                   ws.data_ptr() if nbytes else None, nbytes, stream)
    if code:
        raise MoEError(code, "moe_blockscale_linear")
    return out


def blockscale_linear(x, w, w_scales, out=None):
    """y = x w^T for bf16 x [M, K] and weights [N, K] -> bf16 [M, N]."""
    return _linear(x, w, w_scales, 0, out)


def blockscale_linear_dx(dy, w, w_scales, out=None):
    """Input gradient of blockscale_linear: dx = dy w for bf16 dy [M, N], from
    the same stored weights [N, K] -> bf16 [M, K]."""
    return _linear(dy, w, w_scales, 1, out)


def blockscale_experts(x, slots, offsets, top_k, w13, w13_scales, w2, w2_scales, clamp=0.0,
                       out=None):
    """The experts' products on routed rows: row r of the result is expert
    e's MLP of x's row slots[r] // top_k, for offsets[e] <= r < offsets[e+1]
    (slots and offsets as router_order gives them, or as moe_route_permute_static
    writes perm and offsets).
    w13 [E, 2I, H] (gate rows, then up rows), w2 [E, H, I], contiguous -> bf16
    [len(slots), H], in permuted row order; rows of no expert are left as
    they are."""
    ldx = row_stride(x, _BF16, "x")
    E, I2, H, _ = _weights(w13, w13_scales)
    I = I2 // 2
    _weights(w2, w2_scales)
    if (w13.dim() != 3 or w2.shape != (E, H, I) or I2 % 256 or not w13.is_contiguous()
            or not w2.is_contiguous()):
        raise ValueError("contiguous w13 [E, 2I, H] and w2 [E, H, I] with I a multiple of 128")
    T, dev = x.shape[0], w13.device
    stream = stream_on(dev)
    if x.shape[1] != H or x.device != dev or w2.device != dev:
        raise ValueError("x: [T, %d], all on %s" % (H, dev))
    R = slots.numel()
    fits(top_k, "top_k")
    check(slots, _I32, (R,), dev, "slots")
    check(offsets, _I32, (E + 1,), dev, "offsets")
    out, ldo = _result(out, R, H, dev)
    L = lib()
    nbytes = L.moe_blockscale_experts_workspace(R, H, I)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    code = L.moe_blockscale_experts(
        x.data_ptr(), ldx, T, slots.data_ptr(), top_k, R, offsets.data_ptr(), E, w13.data_ptr(),
        w13_scales.data_ptr(), w2.data_ptr(), w2_scales.data_ptr(), H, I, clamp, out.data_ptr(),
        ldo, ws.data_ptr(), nbytes, stream)
    if code:
        raise MoEError(code, "moe_blockscale_experts")
    return out
