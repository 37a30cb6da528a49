"""FP8 products with one fp32 scale per block of 128, on torch tensors.

Weights are float8_e4m3fn codes [N, K] (or [E, N, K]) with fp32 scales
[ceil(N/128), ceil(K/128)] ([E, ...]); activations come in bf16 and are
quantised per row and 128 columns on the way in.  Thin wrappers of the
``moe_blockscale_*`` calls (``include/moe.h`` states the formulas); work goes
on torch's current stream, and the quantised activations live in torch's
allocator for the length of the call.
"""


def _ceil(n, m):
    return (n + m - 1) // m


def _rows(t, dtype, name):
    """Row stride of a CUDA matrix with contiguous rows."""
    if t.dim() != 2 or t.dtype != dtype or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s: a CUDA %s matrix with contiguous rows" % (name, dtype))
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _weights(torch, w, w_scales):
    """(E, N, K, row stride) of [N, K] or [E, N, K] weights; checks the scales."""
    if (w.dim() not in (2, 3) or w.dtype != torch.float8_e4m3fn or not w.is_cuda
            or (w.shape[-1] > 1 and w.stride(-1) != 1)):
        raise ValueError("w: CUDA float8_e4m3fn codes [N, K] or [E, N, K] with contiguous rows")
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    ldw = w.stride(-2) if N > 1 else max(w.stride(-2), K)
    if E > 1 and w.stride(0) != N * ldw:
        raise ValueError("w: experts at a stride of N rows")
    shape = ((E,) if w.dim() == 3 else ()) + (_ceil(N, 128), _ceil(K, 128))
    if (tuple(w_scales.shape) != shape or w_scales.dtype != torch.float32
            or w_scales.device != w.device or not w_scales.is_contiguous()):
        raise ValueError("w_scales: contiguous float32 %s on %s" % (shape, w.device))
    return E, N, K, ldw


def _offsets(torch, offsets, E, device):
    if offsets is None:
        if E != 1:
            raise ValueError("offsets: wanted for weights of several experts")
        return None
    if (tuple(offsets.shape) != (E + 1,) or offsets.dtype != torch.int32
            or offsets.device != device or not offsets.is_contiguous()):
        raise ValueError("offsets: contiguous int32 [%d] on %s" % (E + 1, device))
    return offsets


def blockscale_quantize(x, slots=None, top_k=1):
    """bf16 rows -> (codes float8_e4m3fn [R, C], scales f32 [ceil(C/128), R]).
    With int32 `slots` [R], row r is x's row slots[r] // top_k (zero where that
    is outside x).  The codes' rows are 16-byte aligned."""
    import torch

    from . import moe_blockscale_quantize
    ldx = _rows(x, torch.bfloat16, "x")
    C = x.shape[1]
    if slots is not None and (slots.dim() != 1 or slots.dtype != torch.int32
                              or slots.device != x.device or not slots.is_contiguous()):
        raise ValueError("slots: contiguous int32 [R] on %s" % x.device)
    R = x.shape[0] if slots is None else slots.shape[0]
    ld = _ceil(C, 16) * 16
    codes = torch.empty(R, ld, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(_ceil(C, 128), R, dtype=torch.float32, device=x.device)
    moe_blockscale_quantize(x, ldx, x.shape[0], slots, top_k, R, C, codes, ld, scales, R,
                            torch.cuda.current_stream(x.device).cuda_stream)
    return (codes if ld == C else codes[:, :C]), scales


def blockscale_matmul(codes, scales, w, w_scales, offsets=None, transpose_w=False, out=None):
    """Quantised rows [M, K] (from blockscale_quantize) times w^T -> bf16
    [M, N]; transpose_w: w is [K, N] (the input gradient of a product with
    w).  offsets int32 [E+1]: the rows of each expert of w [E, ...]."""
    import torch

    from . import moe_blockscale_matmul
    lda = _rows(codes, torch.float8_e4m3fn, "codes")
    E, wr, wc, ldw = _weights(torch, w, w_scales)
    N, K = (wc, wr) if transpose_w else (wr, wc)
    M = codes.shape[0]
    if codes.shape[1] != K or w.device != codes.device:
        raise ValueError("codes: [M, %d] on %s" % (K, w.device))
    ld_as = _rows(scales, torch.float32, "scales")
    if tuple(scales.shape) != (_ceil(K, 128), M) or scales.device != w.device:
        raise ValueError("scales: [%d, %d] on %s" % (_ceil(K, 128), M, w.device))
    _offsets(torch, offsets, E, w.device)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=w.device)
    ldo = _rows(out, torch.bfloat16, "out")
    if tuple(out.shape) != (M, N) or out.device != w.device:
        raise ValueError("out: [%d, %d] on %s" % (M, N, w.device))
    moe_blockscale_matmul(codes, lda, scales, ld_as, w, ldw, w_scales, offsets, E, M, N, K,
                          int(transpose_w), out, ldo,
                          torch.cuda.current_stream(w.device).cuda_stream)
    return out


def _linear(x, w, w_scales, transpose_w, out):
    import torch

    from . import lib, moe_blockscale_linear
    ldx = _rows(x, torch.bfloat16, "x")
    E, wr, wc, ldw = _weights(torch, w, w_scales)
    N, K = (wc, wr) if transpose_w else (wr, wc)
    M, dev = x.shape[0], w.device
    if w.dim() != 2 or x.shape[1] != K or x.device != dev:
        raise ValueError("x [M, %d] and one weight matrix, both on %s" % (K, dev))
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    ldo = _rows(out, torch.bfloat16, "out")
    if tuple(out.shape) != (M, N) or out.device != dev:
        raise ValueError("out: [%d, %d] on %s" % (M, N, dev))
    nbytes = lib().moe_blockscale_workspace(M, K, 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    moe_blockscale_linear(x, ldx, w, ldw, w_scales, M, N, K, int(transpose_w), out, ldo, ws,
                          nbytes, torch.cuda.current_stream(dev).cuda_stream)
    return out


def blockscale_linear(x, w, w_scales, out=None):
    """y = x w^T for bf16 x [M, K] and weights [N, K] -> bf16 [M, N]."""
    return _linear(x, w, w_scales, False, out)


def blockscale_linear_dx(dy, w, w_scales, out=None):
    """Input gradient of blockscale_linear: dx = dy w for bf16 dy [M, N], from
    the same stored weights [N, K] -> bf16 [M, K]."""
    return _linear(dy, w, w_scales, True, out)


def blockscale_experts(x, slots, offsets, top_k, w13, w13_scales, w2, w2_scales, clamp=0.0,
                       out=None):
    """The experts' products on routed rows: row r of the result is expert
    e's MLP of x's row slots[r] // top_k, for offsets[e] <= r < offsets[e+1]
    (slots and offsets as moe_route_permute_static writes perm and offsets).
    w13 [E, 2I, H] (gate rows, then up rows), w2 [E, H, I], contiguous -> bf16
    [len(slots), H], in permuted row order; rows of no expert are left as
    they are."""
    import torch

    from . import lib, moe_blockscale_experts
    ldx = _rows(x, torch.bfloat16, "x")
    E, I2, H, _ = _weights(torch, w13, w13_scales)
    I = I2 // 2
    _weights(torch, w2, w2_scales)
    if (w13.dim() != 3 or tuple(w2.shape) != (E, H, I) or I2 % 256 or not w13.is_contiguous()
            or not w2.is_contiguous()):
        raise ValueError("contiguous w13 [E, 2I, H] and w2 [E, H, I] with I a multiple of 128")
    dev = w13.device
    if x.shape[1] != H or x.device != dev or w2.device != dev:
        raise ValueError("x: [T, %d], all on %s" % (H, dev))
    if (slots.dim() != 1 or slots.dtype != torch.int32 or slots.device != dev
            or not slots.is_contiguous()):
        raise ValueError("slots: contiguous int32 [R] on %s" % dev)
    if offsets is None:
        raise ValueError("offsets: int32 [%d]" % (E + 1))
    _offsets(torch, offsets, E, dev)
    R = slots.shape[0]
    if out is None:
        out = torch.empty(R, H, dtype=torch.bfloat16, device=dev)
    ldo = _rows(out, torch.bfloat16, "out")
    if tuple(out.shape) != (R, H) or out.device != dev:
        raise ValueError("out: [%d, %d] on %s" % (R, H, dev))
    nbytes = lib().moe_blockscale_workspace(R, H, I)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    moe_blockscale_experts(x, ldx, x.shape[0], slots, top_k, R, offsets, E, w13, w13_scales, w2,
                           w2_scales, H, I, clamp, out, ldo, ws, nbytes,
                           torch.cuda.current_stream(dev).cuda_stream)
    return out
