"""Host checks of the torch wrappers, without a GPU: stand-ins with the
attributes that the wrappers read take the place of CUDA tensors."""
import pytest
import torch

from moe_expert_layer_histogram_gb300 import _tensors, blockscale

CUDA = torch.device("cuda:0")


class Fake:
    """Type, shape and strides of a tensor on cuda:0."""
    is_cuda, device = True, CUDA

    def __init__(self, dtype, shape, strides=None):
        if strides is None:
            strides, step = [], 1
            for n in reversed(shape):
                strides.insert(0, step)
                step *= max(n, 1)
        self.dtype, self.shape, self._strides = dtype, torch.Size(shape), tuple(strides)

    def stride(self, dim=None):
        return self._strides if dim is None else self._strides[dim]

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._strides == Fake(self.dtype, self.shape)._strides


def weights(shape, strides=None):
    blocks = shape[:-2] + tuple((n + 127) // 128 for n in shape[-2:])
    return Fake(torch.float8_e4m3fn, shape, strides), Fake(torch.float32, blocks)


@pytest.mark.parametrize("shape,strides,want", [
    ((256, 512), None, (1, 256, 512, 512)),
    ((1, 512), None, (1, 1, 512, 512)),
    ((1, 512), (0, 1), (1, 1, 512, 512)),             # one row: its stride says nothing
    ((3, 256, 500), (256 * 512, 512, 1), (3, 256, 500, 512)),
    ((3, 1, 512), None, (3, 1, 512, 512)),            # one row an expert: the experts' stride
    ((3, 1, 500), (512, 7, 1), (3, 1, 500, 512)),
    ((1, 1, 512), (9, 3, 1), (1, 1, 512, 512)),
])
def test_weight_strides(shape, strides, want):
    assert blockscale._weights(*weights(shape, strides)) == want


@pytest.mark.parametrize("shape,strides", [
    ((3, 1, 512), (0, 0, 1)),                         # one row for all experts
    ((3, 1, 512), (0, 512, 1)),
    ((3, 1, 512), (16, 16, 1)),                       # experts that overlap
    ((3, 256, 512), (0, 512, 1)),
    ((3, 256, 512), (300 * 512, 512, 1)),
    ((256, 512), (1, 256)),
])
def test_weight_strides_refused(shape, strides):
    with pytest.raises(ValueError):
        blockscale._weights(*weights(shape, strides))


BIG = 2 ** 32 + 4                                     # 4, if cut to 32 bits


@pytest.mark.parametrize("shape", [(BIG, 16), (16, BIG), (2 ** 31, 16)])
def test_matrices_past_32_bits_are_refused(shape):
    # (the library takes its sizes as 32-bit integers)
    with pytest.raises(ValueError):
        _tensors.row_stride(Fake(torch.bfloat16, shape), torch.bfloat16, "x")
    with pytest.raises(ValueError):
        blockscale._weights(*weights(shape))
    with pytest.raises(ValueError):
        blockscale._weights(*weights((2,) + shape))


def test_more_slots_than_32_bits_are_refused():
    with pytest.raises(ValueError):
        _tensors.check(Fake(torch.int32, (BIG,)), torch.int32, (BIG,), CUDA, "slots")
    assert _tensors.check(Fake(torch.int32, (4,)), torch.int32, (4,), CUDA, "slots") is None


def test_numbers_past_32_bits_are_refused():
    assert _tensors.fits(2 ** 31 - 1, "top_k") is None
    for n in (2 ** 31, BIG):
        with pytest.raises(ValueError):
            _tensors.fits(n, "top_k")
