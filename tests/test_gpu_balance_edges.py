"""Router balance on unusual logits.  Helpers as in test_gpu_balance.py."""
import numpy as np
import pytest
import torch

from .test_gpu_balance import draw, draw_dw, run

pytestmark = pytest.mark.gpu


def nan_of(sign, payload=0):
    bits = np.uint32((0xFFC00000 if sign else 0x7FC00000) | payload)
    return torch.from_numpy(np.array([bits], np.uint32).view(np.float32)).cuda()[0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(40, 4), (40, 1), (384, 8)])
@pytest.mark.parametrize("at,signs", [((3,), (1,)), ((3, 30), (1, 1)), ((0, 7, 39), (1, 0, 1)),
                                      ((5, 6, 7, 8, 9), (1, 1, 1, 1, 1))])
def test_nan_of_either_sign_makes_the_weights_nan(at, signs, E, K, dtype):
    # however many there are: they come first, in index order, and the token's
    # weights and gradient and the loss are NaN; the other tokens are untouched
    x = draw(9, E, 3)
    want, d_want = run(x.to(dtype), K, 0.01, d_loss=None, dw=draw_dw(9, K, 1))
    for e, sign in zip(at, signs):
        x[4, e] = nan_of(sign, 5 * e)
    r, d = run(x.to(dtype), K, 0.01, d_loss=None, dw=draw_dw(9, K, 1))
    assert bool(torch.isnan(r.weights[4]).all()) and bool(torch.isnan(d[4]).all())
    assert bool(torch.isnan(r.loss))
    first = r.ids[4].tolist()[:len(at)]
    assert first == list(at)[:K]
    rest = [t for t in range(9) if t != 4]
    assert torch.equal(r.ids[rest], want.ids[rest])
    assert torch.equal(r.weights[rest], want.weights[rest]) and torch.equal(d[rest], d_want[rest])
