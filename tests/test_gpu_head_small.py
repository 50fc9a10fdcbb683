"""Gradients of small calls (1024 rows, 2^25 padded multiplications at most): as near to
the definitions as rounding the result to 16 bits lets them be.  d is then held in two
16-bit terms, 2^-17 of each of its values at most (bfloat16; float16 2^-22) is lost; the logits' errors move p by some 2^-18.  So
beside the rounding of the result there is 2^-16 of the gradient's norm."""
import pytest
import torch

import head_ref as R
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head
from test_gpu_head import BF, HF, F32, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


# one slice of the labels, several, odd ones; shares cut along the labels and along the rows; a wide head
SIZES = [(50, 32, 64), (7, 8, 64), (700, 100, 256), (301, 29, 40), (1000, 2, 64), (50, 2000, 64), (129, 700, 77),
         (200, 65, 1000), (1000, 60, 60), (1024, 100, 100), (3, 500, 200)]


@pytest.mark.parametrize("n,v,h", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_gradients(n, v, h, dtype, reduction):
    x, w, b, t = inputs(n, v, h, dtype, F32)
    t[0] = 1
    grad = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda") \
        if reduction == "none" else torch.full((), 1000.0, device="cuda")
    _, lse = head.cross_entropy(x, w, t, b, reduction=reduction)
    got = head.cross_entropy_backward(grad, x, w, t, lse, b, reduction=reduction)
    want = R.cross_entropy(x, w, b, t, -1, reduction, grad)[2:5]
    for g, r, name in zip(got, want, ("dx", "dw", "db")):
        norm = r.norm()
        rounding = ((r.to(g.dtype).double() - r).norm() / norm).item()
        off = ((g.double() - r).norm() / norm).item()
        assert off <= 1.05 * rounding + 2.0 ** -16, (name, off, rounding)
