"""Gradients of rows whose target is nearly certain: exp(z - lse) - 1 is 0 there,
not what the lse lost on its way from the forward call.

Why: the lse is max z + log(sum) in the units of the logits, rounded once, and the
backward call makes the same rounded z again, so a label 40 above the rest has
z - lse = 0, and the others at most e^-40 each."""
import pytest
import torch

from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def inputs(n, v, h, dtype, level):
    """Every row's target is far above the rest, by the row's own length."""
    g = torch.Generator(device="cuda").manual_seed(n + v + h)
    w = torch.randn(v, h, generator=g, device="cuda") * 2 / h ** 0.5
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    at = w[t]
    far = 150 + 100 * torch.rand(n, 1, generator=g, device="cuda")
    x = torch.randn(n, h, generator=g, device="cuda") + far * at / (at * at).sum(1, keepdim=True)
    return x.to(dtype), w.to(dtype), level + 0.25 * torch.randn(v, generator=g, device="cuda"), t.int()


def backward(x, w, b, t, reduction="sum"):
    grad = torch.ones(x.shape[0] if reduction == "none" else (), device="cuda")
    _, lse = head.cross_entropy(x, w, t, b, reduction=reduction)
    return head.cross_entropy_backward(grad, x, w, t, lse, b, reduction=reduction)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,h", [(1, 8), (300, 64), (130, 2048)])
def test_one_label(n, h, dtype, reduction):
    x, w, b, t = inputs(n, 1, h, dtype, 37.0)
    for g in backward(x, w, b, t, reduction) + backward(x, w, None, t, reduction)[:2]:
        assert (g == 0).all()


@pytest.mark.parametrize("reduction", ["none", "sum"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("level", [0.0, 3000.0, -3000.0])
@pytest.mark.parametrize("n,v,h", [(50, 29, 128), (700, 300, 256), (300, 5001, 512)])
def test_certain_targets(n, v, h, level, dtype, reduction):
    x, w, b, t = inputs(n, v, h, dtype, level)
    z = x.double() @ w.double().t() + b.double()
    top = z.topk(2, 1)
    assert (top.indices[:, 0] == t).all() and (top.values[:, 0] - top.values[:, 1] > 40).all()
    # of every row, all of d together is at most 2 V e^-40 (the rounding of z and the exponential: less than twice)
    d = 2 * v * 2.0 ** -57
    dx, dw, db = backward(x, w, b, t, reduction)
    assert (dx.double().abs() <= 2 * d * w.double().abs().max()).all()
    assert (dw.double().abs() <= 2 * d * x.double().abs().sum(0)).all()
    assert (db.double().abs() <= 2 * d * n).all()
