"""Gradients per row (reduction "none"): what stands at a row that takes no part,
or at one whose gradient is not finite, does not reach the other rows."""
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


def case(n, v, h, dtype):
    """Inputs whose rows 3 and n - 2 are kept, 0 and n - 1 ignored and 1 out of range."""
    g = torch.Generator(device="cuda").manual_seed(n + v + h)
    w = (torch.randn(v, h, generator=g, device="cuda") / h ** 0.5).to(dtype)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    b = torch.randn(v, generator=g, device="cuda")
    t = torch.randint(0, v, (n,), generator=g, device="cuda").int()
    t[torch.rand(n, generator=g, device="cuda") < 0.3] = -1
    t[0] = t[n - 1] = -1
    t[1] = v
    t[3] = t[n - 2] = 2
    grad = torch.randn(n, generator=g, device="cuda")
    return x, w, b, t, grad


def backward(x, w, b, t, grad):
    _, lse = head.cross_entropy(x, w, t, b, reduction="none")
    return head.cross_entropy_backward(grad, x, w, t, lse, b, reduction="none")


@pytest.mark.parametrize("n,v,h", [(9, 5, 16), (700, 300, 64)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), 1e13, -3e38])
def test_gradients_of_rows_that_take_no_part(n, v, h, dtype, value):
    x, w, b, t, grad = case(n, v, h, dtype)
    out = (t < 0) | (t >= v)
    grad[out] = 0.0
    want = backward(x, w, b, t, grad)
    assert all(torch.isfinite(g).all() for g in want) and (want[0][out] == 0).all()
    for at in (out, torch.arange(n, device="cuda") == 0, torch.arange(n, device="cuda") == 1,
               torch.arange(n, device="cuda") == n - 1):
        got = backward(x, w, b, t, torch.where(at, torch.full_like(grad, value), grad))
        for p, q in zip(got, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_gradient_that_is_not_finite_stays_with_its_row(dtype, value):
    """dx of the other rows is what it is without; the sums over rows show it."""
    x, w, b, t, grad = case(700, 300, 64, dtype)
    grad[3] = 0.0
    want = backward(x, w, b, t, grad)
    grad[3] = value
    got = backward(x, w, b, t, grad)
    other = torch.arange(700, device="cuda") != 3
    assert torch.equal(got[0][other], want[0][other])
    assert not torch.isfinite(got[0][3]).any()
    assert not torch.isfinite(got[2]).any()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_no_gradient_at_all(dtype):
    x, w, b, t, grad = case(700, 300, 64, dtype)
    for g in backward(x, w, b, t, torch.zeros_like(grad)):
        assert (g == 0).all()
