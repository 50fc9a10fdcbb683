"""The mean error of the logits, in units of 2^-24 of a logit.

The tensor cores cut the float32 accumulator off at every K = 16 step.  What that
loses on average for dense operands of either sign, 0.26 units a step, is put
back by a factor; what is left of it is under 0.13 units a step (float16 loses up
to 0.38), so a factor that is left out, doubled or turned round shows.  Sums that
are exact lose nothing and come out 0.26 units a step too large.  Operands of one
sign lose up to 1.75 units a step, and are short of their value by what is left.
Beside it: the factor, log2(e) and ln(2), each rounded (1.5 units together)."""
import pytest
import torch

from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
N = 32768
CONST = 1.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def operands(kind, h, g):
    x, w = torch.randn(N, h, generator=g, device="cuda"), torch.randn(1, h, generator=g, device="cuda")
    if kind == "towards":  # a target's features
        w = w * 1.5 / h ** 0.5
        x = x + 3.0 * w
    elif kind == "sparse":
        x = x * (torch.rand(N, h, generator=g, device="cuda") < 0.05)
    elif kind == "one-hot":
        x = torch.zeros(N, h, device="cuda")
        x[torch.arange(N), torch.randint(0, h, (N,), generator=g, device="cuda")] = 1.0
    elif kind == "integers":
        x, w = torch.randint(-2, 3, (N, h), generator=g, device="cuda").float(), \
            torch.randint(-2, 3, (1, h), generator=g, device="cuda").float()
    elif kind == "one sign":
        x, w = x.abs(), w.abs()
    return x, w


def mean_error(kind, h, dtype):
    """The slope of the error over the logit: with one label the lse is the logit."""
    num = den = 0.0
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(8 * h + seed)
        x, w = (p.to(dtype) for p in operands(kind, h, g))
        z = (x.double() @ w.double().t())[:, 0]
        _, lse = head.cross_entropy(x, w, torch.zeros(N, dtype=torch.int32, device="cuda"), reduction="none")
        num += ((lse.double() - z) * z).sum().item()
        den += (z * z).sum().item()
    return num / den * 2.0 ** 24


DEPTHS = [16, 64, 512, 2048, 4096, 8192]


@pytest.mark.parametrize("h", DEPTHS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["normal", "towards"])
def test_dense(kind, h, dtype):
    assert abs(mean_error(kind, h, dtype)) <= 0.13 * (h // 16) + CONST


@pytest.mark.parametrize("h", DEPTHS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["one-hot", "integers"])
def test_exact_sums(kind, h, dtype):
    assert abs(mean_error(kind, h, dtype) - 0.26 * (h // 16)) <= CONST


@pytest.mark.parametrize("h", DEPTHS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sparse(h, dtype):
    assert -CONST <= mean_error("sparse", h, dtype) <= 0.26 * (h // 16) + CONST


@pytest.mark.parametrize("h", DEPTHS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_sign(h, dtype):
    assert -(1.75 - 0.26) * (h // 16) - CONST <= mean_error("one sign", h, dtype) <= CONST
