"""Labels that are nearly certain: their log-probability is 0 to within a few
units of 1, however large the logits, never above 0, and their loss never below.

Why: the row's largest logit m is taken from the logits first, and exactly (the
largest logit gives 0), the sum of exp(z - m) is at least 1, and only
z - m - log(sum) is returned."""
import pytest
import torch

from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
# one block, pairs; a member alone, several; more labels than the one-pass kernel holds
SIZES = [(5, 29, 64), (300, 200, 96), (100, 5000, 64), (300, 5001, 512), (140, 40000, 64), (300, 20001, 72)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def inputs(n, v, h, dtype, level):
    """Logits of spread 2 around `level` (from the bias), some rows with one label's 120 above."""
    g = torch.Generator(device="cuda").manual_seed(n + v + h)
    w = torch.randn(v, h, generator=g, device="cuda") * 2 / h ** 0.5
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    sure = torch.rand(n, generator=g, device="cuda") < 0.5
    x = torch.randn(n, h, generator=g, device="cuda")
    at = w[t]
    x = torch.where(sure[:, None], x + 120.0 * at / (at * at).sum(1, keepdim=True), x)
    b = level + 0.25 * torch.randn(v, generator=g, device="cuda")
    return x.to(dtype), w.to(dtype), b, t.int(), sure


@pytest.mark.parametrize("n,h", [(1, 8), (200, 64), (1000, 512), (130, 2048)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_label(n, h, dtype):
    x, w, b, t, _ = inputs(n, 1, h, dtype, 37.0)
    assert (head.log_probs(x, w, b) == 0).all()
    assert (head.log_probs(x, w) == 0).all()
    t.zero_()
    assert (head.cross_entropy(x, w, t, b, reduction="none")[0] == 0).all()
    assert head.cross_entropy(x, w, t, b)[0].item() == 0


@pytest.mark.parametrize("n,v,h", SIZES)
@pytest.mark.parametrize("level", [0.0, 3000.0, -3000.0])
def test_never_above_certain(n, v, h, level):
    x, w, b, t, sure = inputs(n, v, h, BF, level)
    lp = head.log_probs(x, w, b)
    assert (lp <= 0).all()
    # a label 40 or more above the rest is certain: the others add less than 40,000 e^-40
    top = (x.double() @ w.double().t() + b.double()).topk(2, 1).values
    clear = top[:, 0] - top[:, 1] > 40
    assert clear.sum() >= sure.sum() // 4
    assert (lp.max(1).values[clear] == 0).all()
    loss, _ = head.cross_entropy(x, w, t, b, reduction="none")
    assert (loss >= 0).all()
    hit = clear & (lp.argmax(1) == t)
    assert (loss[hit] == 0).all()


@pytest.mark.parametrize("n,v,h", SIZES)
@pytest.mark.parametrize("level", [0.0, 3000.0, -3000.0])
def test_probabilities_sum_to_one(n, v, h, level):
    """The level of the logits does not enter: the same rounded logits are in
    the sum and in what is returned.  A label's error is 2^-23 of its own
    |log_prob| (a difference and a product, each rounded), the sum's log carries
    the same of at most 11 and 2^-21 from the exponentials, their sum and the
    log; over the labels, sum p |log p| <= log V <= 11."""
    x, w, b, _, _ = inputs(n, v, h, BF, level)
    total = head.log_probs(x, w, b).double().exp().sum(1)
    assert ((total - 1).abs() <= 22 * 2.0 ** -23 + 2.0 ** -21).all()
