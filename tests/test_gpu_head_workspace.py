"""What a call leaves in its workspace, or what else stands there, does not reach
the next call's results: the blocks of the one-pass log-probabilities take their
row sums from each other through it."""
import pytest
import torch

from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def inputs(n, v, h, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(v, h, generator=g, device="cuda") * (1 + seed) / h ** 0.5).to(BF)
    x = torch.randn(n, h, generator=g, device="cuda").to(BF)
    b = torch.randn(v, generator=g, device="cuda")
    t = torch.randint(-1, v, (n,), generator=g, device="cuda").int()
    return x, w, b, t


def fills(ws):
    yield ws.zero_
    yield lambda: ws.fill_(255)
    yield lambda: ws.view(torch.float32).fill_(1.0)
    yield lambda: None  # what the last call left


# members: 21 with two rows to a block's pair, 79 of single blocks, one, two, 64 of pairs; and two passes
@pytest.mark.parametrize("n,v,h", [(3000, 5000, 64), (100, 5000, 64), (257, 200, 64), (300, 400, 40), (513, 16384, 64),
                                   (260, 20001, 64)])
def test_log_probs(n, v, h):
    ws = torch.empty(head.log_probs_workspace_size(BF, n, v, h), dtype=torch.uint8, device="cuda")
    for k in range(2):
        x, w, b, _ = inputs(n, v, h, k)
        want = head.log_probs(x, w, b)
        for fill in fills(ws):
            fill()
            assert torch.equal(head.log_probs(x, w, b, workspace=ws), want)
            assert D.read_status(ws) == 0


@pytest.mark.parametrize("n,v,h", [(1000, 3000, 64), (40, 50, 24)])
def test_cross_entropy(n, v, h):
    one = torch.ones((), device="cuda")
    f, g = (torch.empty(head.cross_entropy_workspace_size(BF, n, v, h, k), dtype=torch.uint8, device="cuda")
            for k in (False, True))
    for k in range(2):
        x, w, b, t = inputs(n, v, h, k)
        want_l = head.cross_entropy(x, w, t, b)
        want_g = head.cross_entropy_backward(one, x, w, t, want_l[1], b)
        for fill, fill2 in zip(fills(f), fills(g)):
            fill()
            fill2()
            got = head.cross_entropy(x, w, t, b, workspace=f)
            for p, q in zip(got + head.cross_entropy_backward(one, x, w, t, got[1], b, workspace=g), want_l + want_g):
                assert torch.equal(p, q)
