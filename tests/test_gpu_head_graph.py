"""The label head's calls captured in a CUDA graph: replayed on other inputs, and on
targets of which another number is ignored, they give the bits of the plain calls."""
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


def inputs(n, v, h, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    w = (torch.randn(v, h, generator=g, device="cuda") / h ** 0.5).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.2 * seed, torch.full_like(t, -1), t).int()
    return [x, w, torch.randn(v, generator=g, device="cuda"), t, 1 + 0.1 * torch.randn(h, generator=g, device="cuda"),
            0.1 * torch.randn(h, generator=g, device="cuda")]


def step(x, w, b, t, gamma, beta):
    one = torch.ones((), device="cuda")
    y, mean, rstd = head.layer_norm(x, gamma, beta)
    log_prob = head.log_probs(y, w, b)
    loss, lse = head.cross_entropy(y, w, t, b)
    dy, dw, db = head.cross_entropy_backward(one, y, w, t, lse, b)
    dx, dgamma, dbeta = head.layer_norm_backward(dy, x, gamma, mean, rstd)
    return [y, mean, rstd, log_prob, loss, lse, dy, dw, db, dx, dgamma, dbeta]


# the one-pass log-probabilities on single blocks, on pairs and with one member, and in two passes; odd sizes
@pytest.mark.parametrize("n,v,h,dtype", [(50, 32, 64, BF), (128, 5000, 128, BF), (700, 5000, 128, HF), (301, 997, 77, HF),
                                         (260, 20001, 64, BF)])
def test_a_captured_step(n, v, h, dtype):
    args = inputs(n, v, h, dtype, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(*args)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*args)
    for seed in (2, 1, 3):
        new = inputs(n, v, h, dtype, seed)
        for p, q in zip(args, new):
            p.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, step(*new)):
            assert torch.equal(p, q)
