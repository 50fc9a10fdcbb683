"""The operators around the label head as they are used: a convolutional block's norm,
dropout into the residual stream, the head, and a loss over the decoder's own N-best
lists; its gradients against differences, and the step captured in a CUDA graph."""
import numpy as np
import pytest
import torch

import head_ref
import more_ref as R
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


B, N, L, C, V, GROUPS, P = 3, 4, 9, 32, 24, 4, 0.2


def inputs(seed, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda")

    S = B * N
    lens = torch.randint(1, L + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
    tokens = torch.randint(0, V, (S, L), generator=g, device="cuda").int()
    tokens = torch.where(torch.arange(L, device="cuda") < lens[:, None], tokens, torch.full_like(tokens, -1))
    return dict(x=normal(S, L, C).to(dtype), gw=1 + 0.2 * normal(C), gb=0.1 * normal(C), lw=1 + 0.2 * normal(C),
                lb=0.1 * normal(C), w=(normal(V, C) / C ** 0.5).to(dtype), b=0.1 * normal(V), tokens=tokens, lens=lens,
                rng=torch.tensor([seed, 1], dtype=torch.int64, device="cuda"), old=normal(S, L).abs(), ref=normal(S, L).abs(),
                adv=normal(S), chosen=torch.randint(0, N, (B,), generator=g, device="cuda", dtype=torch.int32),
                rejected=torch.randint(0, N, (B,), generator=g, device="cuda", dtype=torch.int32))


def step(a, which):
    """One training step's loss and gradients: x, the group norm's, the layer norm's, the head's."""
    one = torch.ones((), device="cuda")
    h, gm, gr = head.group_norm(a["x"], GROUPS, a["gw"], a["gb"], lengths=a["lens"], activation="silu")
    z = head.dropout(h, P, a["rng"], residual=a["x"])
    y, lm, lr = head.layer_norm(z, a["lw"], a["lb"])
    nll, lse = head.cross_entropy(y, a["w"], a["tokens"], a["b"], reduction="none")
    if which == "policy":
        loss, stats, dnll = head.policy_loss(nll, a["old"], a["adv"], lengths=a["lens"], ref_nll=a["ref"], kl_weight=0.1,
                                             reduction="sequence_mean", grad=one)
    else:
        loss, _, dnll = head.preference_loss(nll.view(B, N, L), a["chosen"], a["rejected"], lengths=a["lens"].view(B, N),
                                             ref_nll=a["ref"].view(B, N, L), grad=one)
        dnll = dnll.view(B * N, L)
    dy, dw, db = head.cross_entropy_backward(dnll, y, a["w"], a["tokens"], lse, a["b"], reduction="none")
    dz, dlw, dlb = head.layer_norm_backward(dy, z, a["lw"], lm, lr)
    dh = head.dropout_backward(dz, P, a["rng"])
    dx, dgw, dgb = head.group_norm_backward(dh, a["x"], GROUPS, a["gw"], a["gb"], gm, gr, lengths=a["lens"], activation="silu")
    return loss, dict(x=dx.float() + dz.float(), gw=dgw, gb=dgb, lw=dlw, lb=dlb, w=dw, b=db)


def reference(a, which):
    """The same loss in 64 bits, without a rounding between the operators."""
    d = {k: v.double() if v.is_floating_point() else v for k, v in a.items()}
    h = R.GroupNorm(d["x"], GROUPS, d["gw"], d["gb"], a["lens"], 1e-5, "silu").y.view(d["x"].shape)
    keep, scale = R.kept(0, h.numel(), P, *a["rng"].tolist())
    z = d["x"] + torch.where(torch.from_numpy(keep).cuda().view(h.shape), h * float(np.float64(65536) / (65536 - round(P * 65536))),
                             torch.zeros((), dtype=torch.float64, device="cuda"))
    y = head_ref.layer_norm(z.view(-1, C), d["lw"], d["lb"], 1e-5)[0]
    lp = torch.log_softmax(y @ d["w"].t() + d["b"], 1)
    t = a["tokens"].view(-1).long()
    nll = torch.where(t >= 0, -lp.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(lp[:, 0])).view(B * N, L)
    one = torch.ones((), device="cuda")
    if which == "policy":
        return R.policy(nll, d["old"], d["adv"][:, None].expand(-1, L), a["lens"], d["ref"], 0.2, 0.2, 0.1, "sequence_mean",
                        one)["loss"]
    return R.preference(nll.view(B, N, L), a["chosen"], a["rejected"], a["lens"].view(B, N), d["ref"].view(B, N, L), 0.1, 0.0,
                        0.0, False, "mean", one)["loss"]


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_a_step_and_its_gradients(which):
    """Half precision rounds each of the four stages' values to 2^-11 of themselves, forward and backward: eight
    roundings of either sign, 4 sqrt(8) 2^-11 = 6e-3 of a gradient's norm and of the loss's terms (of order 1)."""
    a = inputs(5, HF)
    if which == "preference":
        a["rejected"] = (a["chosen"] + 1) % N
    loss, grads = step(a, which)
    assert abs(loss.item() - reference(a, which).item()) < 6e-3
    for k, g in grads.items():
        # along the gradient itself, and along a direction of its own
        for i in range(2):
            d = g.double() if i == 0 else torch.randn(g.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                                                      dtype=torch.float64) * g.double().norm() / g.numel() ** 0.5
            eps = 1e-4 / d.abs().max().item()
            f = [reference({**a, k: a[k].double() + s * eps * d}, which).item() for s in (1, -1)]
            diff = (f[0] - f[1]) / (2 * eps)
            assert abs((g.double() * d).sum().item() - diff) <= 6e-3 * (g.double().norm() * d.norm()).item(), (k, i)


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_a_captured_step(which):
    a = inputs(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(a, which)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads = step(a, which)
    for seed in (2, 1, 3):
        new = inputs(seed)
        for k in a:
            a[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        wl, wg = step(new, which)
        assert torch.equal(loss, wl) and all(torch.equal(grads[k], wg[k]) for k in wg)


# in one launch, in a cluster, in two launches; in one cluster, in several launches, with a count before
@pytest.mark.parametrize("T,C,groups", [(30, 64, 8), (1500, 64, 2), (30000, 64, 1)])
def test_captured_norms(T, C, groups):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, dy = (torch.randn(2, T, C, generator=g, device="cuda").bfloat16() for _ in range(2))
    w, b = torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")
    n = torch.tensor([T, T // 2], dtype=torch.int32, device="cuda")

    def call():
        y, mean, rstd = head.group_norm(x, groups, w, b, lengths=n, activation="silu")
        return y, mean, rstd, *head.group_norm_backward(dy, x, groups, w, b, mean, rstd, lengths=n, activation="silu")

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for lens in ([T, 1], [0, T], [T // 3, T // 2]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        x.copy_(torch.randn(2, T, C, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, call()))


@pytest.mark.parametrize("S,L", [(40, 30), (3000, 50), (10000, 16)])
def test_captured_losses(S, L):
    g = torch.Generator(device="cuda").manual_seed(S)
    nll, old, ref = (torch.rand(S, L, generator=g, device="cuda") for _ in range(3))
    adv, one = torch.randn(S, generator=g, device="cuda"), torch.ones((), device="cuda")
    n = torch.full((S,), L, dtype=torch.int32, device="cuda")
    c, r = (torch.randint(-1, 2, (S // 2,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2))

    def call():
        return (*head.policy_loss(nll, old, adv, lengths=n, ref_nll=ref, kl_weight=0.1, grad=one),
                *head.preference_loss(nll.view(S // 2, 2, L), c, r, lengths=n.view(S // 2, 2), ref_nll=ref.view(S // 2, 2, L),
                                      grad=one))

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        n.copy_(torch.randint(0, L + 1, (S,), generator=g, device="cuda"))
        nll.copy_(torch.rand(S, L, generator=g, device="cuda"))
        c.copy_(torch.randint(-1, 2, (S // 2,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, call()))
