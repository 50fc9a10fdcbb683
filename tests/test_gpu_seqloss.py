"""The policy and preference losses of N-best lists, with their gradients, against
definitions in 64 bits (more_ref)."""
import pytest
import torch

import more_ref as R
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

F32 = torch.float32
REDUCTIONS = ["none", "mean", "sum", "sequence_mean"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def lists(lead, L, seed=0, ragged=True, per_token=False):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000 + L + sum(lead))

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda")

    old = 2.0 * torch.rand(*lead, L, generator=g, device="cuda") ** 3
    nll, ref = old + 0.3 * normal(*lead, L) * old, old + 0.4 * normal(*lead, L) * old
    adv = normal(*lead, L) if per_token else normal(*lead)
    n = torch.randint(0, L + 1, lead, generator=g, device="cuda", dtype=torch.int32) if ragged else None
    return nll, old, ref, adv, n, g


def bits(p, q):
    return torch.equal(p.view(torch.int32), q.view(torch.int32))


def near(got, want, what=""):
    for k in [k for k in want if not k.startswith("e_")]:
        v, e = want[k], want["e_" + k]
        a = got[k].double().view(v.shape)
        bad = ~((a - v).abs() <= e + R.u * v.abs() + R.TINY[F32]) & ~(torch.isnan(a) & torch.isnan(v))
        assert not bad.any(), (what, k, int(bad.sum()), a[bad][:3].tolist(), v[bad][:3].tolist(), e.expand(v.shape)[bad][:3].tolist())


def check_policy(nll, old, adv, n, ref, reduction, grad=None, lo=0.2, hi=0.3, klw=0.05, ws=None, clean=None):
    lead, L = nll.shape[:-1], nll.shape[-1]
    if grad is None:
        grad = torch.full((), 2.5, device="cuda") if reduction != "none" else torch.randn(
            nll.shape, generator=torch.Generator(device="cuda").manual_seed(L), device="cuda")
    got = head.policy_loss(nll, old, adv, lengths=n, ref_nll=ref, clip_low=lo, clip_high=hi, kl_weight=klw,
                           reduction=reduction, grad=grad, workspace=ws)
    two = head.policy_loss(nll, old, adv, lengths=n, ref_nll=ref, clip_low=lo, clip_high=hi, kl_weight=klw,
                           reduction=reduction)
    assert len(two) == 2 and all(bits(p, q) for p, q in zip(two, got))
    a, b, c = clean if clean is not None else (nll, old, ref)
    S = lead.numel()
    full = adv if adv.dim() == nll.dim() else adv[..., None].expand(nll.shape)
    want = R.policy(a.reshape(S, L), b.reshape(S, L), full.reshape(S, L), None if n is None else n.reshape(S),
                    None if c is None else c.reshape(S, L), lo, hi, klw, reduction,
                    grad.reshape(S, L) if reduction == "none" else grad)
    near(dict(zip(("loss", "stats", "dnll"), got)), want, reduction)
    return got


@pytest.mark.parametrize("lead,L", [((1,), 1), ((3, 5), 1), ((32, 10), 40), ((4,), 37), ((2, 3), 1000), ((7,), 4099), ((), 50),
                                    ((5000,), 3), ((3000, 2), 8), ((2,), 300000), ((1,), 4)])
@pytest.mark.parametrize("reduction", REDUCTIONS)
def test_policy_loss(lead, L, reduction):
    for per_token, ragged, kl in ((False, True, True), (True, False, True), (True, True, False)):
        nll, old, ref, adv, n, _ = lists(lead, L, 1, ragged, per_token)
        if ragged and lead:
            n.view(-1)[0] = L
        elif ragged:
            n.fill_(L // 2)
        check_policy(nll, old, adv, n, ref if kl else None, reduction)


def test_policy_lengths():
    """None, one, all, out of range (clamped); what lies behind them is of no account."""
    nll, old, ref, adv, _, _ = lists((6,), 50)
    n = torch.tensor([0, 1, 50, 23, -4, 99], dtype=torch.int32, device="cuda")
    dead = ~R.frames(nll, n)[1]
    for reduction in REDUCTIONS:
        want = check_policy(nll, old, adv, n, ref, reduction)
        for v in (float("nan"), float("inf"), torch.finfo(F32).min):
            bad = [t.clone() for t in (nll, old, ref)]
            for t in bad:
                t[dead] = v
            got = check_policy(bad[0], bad[1], adv, n, bad[2], reduction, clean=(nll, old, ref))
            for p, q in zip(got, want):
                assert torch.equal(p, q)
            assert (got[2][dead] == 0).all() and (reduction != "none" or (got[0][dead] == 0).all())


def test_policy_without_tokens():
    nll, old, ref, adv, _, _ = lists((6,), 50)
    one = torch.ones((), device="cuda")
    for n, v in ((torch.zeros(6, dtype=torch.int32, device="cuda"), slice(None)), (None, slice(0, 0))):
        for reduction in ("mean", "sum", "sequence_mean"):
            loss, stats, dnll = head.policy_loss(nll[v], old[v], adv[v], lengths=n, ref_nll=ref[v], reduction=reduction, grad=one)
            assert loss.item() == 0 if reduction == "sum" else torch.isnan(loss)
            assert torch.isnan(stats).all() and (dnll == 0).all()
    loss, stats, dnll = head.policy_loss(nll[:, :0], old[:, :0], adv, grad=one)
    assert torch.isnan(loss) and dnll.shape == (6, 0)


def test_policy_at_the_border():
    """Ratios at the float32 neighbours of the border: which side they are on is decided exactly."""
    lo, hi = 0.2, 0.28
    for border, sign in ((torch.tensor(hi, dtype=torch.float64).log1p(), 1.0), (torch.tensor(-lo, dtype=torch.float64).log1p(), -1.0)):
        base = torch.linspace(0.5, 3.0, 2000, dtype=torch.float64)
        old = base.float()
        nll = (old.double() - border).float()
        for _ in range(3):
            nll = torch.nextafter(nll, torch.full_like(nll, -100.0))
        rows = []
        for _ in range(7):
            rows.append(nll)
            nll = torch.nextafter(nll, torch.full_like(nll, 100.0))
        nll, old = torch.stack(rows).cuda(), old.expand(7, -1).contiguous().cuda()
        adv = torch.full(nll.shape, sign, device="cuda")
        _, stats, dnll = head.policy_loss(nll, old, adv, clip_low=lo, clip_high=hi, reduction="sum",
                                          grad=torch.ones((), device="cuda"))
        d = old.double() - nll.double()
        held = d > border.cuda() if sign > 0 else d < border.cuda()
        assert torch.equal(dnll == 0, held) and 0 < held.double().mean() < 1
        assert stats[1].item() == held.float().mean().item()


def test_policy_cancelling_advantages():
    """A list's advantages sum to nothing: the loss is a small rest, and still right to its own digits."""
    nll, old, ref, _, _, g = lists((64, 16), 200, 3, ragged=False)
    nll = old + 1e-4 * torch.randn(old.shape, generator=g, device="cuda") * old
    r = torch.rand(64, 16, generator=g, device="cuda", dtype=torch.float64)
    adv = ((r - r.mean(1, keepdim=True)) / r.std(1, keepdim=True)).float()
    loss, _ = head.policy_loss(nll, old, adv, reduction="sequence_mean")
    rho = torch.exp(old.double() - nll.double())
    want = -(rho * adv.double()[..., None]).mean()
    assert abs(loss.item() / want.item() - 1) < 2e-6 and abs(want.item()) < 1e-4


def test_policy_ends_of_the_range():
    inf, big = float("inf"), 200.0
    nll = torch.tensor([[0.0, big, 0.0, inf, 1.0, 1.0]], device="cuda")
    old = torch.tensor([[big, 0.0, 0.0, 1.0, 1.0, 1.0]], device="cuda")
    for sign in (1.0, -1.0, 0.0):
        adv = torch.full((1,), sign, device="cuda")
        loss, stats, dnll = head.policy_loss(nll, old, adv, reduction="none", grad=torch.ones_like(nll))
        rho = torch.exp(old.double() - nll.double())
        want = -torch.minimum(rho * sign, rho.clamp(0.8, 1.2) * sign)
        assert torch.allclose(loss, want.float(), rtol=1e-6, atol=0)
        assert sign != 0 or (dnll == 0).all()
    # a clip_low of 1 or more holds nothing from below, an infinite clip_high nothing from above
    loss, stats, _ = head.policy_loss(nll[:, 4:], old[:, 4:] - 3, -torch.ones(1, device="cuda"), clip_low=1.0,
                                      grad=torch.ones((), device="cuda"))
    assert stats[1] == 0
    loss, stats, _ = head.policy_loss(nll[:, 4:], old[:, 4:] + 50, torch.ones(1, device="cuda"), clip_high=inf,
                                      grad=torch.ones((), device="cuda"))
    assert stats[1] == 0 and torch.allclose(loss, -torch.exp(torch.tensor(50.0, device="cuda")), rtol=1e-5)
    # a token that the model rules out: the KL term is infinite, the others keep their gradients
    ref = torch.ones_like(nll)
    loss, stats, dnll = head.policy_loss(nll[:, 1:], old[:, 1:], torch.ones(1, device="cuda"), ref_nll=ref[:, 1:],
                                         kl_weight=0.1, reduction="sum", grad=torch.ones((), device="cuda"))
    assert loss == inf and stats[0] == inf and torch.isfinite(dnll[0, [1, 3, 4]]).all() and dnll[0, 2] == inf


def check_preference(nll, c, r, n, ref, reduction, grad=None, beta=0.25, margin=0.25, s=0.125, average=False, ws=None,
                     clean=None):
    B = nll.shape[0]
    if grad is None:
        grad = torch.full((), -1.5, device="cuda") if reduction != "none" else torch.randn(
            B, generator=torch.Generator(device="cuda").manual_seed(B), device="cuda")
    kw = dict(lengths=n, ref_nll=ref, beta=beta, margin=margin, label_smoothing=s, average=average, reduction=reduction)
    got = head.preference_loss(nll, c, r, grad=grad, workspace=ws, **kw)
    two = head.preference_loss(nll, c, r, **kw)
    assert len(two) == 2 and all(bits(p, q) for p, q in zip(two, got))
    a, b = clean if clean is not None else (nll, ref)
    near(dict(zip(("loss", "margins", "dnll"), got)),
         R.preference(a, c, r, n, b, beta, margin, s, average, reduction, grad), reduction)
    return got


def pairs(B, N, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + B * 31 + N)
    c = torch.randint(0, N, (B,), generator=g, device="cuda", dtype=torch.int32)
    r = torch.randint(-1, N, (B,), generator=g, device="cuda", dtype=torch.int32)
    r[0] = (c[0] + 1) % N
    return c, r


@pytest.mark.parametrize("B,N,L", [(1, 1, 1), (1, 2, 1), (3, 2, 7), (32, 10, 40), (5, 3, 256), (4, 4, 257), (3, 2, 1000),
                                   (2, 3, 5001), (3000, 2, 8), (1500, 3, 300), (1, 2, 100000), (9, 16, 4)])
@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
def test_preference_loss(B, N, L, reduction):
    for ragged, with_ref, average, s in ((True, True, False, 0.125), (False, True, True, 0.0), (True, False, True, 1.0)):
        nll, _, ref, _, n, _ = lists((B, N), L, 2, ragged)
        c, r = pairs(B, N)
        check_preference(nll, c, r, n, ref if with_ref else None, reduction, average=average, s=s)


def test_preference_pairs_and_status():
    """No pair, the same hypothesis twice, an index past the end (reported), no pair at all."""
    nll, _, ref, _, n, _ = lists((6, 4), 30)
    c = torch.tensor([0, 1, 2, -1, 5, 3], dtype=torch.int32, device="cuda")
    r = torch.tensor([1, 1, -1, 2, 0, 0], dtype=torch.int32, device="cuda")
    ws = torch.empty(head.preference_loss_workspace_size(6, 4, 30), dtype=torch.uint8, device="cuda")
    for reduction in ("none", "mean", "sum"):
        _, margins, dnll = check_preference(nll, c, r, n, ref, reduction, ws=ws)
        assert D.read_status(ws) == head.DEV_TARGET
        assert (margins[2:5] == 0).all() and (dnll[1:5] == 0).all() and margins[1].item() == -0.25
    c[4] = -7
    check_preference(nll, c, r, n, ref, "mean", ws=ws)
    assert D.read_status(ws) == 0
    none = torch.full_like(c, -1)
    one = torch.ones((), device="cuda")
    loss, margins, dnll = head.preference_loss(nll, none, none, lengths=n, ref_nll=ref, grad=one)
    assert torch.isnan(loss) and (margins == 0).all() and (dnll == 0).all()
    loss, margins, dnll = head.preference_loss(nll, none, none, lengths=n, ref_nll=ref, grad=one, reduction="sum")
    assert loss == 0 and (dnll == 0).all()
    loss, margins, dnll = head.preference_loss(nll[:0], none[:0], none[:0], grad=one)
    assert torch.isnan(loss) and margins.shape == (0,) and dnll.shape == (0, 4, 30)
    c[4] = r[2] = c[3] = 0
    loss, margins, dnll = head.preference_loss(nll[..., :0], c, r, grad=one, beta=0.5)
    assert abs(loss.item() - 0.6931472) < 1e-6 and (margins == 0).all()


def test_without_a_workspace():
    """Small calls may go without one, by the C call too; with one they leave their status in it."""
    nll, old, ref, adv, n, _ = lists((5, 4), 30)
    c, r = torch.tensor([0, 1, 9, 2, 3], dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    one, s = torch.ones((), device="cuda"), torch.cuda.current_stream().cuda_stream
    want = head.preference_loss(nll, c, r, lengths=n, ref_nll=ref)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    for w in (None, ws):
        loss, margins = torch.empty((), device="cuda"), torch.empty(5, device="cuda")
        assert head._lib()["ctcpb_preference_loss"](
            nll.data_ptr(), 30, ref.data_ptr(), 30, c.data_ptr(), r.data_ptr(), n.data_ptr(), 5, 4, 30, 0.1, 0.0, 0.0, 0, 1,
            one.data_ptr(), loss.data_ptr(), margins.data_ptr(), None, None if w is None else w.data_ptr(),
            0 if w is None else 256, s) == D.OK
        assert torch.equal(loss, want[0]) and torch.equal(margins, want[1])
    assert D.read_status(ws) == head.DEV_TARGET
    head.policy_loss(nll, old, adv, lengths=n, workspace=ws)
    assert D.read_status(ws) == 0


def test_preference_lengths():
    nll, _, ref, _, _, _ = lists((5, 3), 40)
    n = torch.tensor([[0, 1, 40], [40, 0, 0], [0, 0, 5], [-3, 99, 7], [20, 20, 20]], dtype=torch.int32, device="cuda")
    c, r = pairs(5, 3, 1)
    c[2], r[2] = 0, 1  # two empty hypotheses
    dead = ~R.frames(nll.view(15, 40), n.view(-1))[1].view(5, 3, 40)
    for average in (False, True):
        want = check_preference(nll, c, r, n, ref, "mean", average=average)
        for v in (float("nan"), float("inf"), torch.finfo(F32).min):
            a, b = nll.clone(), ref.clone()
            a[dead], b[dead] = v, v
            got = check_preference(a, c, r, n, b, "mean", average=average, clean=(nll, ref))
            for p, q in zip(got, want):
                assert torch.equal(p, q)


def test_preference_far_from_even():
    """Margins of hundreds: the loss is the margin itself or nearly nothing, its gradient 1 or nearly nothing."""
    nll = torch.zeros(2, 2, 8, device="cuda")
    nll[0, 1], nll[1, 0] = 100.0, 100.0
    c, r = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    loss, z, dnll = head.preference_loss(nll, c, r, beta=1.0, reduction="none", grad=torch.ones(2, device="cuda"))
    assert z.tolist() == [800.0, -800.0] and loss.tolist() == [0.0, 800.0]
    assert (dnll[0] == 0).all() and (dnll[1, 0] == 1).all() and (dnll[1, 1] == -1).all()


def test_strides():
    nll, old, ref, adv, n, _ = lists((12,), 44, per_token=True)
    want = check_policy(nll, old, adv, n, ref, "mean")
    wide = torch.full((12, 400), float("nan"), device="cuda")
    for off in (4, 1):
        views = []
        for i, t in enumerate((nll, old, ref, adv)):
            wide[:, 100 * i + off:100 * i + off + 44] = t
            views.append(wide[:, 100 * i + off:100 * i + off + 44])
        got = check_policy(views[0], views[1], views[3], n, views[2], "mean")
        for p, q in zip(got, want):
            assert torch.allclose(p, q, rtol=1e-6)
    c, r = pairs(4, 3)
    want = check_preference(nll.view(4, 3, 44), c, r, n.view(4, 3), ref.view(4, 3, 44), "mean")
    for off in (4, 1):
        views = []
        for i, t in enumerate((nll, ref)):
            wide[:, 100 * i + off:100 * i + off + 44] = t
            views.append(wide.as_strided((4, 3, 44), (1200, 400, 1), 100 * i + off))
        got = check_preference(views[0], c, r, n.view(4, 3), views[1], "mean")
        for p, q in zip(got, want):
            assert torch.allclose(p, q, rtol=1e-6)


def test_offsets_past_32_bits():
    nll, old, ref, adv, n, _ = lists((3,), 40)
    far = torch.zeros(2 * 0x60000000 + 40, device="cuda")
    view = far.as_strided((3, 40), (0x60000000, 1))
    view.copy_(nll)
    for p, q in zip(check_policy(view, old, adv, n, ref, "mean"), check_policy(nll, old, adv, n, ref, "mean")):
        assert torch.equal(p, q)
    c, r = torch.tensor([2], dtype=torch.int32, device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda")
    got = head.preference_loss(far.as_strided((1, 3, 40), (0, 0x60000000, 1)), c, r, ref_nll=ref[None])
    want = head.preference_loss(nll[None], c, r, ref_nll=ref[None])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_same_bits_again_and_on_another_stream():
    nll, old, ref, adv, n, _ = lists((300, 8), 333)
    c, r = pairs(300, 8)
    one = torch.ones((), device="cuda")

    def calls():
        return (*head.policy_loss(nll, old, adv, lengths=n, ref_nll=ref, kl_weight=0.1, grad=one),
                *head.preference_loss(nll, c, r, lengths=n, ref_nll=ref, grad=one))

    want = calls()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            got = calls()
        s.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
def test_policy_gradient_against_differences(reduction):
    nll, old, ref, adv, n, g = lists((4, 3), 20)
    one = torch.ones((), device="cuda")
    n.clamp_(min=1)
    _, _, dnll = head.policy_loss(nll, old, adv, lengths=n, ref_nll=ref, clip_low=0.2, clip_high=0.3, kl_weight=0.1,
                                  reduction=reduction, grad=one)
    d = torch.randn(nll.shape, generator=g, device="cuda").double()
    step = 1e-7  # no ratio is so near to the border

    def f(v):
        return R.policy(v.view(12, 20), old.view(12, 20).double(), adv.reshape(12, 1).expand(12, 20).double(), n.view(-1),
                        ref.view(12, 20).double(), 0.2, 0.3, 0.1, reduction, one)["loss"]

    diff = (f(nll.double() + step * d) - f(nll.double() - step * d)) / (2 * step)
    assert abs((dnll.double() * d).sum() - diff) <= 1e-5 * (dnll.double().abs() * d.abs()).sum()


@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_against_differences(average):
    nll, _, ref, _, n, g = lists((4, 3), 20)
    one = torch.ones((), device="cuda")
    c, r = pairs(4, 3)
    _, _, dnll = head.preference_loss(nll, c, r, lengths=n, ref_nll=ref, beta=0.5, margin=0.1, label_smoothing=0.1,
                                      average=average, grad=one)
    d = torch.randn(nll.shape, generator=g, device="cuda").double()
    step = 1e-5

    def f(v):
        return R.preference(v, c, r, n, ref.double(), 0.5, 0.1, 0.1, average, "mean", one)["loss"]

    diff = (f(nll.double() + step * d) - f(nll.double() - step * d)) / (2 * step)
    assert abs((dnll.double() * d).sum() - diff) <= 1e-5 * (dnll.double().abs() * d.abs()).sum()


def test_refusals():
    nll, old, ref, adv, n, _ = lists((4, 3), 20)
    c, r = pairs(4, 3)
    one, small = torch.ones((), device="cuda"), torch.empty(64, dtype=torch.uint8, device="cuda")
    for bad in (lambda: head.policy_loss(nll.cpu(), old, adv), lambda: head.policy_loss(nll.half(), old, adv),
                lambda: head.policy_loss(nll, old[:2], adv), lambda: head.policy_loss(nll, old, adv[:2]),
                lambda: head.policy_loss(nll, old, adv.double()), lambda: head.policy_loss(nll, old, None),
                lambda: head.policy_loss(nll, old, adv, ref_nll=ref.cpu()),
                lambda: head.policy_loss(nll, old, adv, lengths=n.long()),
                lambda: head.policy_loss(nll, old, adv, lengths=n[:1]),
                lambda: head.policy_loss(nll, old, adv, reduction="all"),
                lambda: head.policy_loss(nll, old, adv, grad=torch.ones(4, 3, 20, device="cuda")),
                lambda: head.policy_loss(nll, old, adv, reduction="none", grad=one),
                lambda: head.policy_loss(nll, old, adv, workspace=small),
                lambda: head.preference_loss(nll[0], c, r), lambda: head.preference_loss(nll, c.long(), r),
                lambda: head.preference_loss(nll, c[:1], r), lambda: head.preference_loss(nll, None, r),
                lambda: head.preference_loss(nll, c, r, reduction="sequence_mean"),
                lambda: head.preference_loss(nll, c, r, grad=torch.ones(4, device="cuda")),
                lambda: head.preference_loss(nll, c, r, ref_nll=ref[:1]),
                lambda: head.preference_loss(nll, c, r, workspace=small)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: head.policy_loss(nll, old, adv, clip_low=-0.1), lambda: head.policy_loss(nll, old, adv, clip_high=float("nan")),
                lambda: head.policy_loss(nll, old, adv, kl_weight=float("inf")),
                lambda: head.preference_loss(nll, c, r, label_smoothing=1.5),
                lambda: head.preference_loss(nll, c, r, beta=float("nan"))):
        with pytest.raises(D.CtcpbError):
            bad()
