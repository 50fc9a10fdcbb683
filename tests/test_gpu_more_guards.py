"""Guard margins around every buffer of the C calls around the label head (group norm,
dropout, policy and preference losses), strided outputs, gradients left out, and what
the calls do with workspaces: two on different streams, one after the other's use."""
import pytest
import torch

from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

G, PAT = 1 << 16, 0xA5
TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


class Guarded:
    def __init__(self, nbytes):
        self.n = int(nbytes)
        self.buf = torch.full((self.n + 2 * G,), PAT, dtype=torch.uint8, device="cuda")
        self.view = self.buf[G:G + self.n]

    def typed(self, dtype, *shape):
        return self.view.view(dtype).view(shape)

    def ptr(self):
        return self.view.data_ptr() if self.n else None

    def intact(self):
        return bool((self.buf[:G] == PAT).all()) and bool((self.buf[G + self.n:] == PAT).all())


def stream():
    return torch.cuda.current_stream().cuda_stream


# one block, several, a cluster, two launches, single elements, a group wider than a block, many utterances
@pytest.mark.parametrize("B,T,C,groups,pad", [(1, 7, 64, 8, 0), (5, 37, 96, 4, 8), (3, 700, 512, 32, 0), (1, 30000, 64, 1, 16),
                                              (2, 53, 33, 3, 3), (1, 6, 8192, 1, 0), (900, 3, 24, 3, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_group_norm_writes(B, T, C, groups, pad, dtype):
    g = torch.Generator(device="cuda").manual_seed(B + T + C)
    x = torch.randn(B, T, C, generator=g, device="cuda").to(dtype)
    dy = torch.randn(B, T, C, generator=g, device="cuda").to(dtype)
    w, b = torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")
    n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    e, L, row = x.element_size(), head._lib(), C + pad
    y, mean, rstd = Guarded(e * B * T * row), Guarded(4 * B * groups), Guarded(4 * B * groups)
    ws = Guarded(head.group_norm_workspace_size(dtype, B, T, C, groups, False))
    assert L["ctcpb_group_norm"](TYPE[dtype], 0, x.data_ptr(), T * C, C, w.data_ptr(), b.data_ptr(), n.data_ptr(), 1e-5, 2, B,
                                 T, C, groups, y.ptr(), T * row, row, mean.ptr(), rstd.ptr(), ws.ptr(), ws.n, stream()) == D.OK
    torch.cuda.synchronize()
    assert y.intact() and mean.intact() and rstd.intact() and ws.intact()
    wy, wm, wr = head.group_norm(x, groups, w, b, lengths=n, activation="silu")
    got = y.typed(dtype, B, T, row)
    assert torch.allclose(got[..., :C].float(), wy.float(), rtol=2 * torch.finfo(dtype).eps, atol=1e-6)  # another split of sums
    assert (y.view.view(B * T, e * row)[:, e * C:] == PAT).all()
    assert pad or torch.equal(got, wy) and torch.equal(mean.typed(torch.float32, B, groups), wm)
    want = head.group_norm_backward(dy, x, groups, w, b, wm, wr, lengths=n, activation="silu")
    for dx_on, dw_on, db_on in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        dx, dw, db = Guarded(e * B * T * C), Guarded(4 * C), Guarded(4 * C)
        ws = Guarded(head.group_norm_workspace_size(dtype, B, T, C, groups, True))
        assert L["ctcpb_group_norm_backward"](
            TYPE[dtype], 0, dy.data_ptr(), T * C, C, x.data_ptr(), T * C, C, w.data_ptr(), b.data_ptr(), n.data_ptr(),
            wm.data_ptr(), wr.data_ptr(), 2, B, T, C, groups, dx.ptr() if dx_on else None, T * C, C, dw.ptr() if dw_on else None,
            db.ptr() if db_on else None, ws.ptr(), ws.n, stream()) == D.OK
        torch.cuda.synchronize()
        assert dx.intact() and dw.intact() and db.intact() and ws.intact()
        for on, buf, dt, ref in ((dx_on, dx, dtype, want[0]), (dw_on, dw, torch.float32, want[1]),
                                 (db_on, db, torch.float32, want[2])):
            if on:
                assert torch.equal(buf.typed(dt, *ref.shape), ref)
            else:
                assert (buf.view == PAT).all()


@pytest.mark.parametrize("n,h", [(1, 1), (3, 13), (130, 64), (33, 769), (1, 8192), (700, 1024)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropout_writes(n, h, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + h)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    rng = torch.tensor([7, 9], dtype=torch.int64, device="cuda")
    e = x.element_size()
    for pad in (0, 8):
        y = Guarded(e * n * (h + pad))
        assert head._lib()["ctcpb_dropout"](TYPE[dtype], x.data_ptr(), h, None, 0, 0.3, rng.data_ptr(), n, h, y.ptr(), h + pad,
                                            stream()) == D.OK
        torch.cuda.synchronize()
        assert y.intact() and rng.tolist() == [7, 9]
        assert torch.equal(y.typed(dtype, n, h + pad)[:, :h], head.dropout(x, 0.3, rng))
        assert (y.view.view(n, e * (h + pad))[:, e * h:] == PAT).all()


@pytest.mark.parametrize("S,L", [(1, 1), (7, 13), (320, 40), (3, 4099), (2000, 64), (9000, 12)])
@pytest.mark.parametrize("reduction", [0, 1, 3])
def test_policy_writes(S, L, reduction):
    g = torch.Generator(device="cuda").manual_seed(S + L)
    nll, old, ref = (torch.rand(S, L, generator=g, device="cuda") for _ in range(3))
    adv = torch.randn(S, generator=g, device="cuda")
    n = torch.randint(0, L + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = L
    name = {0: "none", 1: "mean", 3: "sequence_mean"}[reduction]
    grad = torch.ones(S, L, device="cuda") if reduction == 0 else torch.ones((), device="cuda")
    want = head.policy_loss(nll, old, adv, lengths=n, ref_nll=ref, kl_weight=0.1, reduction=name, grad=grad)
    for loss_on, stats_on, dnll_on in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        loss, stats, dnll = Guarded(4 * S * L if reduction == 0 else 4), Guarded(8), Guarded(4 * S * L)
        ws = Guarded(head.policy_loss_workspace_size(S, L))
        assert head._lib()["ctcpb_policy_loss"](
            nll.data_ptr(), L, old.data_ptr(), L, ref.data_ptr(), L, adv.data_ptr(), 0, n.data_ptr(), S, L, 0.2, 0.2, 0.1,
            reduction, grad.data_ptr() if dnll_on else None, loss.ptr() if loss_on else None, stats.ptr() if stats_on else None,
            dnll.ptr() if dnll_on else None, ws.ptr(), ws.n, stream()) == D.OK
        torch.cuda.synchronize()
        assert loss.intact() and stats.intact() and dnll.intact() and ws.intact() and D.read_status(ws.view) == 0
        for on, buf, ref_out in ((loss_on, loss, want[0]), (stats_on, stats, want[1]), (dnll_on, dnll, want[2])):
            assert torch.equal(buf.typed(torch.float32, *ref_out.shape), ref_out) if on else (buf.view == PAT).all()


@pytest.mark.parametrize("B,N,L", [(1, 1, 1), (7, 3, 13), (32, 10, 40), (3, 2, 4099), (2000, 4, 64), (9000, 2, 4)])
@pytest.mark.parametrize("reduction", [0, 1])
def test_preference_writes(B, N, L, reduction):
    g = torch.Generator(device="cuda").manual_seed(B + N + L)
    nll, ref = (torch.rand(B, N, L, generator=g, device="cuda") for _ in range(2))
    c, r = (torch.randint(-1, N, (B,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2))
    n = torch.randint(0, L + 1, (B, N), generator=g, device="cuda", dtype=torch.int32)
    c[0] = r[0] = 0
    name = {0: "none", 1: "mean"}[reduction]
    grad = torch.ones(B, device="cuda") if reduction == 0 else torch.ones((), device="cuda")
    want = head.preference_loss(nll, c, r, lengths=n, ref_nll=ref, reduction=name, grad=grad)
    for loss_on, margins_on, dnll_on in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        loss, margins, dnll = Guarded(4 * B if reduction == 0 else 4), Guarded(4 * B), Guarded(4 * B * N * L)
        ws = Guarded(head.preference_loss_workspace_size(B, N, L))
        assert head._lib()["ctcpb_preference_loss"](
            nll.data_ptr(), L, ref.data_ptr(), L, c.data_ptr(), r.data_ptr(), n.data_ptr(), B, N, L, 0.1, 0.0, 0.0, 0, reduction,
            grad.data_ptr() if dnll_on else None, loss.ptr() if loss_on else None, margins.ptr() if margins_on else None,
            dnll.ptr() if dnll_on else None, ws.ptr(), ws.n, stream()) == D.OK
        torch.cuda.synchronize()
        assert loss.intact() and margins.intact() and dnll.intact() and ws.intact() and D.read_status(ws.view) == 0
        for on, buf, ref_out in ((loss_on, loss, want[0]), (margins_on, margins, want[1]), (dnll_on, dnll, want[2])):
            assert torch.equal(buf.typed(torch.float32, *ref_out.shape), ref_out) if on else (buf.view == PAT).all()


def test_two_streams_at_once():
    """Calls of every kind on two streams, each with workspaces of its own, give the bits of the plain calls."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(6, 9000, 64, generator=g, device="cuda").bfloat16()
    w = torch.randn(64, generator=g, device="cuda")
    nll, old, ref = (torch.rand(700, 300, generator=g, device="cuda") for _ in range(3))
    adv, one = torch.randn(700, generator=g, device="cuda"), torch.ones((), device="cuda")
    c, r = (torch.randint(0, 7, (100,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2))

    def calls(k):
        y, mean, rstd = head.group_norm(x * k, 1, w, w, activation="silu")
        grads = head.group_norm_backward(x, x * k, 1, w, w, mean, rstd, activation="silu")
        return (y, *grads, *head.policy_loss(nll * k, old, adv, ref_nll=ref, kl_weight=0.1, grad=one),
                *head.preference_loss(nll.view(100, 7, 300) * k, c, r, grad=one))

    want = [calls(1), calls(2)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(s[i]):
                got[i].append(calls(i + 1))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


def test_a_workspace_used_again():
    """One workspace for calls of different kinds and sizes, one after the other."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(2, 20000, 64, generator=g, device="cuda").bfloat16()
    nll = torch.rand(3000, 40, generator=g, device="cuda")
    adv, one = torch.randn(3000, generator=g, device="cuda"), torch.ones((), device="cuda")
    size = max(head.group_norm_workspace_size(x.dtype, 2, 20000, 64, 1, True), head.policy_loss_workspace_size(3000, 40))
    ws = torch.full((size,), PAT, dtype=torch.uint8, device="cuda")
    y, mean, rstd = head.group_norm(x, 1)
    want = head.group_norm_backward(x, x, 1, None, None, mean, rstd), head.policy_loss(nll, nll, adv, grad=one)
    for _ in range(3):
        a = head.group_norm_backward(x, x, 1, None, None, mean, rstd, workspace=ws)
        b = head.policy_loss(nll, nll, adv, grad=one, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip((*a, *b), (*want[0], *want[1])))
