"""Log-probabilities and cross entropy of the label head against plain
definitions in 64 bits (head_ref): types, odd and single sizes, strides and
offsets, ignored and invalid targets, labels taken out, large losses, pieces of
the vocabulary, another stream."""
import pytest
import torch

import head_ref as R
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def inputs(n, v, h, dtype, bias=F32, seed=0, ignore=0.2):
    g = gen(seed * 1000 + n * 7 + v * 3 + h)
    w = torch.randn(v, h, generator=g, device="cuda") * 1.5 / h ** 0.5
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    x = torch.randn(n, h, generator=g, device="cuda") + 2.0 * w[t]
    t = torch.where(torch.rand(n, generator=g, device="cuda") < ignore, torch.full_like(t, -1), t).int()
    b = None if bias is None else (torch.randn(v, generator=g, device="cuda") * 0.5).to(bias)
    return x.to(dtype), w.to(dtype), b, t


def assert_within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    ok = torch.isfinite(want)
    over = ((got - want).abs() - bound)[ok]
    assert over.numel() == 0 or over.max().item() <= 0, \
        f"{what}: {(over > 0).sum().item()} of {over.numel()} beyond the bound, by up to {over.max().item():.3g}"


def check_log_probs(x, w, b, got):
    z = R.logits(x, w, b)
    lse = torch.logsumexp(z, 1, keepdim=True)
    e = R.logits_bound(x, w, b)
    bound = e + e.max(1, keepdim=True).values + R.exp_log_bound(z, lse) + 2.0 ** -24 * (z - lse).abs()
    assert got.dtype == torch.float32
    assert_within(got, z - lse, bound, "log_prob")


SIZES = [(1, 1, 1), (1, 29, 64), (3, 33, 17), (128, 5000, 512), (129, 257, 64), (127, 256, 200), (300, 1000, 769),
         (2048, 129, 96), (1, 70001, 40), (500, 64, 2048), (4097, 32, 8), (40, 31, 8192)]


@pytest.mark.parametrize("n,v,h", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_log_probs(n, v, h, dtype):
    x, w, b, _ = inputs(n, v, h, dtype, F32 if (n + v) % 2 else dtype)
    ws = torch.empty(head.log_probs_workspace_size(dtype, n, v, h), dtype=torch.uint8, device="cuda")
    got = head.log_probs(x, w, b, workspace=ws)
    check_log_probs(x, w, b, got)
    assert D.read_status(ws) == 0


def test_log_probs_without_bias_of_a_batch():
    x, w, _, _ = inputs(6 * 50, 500, 128, BF, None)
    got = head.log_probs(x.view(6, 50, 128), w)
    assert got.shape == (6, 50, 500)
    check_log_probs(x, w, None, got.view(300, 500))


def test_log_probs_strides_and_offsets():
    """Rows of a wider tensor, rows off 16-byte boundaries, padded output rows."""
    x, w, b, _ = inputs(200, 301, 96, BF)
    want = head.log_probs(x, w, b)
    wide = torch.zeros(200, 160, dtype=BF, device="cuda")
    wide[:, 16:112] = x
    odd = torch.zeros(200, 99, dtype=BF, device="cuda")
    odd[:, 1:97] = x
    ww = torch.zeros(301, 101, dtype=BF, device="cuda")
    ww[:, 3:99] = w
    for xi in (wide[:, 16:112], odd[:, 1:97]):
        for wi in (w, ww[:, 3:99]):
            assert torch.equal(head.log_probs(xi, wi, b), want)
    pad = torch.full((200, 304), 7.0, device="cuda")
    got = head.log_probs(x, w, b, out=pad[:, :301])
    assert torch.equal(got, want) and (pad[:, 301:] == 7.0).all()
    off = torch.full((200 * 303 + 1,), 7.0, device="cuda")[1:].view(200, 303)
    got = head.log_probs(x, w, b, out=off[:, :301])
    assert torch.equal(got, want) and (off[:, 301:] == 7.0).all()


def test_what_lies_past_a_row_is_not_read():
    """Rows on 16-byte boundaries whose width is no multiple of 16 bytes: the
    next elements, NaN here, take no part; and outputs end where they should."""
    x, w, b, t = inputs(200, 301, 93, BF)
    want = head.log_probs(x, w, b)
    wx = torch.full((200, 160), float("nan"), dtype=BF, device="cuda")
    wx[:, :93] = x
    ww = torch.full((301, 96), float("nan"), dtype=BF, device="cuda")
    ww[:, :93] = w
    pad = torch.full((200, 304), 7.0, device="cuda")
    assert torch.equal(head.log_probs(wx[:, :93], ww[:, :93], b, out=pad[:, :301]), want) and (pad[:, 301:] == 7.0).all()
    loss, lse = head.cross_entropy(x, w, t, b)
    loss2, lse2 = head.cross_entropy(wx[:, :93], ww[:, :93], t, b)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    one = torch.ones((), device="cuda")
    for p, q in zip(head.cross_entropy_backward(one, x, w, t, lse, b),
                    head.cross_entropy_backward(one, wx[:, :93], ww[:, :93], t, lse, b)):
        assert torch.equal(p, q)


def test_log_probs_labels_taken_out_and_special_values():
    x, w, b, _ = inputs(140, 300, 64, BF)
    b[::3] = -float("inf")
    got = head.log_probs(x, w, b)
    check_log_probs(x, w, b, got)
    assert (got[:, ::3] == -float("inf")).all()
    # a row whose labels are all out is NaN; a row with a NaN feature stays alone
    none = torch.full_like(b, -float("inf"))
    assert torch.isnan(head.log_probs(x, w, none)).all()
    x2 = x.clone()
    x2[5, 3] = float("nan")
    got2 = head.log_probs(x2, w, b)
    keep = torch.arange(140, device="cuda") != 5
    assert torch.isnan(got2[5]).any() and torch.equal(got2[keep], got[keep])


def test_log_probs_of_far_apart_logits():
    """Logits hundreds apart: the sum must not overflow or lose the largest."""
    x, w, b, _ = inputs(64, 200, 64, BF)
    b = b + torch.linspace(-4e4, 4e4, 200, device="cuda")
    check_log_probs(x, w, b, head.log_probs(x, w, b))


def check_cross_entropy(x, w, b, t, reduction="mean", ignore=-1, grad=None, ws=None):
    n, h = x.shape
    v = w.shape[0]
    dt = x.dtype
    if grad is None:
        grad = torch.full((), 1024.0 if dt == HF else 1.0, device="cuda")
    loss, lse = head.cross_entropy(x, w, t, b, ignore_index=ignore, reduction=reduction)
    dx, dw, db = head.cross_entropy_backward(grad, x, w, t, lse, b, ignore_index=ignore, reduction=reduction,
                                             workspace=ws)
    rl, rlse, rdx, rdw, rdb, bx, bw, bb = R.cross_entropy(x, w, b, t, ignore, reduction, grad)
    keep = (t != ignore) & (t >= 0) & (t < v)
    xk = torch.where(keep[:, None], x, torch.zeros_like(x))
    e = R.logits_bound(xk, w, b).max(1).values if n else torch.zeros(0, device="cuda").double()
    z = R.logits(xk, w, b)
    el = torch.where(keep, e + R.exp_log_bound(z, rlse), torch.zeros_like(rlse))
    assert_within(lse, rlse, el, "lse")
    row = el + e + 2.0 ** -23 * rlse.abs()
    k = max(int(keep.sum()), 1)
    fold = row if reduction == "none" else row.sum() / (k if reduction == "mean" else 1)
    assert_within(loss, rl, fold + 4 * 2.0 ** -24 * rl.abs().nan_to_num(), "loss")
    # d is rounded to 16 bits, its exponential carries the logits' errors
    # relatively; then the sums (float32) and the rounding of the result.
    # float16: d is kept at 2^15 of the largest, so what is lost below its
    # range is 2^-24 / 2^15 of that for each term of a sum.
    u, rel = R.U[dt], float((2 * el.max() + 2.0 ** -18).item()) if n else 0.0
    gm = grad.abs().max().double() / (k if reduction == "mean" else 1) if grad.numel() else torch.zeros(()).cuda().double()
    lost = 2.0 ** -39 * gm if dt == HF else 0.0
    assert_within(dx, rdx, (u + rel) * bx + u * rdx.abs() + lost * w.double().abs().sum(0)[None] + R.TINY[dt], "dx")
    assert_within(dw, rdw, (u + rel) * bw + u * rdw.abs() + lost * xk.double().abs().sum(0)[None] + R.TINY[dt], "dw")
    assert dx.dtype == dw.dtype == dt
    if b is not None:
        assert db.dtype == b.dtype
        assert_within(db, rdb, (rel + 2.0 ** -20) * bb + R.U[b.dtype] * rdb.abs() + R.TINY[b.dtype], "db")
    else:
        assert db is None
    assert (dx[~keep] == 0).all()
    return loss, lse, dx, dw, db


@pytest.mark.parametrize("n,v,h", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cross_entropy(n, v, h, dtype):
    x, w, b, t = inputs(n, v, h, dtype, F32 if (n + v) % 2 else dtype)
    if n == 1:
        t = torch.zeros_like(t)
    check_cross_entropy(x, w, b, t)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("bias", [None, F32])
def test_cross_entropy_reductions(reduction, dtype, bias):
    x, w, b, t = inputs(333, 700, 128, dtype, bias)
    grad = torch.randn(333, generator=gen(5), device="cuda") * 3 if reduction == "none" else \
        torch.full((), -0.7 if reduction == "sum" else 300.0, device="cuda")
    check_cross_entropy(x, w, b, t, reduction, grad=grad)


def test_cross_entropy_of_many_rows_and_of_a_long_depth():
    """Several tiles of rows, work shared along K in both products."""
    x, w, b, t = inputs(3000, 2000, 320, BF)
    check_cross_entropy(x, w, b, t)
    x, w, b, t = inputs(150, 40000, 64, BF, BF)
    check_cross_entropy(x, w, b, t, "sum")


def test_cross_entropy_in_pieces_of_the_vocabulary():
    """d of 20,000 rows x 15,001 labels takes three pieces."""
    x, w, b, t = inputs(20000, 15001, 72, BF, F32, ignore=0.0)
    check_cross_entropy(x, w, b, t)


def test_ignored_rows_take_no_part():
    """Padding may hold anything: NaN and infinities of ignored rows reach no sum."""
    x, w, b, t = inputs(500, 300, 128, BF, ignore=0.3)
    want = check_cross_entropy(x, w, b, t)
    x2 = x.clone()
    x2[t == -1] = float("nan")
    x2[int((t == -1).nonzero()[0])] = float("inf")
    loss, lse = head.cross_entropy(x2, w, t, b)
    got = (loss, lse, *head.cross_entropy_backward(torch.ones((), device="cuda"), x2, w, t, lse, b))
    for a, c in zip(got, want):
        assert torch.equal(a, c)
    assert (lse[t == -1] == 0).all()


def test_every_row_ignored():
    x, w, b, t = inputs(70, 90, 64, BF)
    t = torch.full_like(t, 11)
    one = torch.ones((), device="cuda")
    for red in ("mean", "sum"):
        loss, lse = head.cross_entropy(x, w, t, b, ignore_index=11, reduction=red)
        assert torch.isnan(loss) if red == "mean" else loss.item() == 0.0
        for g in head.cross_entropy_backward(one, x, w, t, lse, b, ignore_index=11, reduction=red):
            assert (g == 0).all()
    loss, lse = head.cross_entropy(x, w, t, b, ignore_index=11, reduction="none")
    assert (loss == 0).all() and (lse == 0).all()


def test_no_rows():
    x, w, b, t = inputs(4, 50, 64, BF)
    x, t = x[:0], t[:0]
    assert head.log_probs(x, w, b).shape == (0, 50)
    assert torch.isnan(head.cross_entropy(x, w, t, b)[0])
    loss, lse = head.cross_entropy(x, w, t, b, reduction="sum")
    assert loss.item() == 0.0 and lse.shape == (0,)
    dx, dw, db = head.cross_entropy_backward(torch.ones((), device="cuda"), x, w, t, lse, b)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    assert head.cross_entropy(x, w, t, b, reduction="none")[0].shape == (0,)


def test_targets_out_of_range_are_ignored_and_reported():
    x, w, b, t = inputs(300, 200, 64, BF, ignore=0.1)
    ws = torch.empty(head.cross_entropy_workspace_size(BF, 300, 200, 64, False), dtype=torch.uint8, device="cuda")
    head.cross_entropy(x, w, t, b, workspace=ws)
    assert D.read_status(ws) == 0
    t2 = t.clone()
    t2[7], t2[290] = 200, -5
    loss, lse = head.cross_entropy(x, w, t2, b, workspace=ws)
    assert D.read_status(ws) == head.DEV_TARGET
    t3 = t.clone()
    t3[7] = t3[290] = -1
    want, _ = head.cross_entropy(x, w, t3, b, workspace=ws)
    assert loss.item() == want.item() and D.read_status(ws) == 0
    # a label may itself be the ignored one
    check_cross_entropy(x, w, b, t.clamp(min=0), ignore=0)


def test_a_target_label_taken_out():
    """A label of bias -inf has an infinite loss, and the others' gradients are finite."""
    x, w, b, t = inputs(130, 100, 64, BF, ignore=0.0)
    b[7] = -float("inf")
    t[t == 7] = 8
    check_cross_entropy(x, w, b, t)
    t[3] = 7
    loss, _ = head.cross_entropy(x, w, t, b, reduction="none")
    assert loss[3].item() == float("inf") and torch.isfinite(loss[torch.arange(130, device="cuda") != 3]).all()


def test_strided_operands():
    x, w, b, t = inputs(260, 190, 104, HF)
    want = check_cross_entropy(x, w, b, t)
    odd = torch.zeros(260, 107, dtype=HF, device="cuda")
    odd[:, 2:106] = x
    ww = torch.zeros(190, 109, dtype=HF, device="cuda")
    ww[:, 5:109] = w
    loss, lse = head.cross_entropy(odd[:, 2:106], ww[:, 5:109], t, b)
    got = (loss, lse, *head.cross_entropy_backward(torch.full((), 1024.0, device="cuda"), odd[:, 2:106], ww[:, 5:109],
                                                   t, lse, b))
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_same_bits_again_and_on_another_stream():
    x, w, b, t = inputs(1500, 3001, 256, BF)
    one = torch.ones((), device="cuda")

    def step():
        loss, lse = head.cross_entropy(x, w, t, b)
        return (head.log_probs(x, w, b), loss, lse, *head.cross_entropy_backward(one, x, w, t, lse, b))

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [step() for _ in range(3)]
    s.synchronize()
    for g in got:
        for a, c in zip(g, want):
            assert torch.equal(a, c)


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the 64-bit loss."""
    x, w, b, t = inputs(64, 50, 32, BF)
    loss, lse = head.cross_entropy(x, w, t, b)
    grads = head.cross_entropy_backward(torch.ones((), device="cuda"), x, w, t, lse, b)
    args = [x.double(), w.double(), b.double()]
    one = torch.ones((), device="cuda")
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=gen(i), device="cuda").double()
        step = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + step * d, args[i] - step * d
        diff = (R.cross_entropy(*up, t, -1, "mean", one)[0] - R.cross_entropy(*dn, t, -1, "mean", one)[0]) / (2 * step)
        # both roundings to 16 bits, over a sum of terms of either sign
        tol = 2 * R.U[BF] * (g.double().abs() * d.abs()).sum()
        assert abs((g.double() * d).sum() - diff) <= tol


def test_large_offsets():
    """log_prob past 2^31 elements: the last rows are right."""
    n, v, h = 70000, 32768, 16
    g = gen(1)
    x = torch.randn(n, h, generator=g, device="cuda").to(BF)
    w = torch.randn(v, h, generator=g, device="cuda").to(BF)
    got = head.log_probs(x, w)
    for r in (0, 65535, 69990):
        check_log_probs(x[r:r + 10], w, None, got[r:r + 10])


def test_decoder_reads_the_head():
    """log_probs into padded rows, decoded as it is: the same as decoding a contiguous copy."""
    x, w, b, _ = inputs(4 * 60, 29, 64, BF)
    pad = torch.empty(4, 60, 32, device="cuda")
    lp = head.log_probs(x.view(4, 60, 64), w, b, out=pad[..., :29])
    cfg = D.Config(beam=8, nbest=3)
    a, c = D.decode_offline(cfg, lp), D.decode_offline(cfg, lp.contiguous())
    for u, v in zip(a, c):
        assert torch.equal(u, v)


def test_refusals():
    x, w, b, t = inputs(10, 20, 64, BF)
    for bad in (lambda: head.log_probs(x.float(), w.float(), b),
                lambda: head.cross_entropy(x.float(), w.float(), t, b)):
        with pytest.raises(D.CtcpbError) as e:
            bad()
        assert e.value.code == D.EINVAL
    lse = torch.zeros(10, device="cuda")
    one = torch.ones((), device="cuda")
    for bad in (lambda: head.log_probs(x.cpu(), w, b), lambda: head.log_probs(x, w.half(), b),
                lambda: head.log_probs(x, w[:, :32], b), lambda: head.log_probs(x, w, b[:5]),
                lambda: head.log_probs(x, w, b.half()),
                lambda: head.log_probs(x, w, b, out=torch.empty(10, 21, device="cuda")),
                lambda: head.log_probs(x, w, b, out=torch.empty(20, 10, device="cuda").t()),
                lambda: head.log_probs(x, w, b, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                lambda: head.cross_entropy(x, w, t.long(), b), lambda: head.cross_entropy(x, w, t[:5], b),
                lambda: head.cross_entropy(x, w, t, b, reduction="max"),
                lambda: head.cross_entropy_backward(one, x, w, t, lse[:4], b),
                lambda: head.cross_entropy_backward(lse, x, w, t, lse, b),
                lambda: head.cross_entropy_backward(one.double(), x, w, t, lse, b)):
        with pytest.raises(ValueError):
            bad()
    L, big = head._lib(), 1 << 40
    p = x.data_ptr() // 256 * 256
    f = L["ctcpb_log_probs"]
    assert f(1, 0, p, 64, p, 64, None, 10, 20, 64, p, 20, p + 16, big, None) == D.EALIGN
    assert f(1, 0, p, 64, p, 64, None, 10, 20, 64, p, 20, p, 16, None) == D.ESIZE
    assert f(1, 0, p, 63, p, 64, None, 10, 20, 64, p, 20, p, big, None) == D.EINVAL
    assert f(1, 0, p, 64, p, 64, None, 10, 20, 64, p, 19, p, big, None) == D.EINVAL
    assert f(1, 0, None, 64, p, 64, None, 10, 20, 64, p, 20, p, big, None) == D.ENULL
    assert f(1, 2, p, 64, p, 64, p, 10, 20, 64, p, 20, p, big, None) == D.EINVAL
    assert f(1, 0, p, 8193, p, 8193, None, 10, 20, 8193, p, 20, p, big, None) == D.EINVAL
