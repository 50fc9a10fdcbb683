"""Group norm with an activation, and its backward pass, against definitions in 64
bits (more_ref), at the widths, lengths and strides where they can go wrong."""
import pytest
import torch

import more_ref as R
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def inputs(B, T, C, dtype, params, ragged=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 100 + B * 7 + T * 3 + C)
    x = torch.randn(B, T, C, generator=g, device="cuda") * 1.5 + torch.randn(B, 1, C, generator=g, device="cuda")
    w = 1 + 0.3 * torch.randn(C, generator=g, device="cuda")
    b = 0.2 * torch.randn(C, generator=g, device="cuda")
    dy = torch.randn(B, T, C, generator=g, device="cuda")
    n = torch.randint(T // 2, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    return x.to(dtype), w.to(params), b.to(params), dy.to(dtype), n


def within(got, want, bound, dtype, what):
    bad = ~((got.double() - want).abs() <= R.rounded(bound, want, dtype))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           (got.double() - want).abs()[bad][:3].tolist(), bound.expand(bad.shape)[bad][:3].tolist())


def check(x, w, b, dy, n, G, act, ws=None, ref_x=None):
    """``ref_x``: x with what lies behind the lengths made harmless."""
    r = R.GroupNorm(x if ref_x is None else ref_x, G, w, b, n, EPS, act)
    y, mean, rstd = head.group_norm(x, G, w, b, lengths=n, eps=EPS, activation=act)
    some = r.n > 0
    m, e_m = r.mean[:, 0, :, 0], r.e_mean[:, 0, :, 0]
    assert ((mean.double() - m).abs() <= e_m + 2 * R.u * m.abs()).all()
    assert ((rstd.double() / r.r[:, 0, :, 0] - 1).abs() <= r.e_r[:, 0, :, 0])[some].all()
    assert (mean[~some] == 0).all() and (rstd[~some] == 0).all()
    within(y, r.flat(r.y), r.flat(r.e_y), x.dtype, "y")
    got = head.group_norm_backward(dy, x, G, w, b, mean, rstd, lengths=n, activation=act, workspace=ws)
    clean = torch.where(R.frames(x, n)[1][..., None], dy, torch.zeros((), dtype=dy.dtype, device="cuda"))
    want, bounds = r.backward(clean)
    for g, v, e, t, what in zip(got, want, bounds, (x.dtype, got[1].dtype, got[2].dtype), ("dx", "dweight", "dbias")):
        within(g, v, e, t, what)
    live = R.frames(x, n)[1]
    assert (y[~live] == 0).all() and (got[0][~live] == 0).all()
    return y, mean, rstd, *got


# widths of a group: whole 16-byte vectors, 8 and 4 bytes, single elements, one group, a group for each channel;
# wider than a block takes at once; lengths of one, of no whole block's rows, of a cluster, of more than it holds
SHAPES = [(1, 1, 8, 1), (3, 1, 512, 32), (2, 2, 6, 3), (1, 50, 64, 8), (5, 37, 96, 4), (4, 33, 40, 10), (3, 65, 36, 6),
          (2, 129, 771, 3), (7, 20, 33, 33), (2, 300, 512, 32), (3, 500, 1024, 32), (2, 77, 2048, 1), (2, 19, 4098, 1),
          (2, 9, 8192, 1), (1, 5, 8191, 1), (2, 4000, 64, 2), (1, 20000, 24, 3), (300, 8, 16, 2), (2, 3000, 7, 1),
          (1, 40000, 64, 1), (3, 5000, 771, 1), (2, 9000, 260, 2)]


@pytest.mark.parametrize("B,T,C,G", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_group_norm(B, T, C, G, dtype):
    i = B + T + C
    x, w, b, dy, n = inputs(B, T, C, dtype, F32 if i % 2 else dtype, ragged=i % 3 != 0)
    check(x, w, b, dy, n, G, ("silu", "relu", "none")[i % 3] if dtype != BF else "silu")


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_activations(act):
    check(*inputs(3, 40, 64, F32, F32), 4, act)


def test_without_parameters():
    x, w, b, dy, n = inputs(3, 40, 96, BF, BF)
    check(x, None, None, dy, n, 6, "silu")
    check(x, w, None, dy, n, 6, "silu")
    check(x, None, b, dy, n, 6, "relu")
    y, mean, rstd = head.group_norm(x, 6)
    assert head.group_norm_backward(dy, x, 6, None, None, mean, rstd, param_dtype=F32)[1].dtype == F32


def test_lengths():
    """None, one, all, and what is out of range (clamped); what lies behind them is not read."""
    x, w, b, dy, _ = inputs(6, 70, 64, F32, F32, ragged=False)
    n = torch.tensor([0, 1, 70, 35, -5, 1000], dtype=torch.int32, device="cuda")
    want = check(x, w, b, dy, n, 8, "silu")
    bad, bad_dy = x.clone(), dy.clone()
    dead = ~R.frames(x, n)[1]
    for v in (float("nan"), float("inf"), torch.finfo(F32).min):
        bad[dead], bad_dy[dead] = v, v
        got = check(bad, w, b, bad_dy, n, 8, "silu", ref_x=x)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
    none = torch.zeros(6, dtype=torch.int32, device="cuda")
    y, mean, rstd, dx, dw, db = check(x, w, b, dy, none, 8, "silu")
    assert (y == 0).all() and (dw == 0).all() and (db == 0).all()


def test_special_values_stay_in_their_groups():
    x, w, b, dy, n = inputs(4, 30, 64, BF, F32, ragged=False)
    want = head.group_norm(x, 4, w, b, activation="silu")[0]
    x[1, 7, 20], x[3, 0, 63] = float("nan"), float("inf")
    got = head.group_norm(x, 4, w, b, activation="silu")[0].view(4, 30, 4, 16)
    keep = torch.ones(4, 30, 4, 16, dtype=torch.bool, device="cuda")
    keep[1, :, 1] = keep[3, :, 3] = False
    assert torch.equal(got[keep], want.view(4, 30, 4, 16)[keep]) and torch.isnan(got[~keep]).all()


def test_constant_and_offset_groups():
    """A constant group has variance 0; a large common offset does not eat the differences."""
    x, w, b, dy, n = inputs(3, 50, 64, F32, F32, ragged=False)
    x[0, :, :16] = 5.0
    x[1] += 1000.0
    x[2, 0] = 300.0  # one frame far from the others
    y, mean, rstd, *_ = check(x, w, b, dy, n, 4, "none")
    assert torch.equal(y[0, :, :16], b[:16].expand(50, 16))
    assert abs(rstd[0, 0].item() * EPS ** 0.5 - 1) < 1e-6


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides(dtype):
    x, w, b, dy, n = inputs(4, 60, 72, dtype, F32)
    want = check(x, w, b, dy, n, 9, "silu")
    wide = torch.full((4, 70, 200), float("nan"), dtype=dtype, device="cuda")
    for off in (8, 13):  # rows on 16-byte boundaries, and on none
        wide[:, :60, off:off + 72] = x
        wide[:, :60, 100 + off:172 + off] = dy
        got = check(wide[:, :60, off:off + 72], w, b, wide[:, :60, 100 + off:172 + off], n, 9, "silu")
        for p, q in zip(got, want):
            assert p.shape == q.shape
    # time first, and channels that are not contiguous (copied)
    got = check(x.transpose(0, 1).contiguous().transpose(0, 1), w, b, dy, n, 9, "silu")
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    got = check(x.transpose(1, 2).contiguous().transpose(1, 2), w, b, dy.transpose(1, 2).contiguous().transpose(1, 2), n, 9,
                "silu")
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    # one utterance for all of a batch
    check(x[:1].expand(4, 60, 72), w, b, dy, n, 9, "silu")


def test_offsets_past_32_bits():
    x, w, b, dy, _ = inputs(2, 40, 64, BF, F32, ragged=False)
    far = torch.zeros((1 << 31) + 64 + 40 * 64, dtype=BF, device="cuda")
    view = far.as_strided((2, 40, 64), ((1 << 31) + 64, 64, 1))
    view.copy_(x)
    want = head.group_norm(x, 8, w, b, activation="silu")
    got = head.group_norm(view, 8, w, b, activation="silu")
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for p, q in zip(head.group_norm_backward(dy, view, 8, w, b, *want[1:], activation="silu"),
                    head.group_norm_backward(dy, x, 8, w, b, *want[1:], activation="silu")):
        assert torch.equal(p, q)
    # rows far apart
    tall = far[:(39 * 50000000 + 64)].as_strided((1, 40, 64), (0, 50000000, 1))
    tall.copy_(x[:1])
    assert torch.equal(head.group_norm(tall, 8, w, b)[0], head.group_norm(x[:1], 8, w, b)[0])


def test_no_utterances_and_no_frames():
    x, w, b, dy, n = inputs(2, 9, 16, F32, F32)
    for v, d in ((x[:0], dy[:0]), (x[:, :0], dy[:, :0])):
        y, mean, rstd = head.group_norm(v, 2, w, b)
        assert y.shape == v.shape and (mean == 0).all() and (rstd == 0).all()
        dx, dw, db = head.group_norm_backward(d, v, 2, w, b, mean, rstd)
        assert dx.shape == v.shape and (dw == 0).all() and (db == 0).all()


def test_more_utterances_than_partial_sums():
    """A block then takes several utterances, one after the other."""
    check(*inputs(5000, 3, 64, BF, F32), 8, "silu")
    check(*inputs(1100, 2, 8192, BF, F32, seed=1), 1, "relu")


def test_same_bits_again_and_on_another_stream():
    x, w, b, dy, n = inputs(9, 700, 256, BF, F32)
    want = check(x, w, b, dy, n, 8, "silu")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y, mean, rstd = head.group_norm(x, 8, w, b, lengths=n, activation="silu")
        got = (y, mean, rstd, *head.group_norm_backward(dy, x, 8, w, b, mean, rstd, lengths=n, activation="silu"))
    s.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradient_against_differences(act):
    x, w, b, dy, n = inputs(2, 9, 24, F32, F32)
    y, mean, rstd = head.group_norm(x, 3, w, b, lengths=n, activation=act)
    grads = head.group_norm_backward(dy, x, 3, w, b, mean, rstd, lengths=n, activation=act)
    args = [x.double(), w.double(), b.double()]
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").double()
        step = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + step * d, args[i] - step * d
        f = [R.GroupNorm(v[0], 3, v[1], v[2], n, EPS, act).y.view(x.shape) for v in (up, dn)]
        diff = ((f[0] - f[1]) * dy.double()).sum() / (2 * step)
        assert abs((g.double() * d).sum() - diff) <= 1e-5 * (g.double().abs() * d.abs()).sum()


def test_refusals():
    x, w, b, dy, n = inputs(2, 10, 64, BF, BF)
    y, mean, rstd = head.group_norm(x, 8, w, b)
    for bad in (lambda: head.group_norm(x.cpu(), 8), lambda: head.group_norm(x[0], 8), lambda: head.group_norm(x.double(), 8),
                lambda: head.group_norm(x, 7), lambda: head.group_norm(x, 0), lambda: head.group_norm(x, 8, w.half()),
                lambda: head.group_norm(x, 8, w, b.float()), lambda: head.group_norm(x, 8, w[:3]),
                lambda: head.group_norm(x, 8, activation="gelu"), lambda: head.group_norm(x, 8, lengths=n.long()),
                lambda: head.group_norm(x, 8, lengths=n[:1]), lambda: head.group_norm(x, 8, lengths=n.cpu()),
                lambda: head.group_norm(x, 8, outputs=(y[:1], mean, rstd)), lambda: head.group_norm(x, 8, outputs=(x, mean, rstd)),
                lambda: head.group_norm_backward(dy.float(), x, 8, w, b, mean, rstd),
                lambda: head.group_norm_backward(dy[:1], x, 8, w, b, mean, rstd),
                lambda: head.group_norm_backward(dy, x, 8, w, b, mean[:1], rstd),
                lambda: head.group_norm_backward(dy, x, 8, None, None, mean, rstd, param_dtype=HF),
                lambda: head.group_norm_backward(dy, x, 8, w, b, mean, rstd,
                                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(D.CtcpbError):
        head.group_norm(x, 8, eps=-1.0)
    with pytest.raises(D.CtcpbError):
        head.group_norm(torch.zeros(1, 1, 8193, device="cuda"), 1)
