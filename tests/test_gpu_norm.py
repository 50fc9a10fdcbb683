"""Layer norm and its backward pass against definitions in 64 bits (head_ref)."""
import pytest
import torch

import head_ref as R
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


def inputs(n, h, dtype, params, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 100 + n * 3 + h)
    x = torch.randn(n, h, generator=g, device="cuda") * 2 + torch.randn(n, 1, generator=g, device="cuda")
    w = 1 + 0.3 * torch.randn(h, generator=g, device="cuda")
    b = 0.2 * torch.randn(h, generator=g, device="cuda")
    dy = torch.randn(n, h, generator=g, device="cuda")
    return x.to(dtype), w.to(params), b.to(params), dy.to(dtype)


def check(x, w, b, dy, ws=None):
    n, h = x.shape
    y, mean, rstd = head.layer_norm(x, w, b, eps=EPS)
    ry, rm, rr, xh = R.layer_norm(x, w, b, EPS)
    # a float32 sum of h values: a few units of sum |x| / h; the variance's is
    # relative (positive terms, the mean's error enters squared)
    s = x.double().abs().mean(1)
    em = 16 * R.U[F32] * s
    er = 32 * R.U[F32]
    assert ((mean.double() - rm).abs() <= em).all()
    assert ((rstd.double() / rr - 1).abs() <= er + (em * rr) ** 2).all()
    wa = torch.ones(h, device="cuda").double() if w is None else w.double().abs()
    ba = torch.zeros(h, device="cuda").double() if b is None else b.double().abs()
    ey = wa * ((em * rr)[:, None] + 40 * R.U[F32] * xh.abs()) + 4 * R.U[F32] * ba
    assert ((y.double() - ry).abs() <= ey + R.U[x.dtype] * ry.abs() + R.TINY[x.dtype]).all()
    dx, dw, db = head.layer_norm_backward(dy, x, w, mean, rstd, workspace=ws)
    rdx, rdw, rdb = R.layer_norm_backward(dy, x, w, EPS)
    t = dy.double().abs() * wa
    exh = (em * rr)[:, None] + 40 * R.U[F32] * xh.abs()  # what xh is off by
    edx = rr[:, None] * (64 * R.U[F32] * (t + t.mean(1, keepdim=True) + xh.abs() * (t * xh.abs()).mean(1, keepdim=True)) +
                         exh * (t * xh.abs()).mean(1, keepdim=True) + xh.abs() * (t * exh).mean(1, keepdim=True))
    assert ((dx.double() - rdx).abs() <= edx + R.U[x.dtype] * rdx.abs() + R.TINY[x.dtype]).all()
    # float32 sums over n rows: chains of n / 304 rows, then 304 blocks
    depth = 8 * (n / 304 + 60) ** 0.5 * R.U[F32]
    up = R.U[dw.dtype]
    dya = dy.double().abs()
    assert ((dw.double() - rdw).abs() <= depth * (dya * xh.abs()).sum(0) + (dya * exh).sum(0) + up * rdw.abs() +
            R.TINY[dw.dtype]).all()
    assert ((db.double() - rdb).abs() <= depth * dya.sum(0) + up * rdb.abs() + R.TINY[db.dtype]).all()
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("n,h", [(1, 1), (1, 512), (5, 8), (7, 31), (33, 512), (200, 513), (9, 1000), (64, 1024),
                                 (19, 1025), (3, 4096), (2, 4099), (2, 8192), (5000, 64), (700, 769)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_layer_norm(n, h, dtype):
    x, w, b, dy = inputs(n, h, dtype, F32 if (n + h) % 2 else dtype)
    check(x, w, b, dy)


def test_without_parameters():
    x, w, b, dy = inputs(40, 96, BF, BF)
    check(x, None, None, dy)
    check(x, w, None, dy)
    y, mean, rstd = head.layer_norm(x, None, b)
    _, dw, _ = head.layer_norm_backward(dy, x, None, mean, rstd, param_dtype=F32)
    assert dw.dtype == F32


def test_many_rows():
    check(*inputs(40000, 256, BF, F32))


def test_constant_and_offset_rows():
    """A constant row has variance 0 (rstd = 1 / sqrt(eps)); a large common
    offset does not eat the differences."""
    x, w, b, dy = inputs(20, 512, F32, F32)
    x[3] = 5.0
    x[4] = 0.0
    x[5] += 1000.0
    y, mean, rstd = head.layer_norm(x, w, b, eps=EPS)
    assert torch.equal(y[3], b) and torch.equal(y[4], b)
    assert abs(rstd[3].item() * EPS ** 0.5 - 1) < 1e-6
    check(x, w, b, dy)


def test_special_values_stay_in_their_rows():
    x, w, b, dy = inputs(20, 100, BF, F32)
    want = head.layer_norm(x, w, b)[0]
    x2 = x.clone()
    x2[6, 3], x2[9, 0] = float("nan"), float("inf")
    got = head.layer_norm(x2, w, b)[0]
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[[6, 9]] = False
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[~keep]).all()


def test_strides_and_shapes():
    x, w, b, dy = inputs(60, 72, HF, HF)
    want = check(x, w, b, dy)
    wide = torch.zeros(60, 200, dtype=HF, device="cuda")
    for off in (8, 13):
        wide[:, off:off + 72] = x
        wide[:, 100 + off:172 + off] = dy
        xs, ds = wide[:, off:off + 72], wide[:, 100 + off:172 + off]
        y, mean, rstd = head.layer_norm(xs, w, b, eps=EPS)
        got = (y, mean, rstd, *head.layer_norm_backward(ds, xs, w, mean, rstd))
        for a, c in zip(got[:4], want[:4]):
            assert torch.allclose(a.float(), c.float(), rtol=2 ** -10, atol=1e-6)  # another split of the row's sums
    y3, m3, r3 = head.layer_norm(x.view(3, 20, 72), w, b, eps=EPS)
    assert y3.shape == (3, 20, 72) and m3.shape == (3, 20) and torch.equal(y3.view(60, 72), want[0])
    dx3, dw3, db3 = head.layer_norm_backward(dy.view(3, 20, 72), x.view(3, 20, 72), w, m3, r3)
    assert torch.equal(dx3.view(60, 72), want[3]) and torch.equal(dw3, want[4]) and torch.equal(db3, want[5])


def test_no_rows():
    x, w, b, dy = inputs(3, 40, F32, F32)
    y, mean, rstd = head.layer_norm(x[:0], w, b)
    dx, dw, db = head.layer_norm_backward(dy[:0], x[:0], w, mean, rstd)
    assert y.shape == dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()


def test_same_bits_again_and_on_another_stream():
    x, w, b, dy = inputs(9000, 512, BF, F32)
    want = check(x, w, b, dy)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y, mean, rstd = head.layer_norm(x, w, b, eps=EPS)
        got = (y, mean, rstd, *head.layer_norm_backward(dy, x, w, mean, rstd))
    s.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_gradient_against_differences():
    x, w, b, dy = inputs(6, 40, F32, F32)
    y, mean, rstd = head.layer_norm(x, w, b, eps=EPS)
    grads = head.layer_norm_backward(dy, x, w, mean, rstd)
    args = [x.double(), w.double(), b.double()]
    for i, g in enumerate(grads):
        d = torch.randn(args[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").double()
        step = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + step * d, args[i] - step * d
        diff = ((R.layer_norm(*up, EPS)[0] - R.layer_norm(*dn, EPS)[0]) * dy.double()).sum() / (2 * step)
        assert abs((g.double() * d).sum() - diff) <= 1e-5 * (g.double().abs() * d.abs()).sum()


def test_refusals():
    x, w, b, dy = inputs(10, 64, BF, BF)
    y, mean, rstd = head.layer_norm(x, w, b)
    for bad in (lambda: head.layer_norm(x.cpu(), w, b), lambda: head.layer_norm(x, w.half(), b),
                lambda: head.layer_norm(x, w[:5], b), lambda: head.layer_norm(x, w.float(), b),
                lambda: head.layer_norm(x.double(), None, None),
                lambda: head.layer_norm_backward(dy.float(), x, w, mean, rstd),
                lambda: head.layer_norm_backward(dy[:5], x, w, mean, rstd),
                lambda: head.layer_norm_backward(dy, x, w, mean[:3], rstd),
                lambda: head.layer_norm_backward(dy, x, w, mean, rstd,
                                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(D.CtcpbError):
        head.layer_norm(x, w, b, eps=-1.0)
    wide = torch.zeros(2, 8193, device="cuda")
    with pytest.raises(D.CtcpbError):
        head.layer_norm(wide)
