"""The C entry points around the label head (group norm, dropout, policy and preference
losses) refuse bad arguments on the host; the generator's definition against its
published vectors (no GPU needed: nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import more_ref as R
from ctc_prefix_beam_gb300 import build as B
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

BIG, P = 1 << 40, 1 << 20  # a size, and an aligned non-null pointer that is never read
F32, BF16, F16 = 0, 1, 2
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    B.build()
    D.lib()
    return head._lib()


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0), "d16cfe09 94fdcceb 5001e420 24126ea1")])
def test_generator_vectors(ctr, key, want):
    """Known answers that the generator's authors publish."""
    got = R.philox([np.array([c], np.uint64) for c in ctr], key)[:, 0]
    assert " ".join("%08x" % v for v in got) == want


def test_size_queries(lib):
    BF = torch.bfloat16
    assert 0 < head.group_norm_workspace_size(BF, 2, 10, 64, 4, True) < head.group_norm_workspace_size(BF, 64, 500, 512, 32, True)
    assert head.group_norm_workspace_size(BF, 32, 500, 512, 32, False) == 0
    assert 0 < head.group_norm_workspace_size(BF, 1, 100000, 512, 1, False) < 1 << 20
    assert head.group_norm_workspace_size(BF, 0, 10, 64, 4, True) == 0
    # a small share of the tensors, whatever the shape
    for shape in ((1 << 20, 16, 8192, 1), (1 << 24, 1, 64, 1), (1, 1 << 24, 8, 8), (1 << 12, 1 << 12, 513, 27)):
        for dtype, e in ((BF, 2), (torch.float32, 4)):
            assert head.group_norm_workspace_size(dtype, *shape, True) <= (64 << 20) + shape[0] * shape[1] * shape[2] * e // 50
    # small calls have only the status in it, and may go without
    assert head.policy_loss_workspace_size(320, 40) == head.preference_loss_workspace_size(32, 10, 40) == 256
    for n in (head.policy_loss_workspace_size(4096, 1024), head.preference_loss_workspace_size(1024, 4, 1000),
              head.policy_loss_workspace_size(1 << 24, 255), head.policy_loss_workspace_size(10000, 1),
              head.preference_loss_workspace_size(100, 2, 4)):
        assert n % 256 == 0 and 256 < n < 1 << 20
    n = ctypes.c_size_t()
    g, p, q = (lib["ctcpb_%s_workspace_size" % x] for x in ("group_norm", "policy_loss", "preference_loss"))
    for bad in ((-1, 4, 64, 4), (4, -1, 64, 4), (4, 4, 0, 1), (4, 4, 64, 0), (4, 4, 64, 5), (4, 4, 8193, 1),
                (1 << 13, 1 << 12, 64, 4), (0, (1 << 24) + 1, 64, 4), ((1 << 24) + 1, 0, 64, 4)):
        assert g(BF16, *bad, 1, ctypes.byref(n)) == D.EINVAL, bad
    assert g(7, 4, 4, 64, 4, 1, ctypes.byref(n)) == D.EINVAL and g(BF16, 4, 4, 64, 4, 2, ctypes.byref(n)) == D.EINVAL
    assert g(BF16, 4, 4, 64, 4, 1, None) == D.ENULL
    for bad in ((-1, 4), (4, -1), ((1 << 24) + 1, 4), (4, (1 << 24) + 1), (1 << 16, 1 << 16)):
        assert p(*bad, ctypes.byref(n)) == D.EINVAL, bad
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, -1), (1 << 22, 8, 4), (1, 4, (1 << 24) + 1)):
        assert q(*bad, ctypes.byref(n)) == D.EINVAL, bad
    assert p(4, 4, None) == D.ENULL and q(4, 4, 4, None) == D.ENULL


def test_group_norm_refusals(lib):
    f, g = lib["ctcpb_group_norm"], lib["ctcpb_group_norm_backward"]

    def fwd(type=BF16, ptype=F32, x=P, xb=640, xt=64, w=P, b=P, n=P, eps=1e-5, act=2, B=4, T=10, C=64, G=8, y=P, yb=640,
            yt=64, mean=P, rstd=P, ws=P, nb=BIG):
        return f(type, ptype, x, xb, xt, w, b, n, eps, act, B, T, C, G, y, yb, yt, mean, rstd, ws, nb, None)

    assert fwd(B=0, x=None, y=None) == D.OK
    assert fwd(T=0, x=None, y=None, mean=None, rstd=None) == D.OK
    for kw in (dict(type=3), dict(ptype=F16), dict(eps=-1.0), dict(eps=NAN), dict(act=3), dict(act=-1), dict(B=-1),
               dict(T=-1), dict(C=0), dict(G=0), dict(G=5), dict(C=16384, G=1, xt=16384, yt=16384), dict(xt=63), dict(yt=63),
               dict(xb=-1), dict(yb=-1), dict(B=1 << 12, T=(1 << 12) + 1)):
        assert fwd(**kw) == D.EINVAL, kw
    for kw in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None)):
        assert fwd(**kw) == D.ENULL, kw
    far = dict(B=1, T=100000, G=1, xb=0, yb=0)  # in two launches
    assert fwd(ws=None, **far) == D.ENULL and fwd(ws=P + 16, **far) == D.EALIGN and fwd(nb=16, **far) == D.ESIZE

    def bwd(type=BF16, ptype=F32, dy=P, db=640, dt=64, x=P, xb=640, xt=64, w=P, b=P, n=P, mean=P, rstd=P, act=2, B=4, T=10,
            C=64, G=8, dx=P, ob=640, ot=64, dw=P, dbias=P, ws=P, nb=BIG):
        return g(type, ptype, dy, db, dt, x, xb, xt, w, b, n, mean, rstd, act, B, T, C, G, dx, ob, ot, dw, dbias, ws, nb, None)

    assert bwd(dx=None, dw=None, dbias=None) == D.OK
    assert bwd(B=0, dy=None, x=None, dw=None, dbias=None) == D.OK
    for kw in (dict(type=3), dict(ptype=F16), dict(act=7), dict(dt=63), dict(xt=63), dict(ot=63), dict(db=-1), dict(ob=-1),
               dict(G=7)):
        assert bwd(**kw) == D.EINVAL, kw
    for kw in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(ws=None)):
        assert bwd(**kw) == D.ENULL, kw
    assert bwd(ws=P + 16) == D.EALIGN and bwd(nb=16) == D.ESIZE


def test_dropout_refusals(lib):
    f = lib["ctcpb_dropout"]

    def call(type=BF16, x=P, ldx=64, r=P, ldr=64, p=0.1, rng=P, N=4, H=64, y=P, ldy=64):
        return f(type, x, ldx, r, ldr, p, rng, N, H, y, ldy, None)

    assert call(N=0, x=None, y=None, rng=None) == D.OK
    for kw in (dict(type=3), dict(ldx=63), dict(ldr=63), dict(ldy=63), dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(N=-1),
               dict(N=(1 << 24) + 1), dict(H=0), dict(H=8193)):
        assert call(**kw) == D.EINVAL, kw
    for kw in (dict(x=None), dict(y=None), dict(rng=None)):
        assert call(**kw) == D.ENULL, kw


def test_policy_refusals(lib):
    f = lib["ctcpb_policy_loss"]

    def call(nll=P, ld=40, old=P, ldo=40, ref=P, ldr=40, adv=P, lda=0, n=P, S=4, L=40, lo=0.2, hi=0.2, kl=0.1, red=1, grad=P,
             loss=P, stats=P, dnll=P, ws=P, nb=BIG):
        return f(nll, ld, old, ldo, ref, ldr, adv, lda, n, S, L, lo, hi, kl, red, grad, loss, stats, dnll, ws, nb, None)

    for kw in (dict(ld=39), dict(ldo=39), dict(ldr=39), dict(lda=39), dict(lda=-1), dict(S=-1), dict(L=-1), dict(lo=-0.1),
               dict(lo=NAN), dict(lo=INF), dict(hi=-0.1), dict(hi=NAN), dict(kl=NAN), dict(kl=INF), dict(red=4), dict(red=-1)):
        assert call(**kw) == D.EINVAL, kw
    for kw in (dict(nll=None), dict(old=None), dict(adv=None), dict(grad=None), dict(ws=None, S=10000)):
        assert call(**kw) == D.ENULL, kw
    assert call(ws=P + 16) == D.EALIGN and call(nb=200) == D.ESIZE and call(nb=300, S=10000) == D.ESIZE


def test_preference_refusals(lib):
    f = lib["ctcpb_preference_loss"]

    def call(nll=P, ld=40, ref=P, ldr=40, c=P, r=P, n=P, B=4, N=5, L=40, beta=0.1, margin=0.0, s=0.0, avg=0, red=1, grad=P,
             loss=P, margins=P, dnll=P, ws=P, nb=BIG):
        return f(nll, ld, ref, ldr, c, r, n, B, N, L, beta, margin, s, avg, red, grad, loss, margins, dnll, ws, nb, None)

    for kw in (dict(ld=39), dict(ldr=39), dict(B=-1), dict(N=0), dict(L=-1), dict(beta=NAN), dict(beta=INF), dict(margin=INF),
               dict(s=-0.1), dict(s=1.1), dict(s=NAN), dict(avg=2), dict(red=3), dict(red=-1)):
        assert call(**kw) == D.EINVAL, kw
    for kw in (dict(nll=None), dict(c=None), dict(r=None), dict(grad=None), dict(ws=None, B=10000)):
        assert call(**kw) == D.ENULL, kw
    assert call(ws=P + 16) == D.EALIGN and call(nb=200) == D.ESIZE and call(nb=300, B=10000) == D.ESIZE


def test_tensors_must_be_on_a_gpu():
    x, i = torch.zeros(2, 4, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: head.group_norm(x, 2), lambda: head.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64)),
                 lambda: head.policy_loss(x, x, x), lambda: head.preference_loss(x, i, i)):
        with pytest.raises(ValueError):
            call()
