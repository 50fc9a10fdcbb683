"""The label head's C entry points refuse bad arguments on the host, and its
size queries are consistent (no GPU needed: nothing is launched)."""
import ctypes

import pytest
import torch

from ctc_prefix_beam_gb300 import build as B
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

BIG, P = 1 << 40, 1 << 20  # a size, and an aligned non-null pointer that is never read
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    B.build()
    D.lib()
    return head._lib()


def test_size_queries(lib):
    a = head.log_probs_workspace_size(torch.bfloat16, 100, 5000, 512)
    b = head.log_probs_workspace_size(torch.bfloat16, 1000, 5000, 512)
    assert 0 < a < b and a % 256 == 0
    f = head.cross_entropy_workspace_size(torch.float16, 1000, 5000, 512, False)
    g = head.cross_entropy_workspace_size(torch.float16, 1000, 5000, 512, True)
    assert 0 < f < g and f % 256 == 0 and g % 256 == 0
    # d is held in pieces: four times the vocabulary is far from four times the memory
    g1 = head.cross_entropy_workspace_size(torch.bfloat16, 8192, 65536, 64, True)
    g4 = head.cross_entropy_workspace_size(torch.bfloat16, 8192, 262144, 64, True)
    assert g4 < 1.5 * g1
    assert 0 < head.layer_norm_workspace_size(10, 512) < head.layer_norm_workspace_size(100000, 512)
    assert head.layer_norm_workspace_size(0, 512) > 0
    n = ctypes.c_size_t()
    q, c, l = (lib["ctcpb_%s_workspace_size" % x] for x in ("log_probs", "cross_entropy", "layer_norm"))
    for bad in ((F32, 10, 20, 64), (BF16, -1, 20, 64), (BF16, 10, 0, 64), (BF16, 10, (1 << 20) + 1, 64),
                (BF16, 10, 20, 0), (BF16, 10, 20, 8193), (BF16, (1 << 24) + 1, 20, 64), (7, 10, 20, 64)):
        assert q(*bad, ctypes.byref(n)) == D.EINVAL
        assert c(*bad, 1, ctypes.byref(n)) == D.EINVAL
    assert q(BF16, 10, 20, 64, None) == D.ENULL and c(BF16, 10, 20, 64, 0, None) == D.ENULL
    assert c(BF16, 10, 20, 64, 2, ctypes.byref(n)) == D.EINVAL
    assert l(-1, 64, ctypes.byref(n)) == D.EINVAL and l(5, 64, None) == D.ENULL


def test_layer_norm_refusals(lib):
    f, g = lib["ctcpb_layer_norm"], lib["ctcpb_layer_norm_backward"]

    def fwd(type=BF16, ptype=F32, x=P, ldx=64, w=P, b=P, eps=1e-5, N=4, H=64, y=P, ldy=64, mean=P, rstd=P):
        return f(type, ptype, x, ldx, w, b, eps, N, H, y, ldy, mean, rstd, None)

    assert fwd(N=0, x=None, y=None) == D.OK
    for kw in (dict(type=3), dict(ptype=F16), dict(eps=-1.0), dict(eps=float("nan")), dict(N=-1), dict(H=0),
               dict(H=8193), dict(ldx=63), dict(ldy=63)):
        assert fwd(**kw) == D.EINVAL, kw
    for kw in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None)):
        assert fwd(**kw) == D.ENULL, kw

    def bwd(type=BF16, ptype=F32, dy=P, lddy=64, x=P, ldx=64, w=P, mean=P, rstd=P, N=4, H=64, dx=P, lddx=64, dw=P, db=P,
            ws=P, nb=BIG):
        return g(type, ptype, dy, lddy, x, ldx, w, mean, rstd, N, H, dx, lddx, dw, db, ws, nb, None)

    assert bwd(dx=None, dw=None, db=None) == D.OK
    for kw in (dict(type=3), dict(ptype=F16), dict(lddy=63), dict(ldx=63), dict(lddx=63), dict(H=9000)):
        assert bwd(**kw) == D.EINVAL, kw
    for kw in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(ws=None)):
        assert bwd(**kw) == D.ENULL, kw
    assert bwd(ws=P + 16) == D.EALIGN and bwd(nb=16) == D.ESIZE


def test_log_probs_refusals(lib):
    f = lib["ctcpb_log_probs"]

    def call(type=BF16, btype=F32, x=P, ldx=64, w=P, ldw=64, b=P, N=4, V=20, H=64, out=P, ldo=20, ws=P, nb=BIG):
        return f(type, btype, x, ldx, w, ldw, b, N, V, H, out, ldo, ws, nb, None)

    assert call(N=0, x=None, out=None) == D.OK
    for kw in (dict(type=F32), dict(btype=F16), dict(ldx=63), dict(ldw=63), dict(ldo=19), dict(N=-1), dict(V=0), dict(H=0)):
        assert call(**kw) == D.EINVAL, kw
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(ws=None)):
        assert call(**kw) == D.ENULL, kw
    assert call(ws=P + 16) == D.EALIGN and call(nb=256) == D.ESIZE


def test_cross_entropy_refusals(lib):
    f, g = lib["ctcpb_cross_entropy"], lib["ctcpb_cross_entropy_backward"]

    def fwd(type=F16, btype=F32, x=P, ldx=64, w=P, ldw=64, b=P, t=P, N=4, V=20, H=64, ign=-1, red=1, loss=P, lse=P, ws=P,
            nb=BIG):
        return f(type, btype, x, ldx, w, ldw, b, t, N, V, H, ign, red, loss, lse, ws, nb, None)

    assert fwd(N=0, red=0) == D.OK
    for kw in (dict(type=F32), dict(btype=BF16), dict(ldx=63), dict(ldw=63), dict(red=3), dict(red=-1), dict(N=-1)):
        assert fwd(**kw) == D.EINVAL, kw
    for kw in (dict(x=None), dict(w=None), dict(t=None), dict(loss=None), dict(lse=None), dict(ws=None)):
        assert fwd(**kw) == D.ENULL, kw
    assert fwd(ws=P + 128) == D.EALIGN and fwd(nb=256) == D.ESIZE

    def bwd(type=F16, btype=F32, grad=P, x=P, ldx=64, w=P, ldw=64, b=P, t=P, lse=P, N=4, V=20, H=64, ign=-1, red=1, dx=P,
            lddx=64, dw=P, lddw=64, db=P, ws=P, nb=BIG):
        return g(type, btype, grad, x, ldx, w, ldw, b, t, lse, N, V, H, ign, red, dx, lddx, dw, lddw, db, ws, nb, None)

    assert bwd(dx=None, dw=None, db=None) == D.OK
    for kw in (dict(type=F32), dict(btype=BF16), dict(ldx=63), dict(ldw=63), dict(lddx=63), dict(lddw=63), dict(red=5)):
        assert bwd(**kw) == D.EINVAL, kw
    for kw in (dict(grad=None), dict(x=None), dict(w=None), dict(t=None), dict(lse=None), dict(ws=None)):
        assert bwd(**kw) == D.ENULL, kw
    assert bwd(ws=P + 128) == D.EALIGN and bwd(nb=256) == D.ESIZE


def test_tensors_must_be_on_a_gpu():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    for call in (lambda: head.layer_norm(x), lambda: head.log_probs(x, w),
                 lambda: head.cross_entropy(x, w, torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
