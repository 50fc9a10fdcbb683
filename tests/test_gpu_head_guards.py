"""Guard margins around every buffer of the label head's C calls: workspaces and
outputs are views into larger patterned buffers whose margins must be unchanged
after the calls.  Strided outputs keep what lies between their rows.  Also the
calls that leave some gradients out."""
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
        return self.view.data_ptr()

    def intact(self):
        return bool((self.buf[:G] == PAT).all()) and bool((self.buf[G + self.n:] == PAT).all())


def stream():
    return torch.cuda.current_stream().cuda_stream


def make(n, v, h, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n + v + h)
    w = (torch.randn(v, h, generator=g, device="cuda") / h ** 0.5).to(dtype)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    b = torch.randn(v, generator=g, device="cuda")
    t = torch.randint(-1, v, (n,), generator=g, device="cuda").int()
    return x, w, b, t


@pytest.mark.parametrize("n,v,h,ldo", [(130, 300, 64, 300), (130, 301, 72, 308), (130, 301, 71, 303), (5, 29, 33, 29),
                                       (700, 5000, 128, 5000), (1, 70000, 64, 70000)])
def test_log_probs_writes(n, v, h, ldo):
    x, w, b, _ = make(n, v, h, torch.bfloat16)
    want = head.log_probs(x, w, b)
    out, ws = Guarded(4 * n * ldo), Guarded(head.log_probs_workspace_size(torch.bfloat16, n, v, h))
    rc = head._lib()["ctcpb_log_probs"](1, 0, x.data_ptr(), h, w.data_ptr(), h, b.data_ptr(), n, v, h, out.ptr(), ldo,
                                        ws.ptr(), ws.n, stream())
    torch.cuda.synchronize()
    assert rc == D.OK and out.intact() and ws.intact() and D.read_status(ws.view) == 0
    got = out.typed(torch.float32, n, ldo)
    assert torch.equal(got[:, :v], want)
    assert (out.view.view(n, ldo * 4)[:, v * 4:] == PAT).all()


@pytest.mark.parametrize("n,v,h", [(130, 300, 64), (257, 1000, 71), (3, 29, 33), (600, 5001, 136), (50, 32, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_cross_entropy_writes(n, v, h, dtype):
    x, w, b, t = make(n, v, h, dtype)
    L = head._lib()
    loss, lse = Guarded(4), Guarded(4 * n)
    ws = Guarded(head.cross_entropy_workspace_size(dtype, n, v, h, False))
    rc = L["ctcpb_cross_entropy"](TYPE[dtype], 0, x.data_ptr(), h, w.data_ptr(), h, b.data_ptr(), t.data_ptr(), n, v, h, -1,
                                  1, loss.ptr(), lse.ptr(), ws.ptr(), ws.n, stream())
    torch.cuda.synchronize()
    assert rc == D.OK and loss.intact() and lse.intact() and ws.intact()
    wl, wlse = head.cross_entropy(x, w, t, b)
    assert torch.equal(loss.typed(torch.float32, 1)[0], wl) and torch.equal(lse.typed(torch.float32, n), wlse)
    one = torch.ones(1, device="cuda")
    want = head.cross_entropy_backward(one[0], x, w, t, wlse, b)
    pad = 3  # rows further apart than they are long
    for dx_on, dw_on, db_on in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        dx, dw, db = Guarded(2 * n * (h + pad)), Guarded(2 * v * (h + pad)), Guarded(4 * v)
        ws = Guarded(head.cross_entropy_workspace_size(dtype, n, v, h, True))
        rc = L["ctcpb_cross_entropy_backward"](
            TYPE[dtype], 0, one.data_ptr(), x.data_ptr(), h, w.data_ptr(), h, b.data_ptr(), t.data_ptr(), lse.ptr(), n, v,
            h, -1, 1, dx.ptr() if dx_on else None, h + pad, dw.ptr() if dw_on else None, h + pad,
            db.ptr() if db_on else None, ws.ptr(), ws.n, stream())
        torch.cuda.synchronize()
        assert rc == D.OK and dx.intact() and dw.intact() and db.intact() and ws.intact()
        assert D.read_status(ws.view) == 0
        for on, buf, rows, ref in ((dx_on, dx, n, want[0]), (dw_on, dw, v, want[1])):
            if on:
                assert torch.equal(buf.typed(dtype, rows, h + pad)[:, :h], ref)
                assert (buf.view.view(rows, 2 * (h + pad))[:, 2 * h:] == PAT).all()
            else:
                assert (buf.view == PAT).all()
        if db_on:
            assert torch.equal(db.typed(torch.float32, v), want[2])


@pytest.mark.parametrize("n,h", [(130, 64), (33, 769), (7, 4100), (1, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_norm_writes(n, h, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + h)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    dy = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    w, b = torch.randn(h, generator=g, device="cuda"), torch.randn(h, generator=g, device="cuda")
    e = 4 if dtype == torch.float32 else 2
    L = head._lib()
    y, mean, rstd = Guarded(e * n * h), Guarded(4 * n), Guarded(4 * n)
    assert L["ctcpb_layer_norm"](TYPE[dtype], 0, x.data_ptr(), h, w.data_ptr(), b.data_ptr(), 1e-5, n, h, y.ptr(), h,
                                 mean.ptr(), rstd.ptr(), stream()) == D.OK
    torch.cuda.synchronize()
    assert y.intact() and mean.intact() and rstd.intact()
    wy, wm, wr = head.layer_norm(x, w, b)
    assert torch.equal(y.typed(dtype, n, h), wy) and torch.equal(mean.typed(torch.float32, n), wm)
    want = head.layer_norm_backward(dy, x, w, wm, wr)
    for dx_on, dw_on, db_on in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        dx, dw, db, ws = Guarded(e * n * h), Guarded(4 * h), Guarded(4 * h), Guarded(head.layer_norm_workspace_size(n, h))
        assert L["ctcpb_layer_norm_backward"](
            TYPE[dtype], 0, dy.data_ptr(), h, x.data_ptr(), h, w.data_ptr(), mean.ptr(), rstd.ptr(), n, h,
            dx.ptr() if dx_on else None, h, dw.ptr() if dw_on else None, db.ptr() if db_on else None, ws.ptr(), ws.n,
            stream()) == D.OK
        torch.cuda.synchronize()
        assert dx.intact() and dw.intact() and db.intact() and ws.intact()
        for on, got, ref in ((dx_on, dx.typed(dtype, n, h), want[0]), (dw_on, dw.typed(torch.float32, h), want[1]),
                             (db_on, db.typed(torch.float32, h), want[2])):
            if on:
                assert torch.equal(got, ref)
            else:
                assert (got.view(torch.uint8) == PAT).all()
