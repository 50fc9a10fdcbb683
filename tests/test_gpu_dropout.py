"""Dropout: the same bits as the generator's definition (more_ref) and float32
arithmetic give, for every layout."""
import pytest
import torch

import more_ref as R
from ctc_prefix_beam_gb300 import decoder as D
from ctc_prefix_beam_gb300 import head

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SEED, OFFSET = -0x123456789ABCDEF, 0x7FFFFFFF12345678


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from ctc_prefix_beam_gb300 import build
    build.build()
    D.lib()
    assert torch.cuda.is_available()


def rng(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def inputs(shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * 3).to(dtype), torch.randn(shape, generator=g,
                                                                                      device="cuda").to(dtype)


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (1, 8), (3, 8), (5, 13), (50, 64), (301, 769), (2, 3, 8192), (40, 16, 512),
                                   (1, 8191), (9,)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout(shape, dtype, p):
    x, r = inputs(shape, dtype)
    assert same(head.dropout(x, p, rng()), R.dropout(x, p, SEED, OFFSET))
    assert same(head.dropout(x, p, rng(), residual=r), R.dropout(x, p, SEED, OFFSET, r))
    assert same(head.dropout_backward(r, p, rng()), R.dropout(r, p, SEED, OFFSET))


def test_probabilities():
    x, r = inputs((40, 100), F32)
    assert same(head.dropout(x, 0.0, rng()), x)
    assert (head.dropout(x, 1.0, rng()) == 0).all() and same(head.dropout(x, 1.0, rng(), residual=r), r)
    assert (head.dropout(x, 1 - 2.0 ** -20, rng()) == 0).all()  # rounds to 1
    for p in (2.0 ** -16, 1 - 2.0 ** -16, 0.3):
        assert same(head.dropout(x, p, rng()), R.dropout(x, p, SEED, OFFSET))
    big = torch.ones(4000, 1000, device="cuda")
    share = (head.dropout(big, 0.3, rng()) == 0).double().mean().item()
    assert abs(share - 0.3) < 6 * (0.3 * 0.7 / big.numel()) ** 0.5 + 2.0 ** -16


def test_seeds_and_offsets():
    x, _ = inputs((64, 64), BF)
    seen = []
    for seed, off in ((0, 0), (1, 0), (0, 1), (1 << 32, 0), (0, 1 << 32), (-1, -1)):
        y = head.dropout(x, 0.5, rng(seed, off))
        assert same(y, R.dropout(x, 0.5, seed, off))
        seen.append(y)
    for i in range(len(seen)):
        for j in range(i):
            assert not torch.equal(seen[i], seen[j])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_give_the_same_elements(dtype):
    """An element's fate goes by its index in the shape."""
    for h in (72, 61):
        x, r = inputs((50, h), dtype)
        want = R.dropout(x, 0.4, SEED, OFFSET, r)
        wide = torch.full((50, 300), float("nan"), dtype=dtype, device="cuda")
        for off in (8, 13):
            wide[:, off:off + h] = x
            wide[:, 150 + off:150 + off + h] = r
            assert same(head.dropout(wide[:, off:off + h], 0.4, rng(), residual=wide[:, 150 + off:150 + off + h]), want)
        assert same(head.dropout(x.t().contiguous().t(), 0.4, rng(), residual=r), want)
        # outputs with a stride, by the C call: what lies between the rows stays
        out = torch.full((50, 80), 7.0, dtype=dtype, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        seed = rng()
        assert head._lib()["ctcpb_dropout"](head._TYPES[dtype], x.data_ptr(), h, r.data_ptr(), h, 0.4, seed.data_ptr(), 50, h,
                                            out.data_ptr(), 80, s) == D.OK
        torch.cuda.synchronize()
        assert same(out[:, :h].contiguous(), want) and (out[:, h:] == 7).all()


def test_in_place():
    x, r = inputs((33, 100), HF)
    want = R.dropout(x, 0.2, SEED, OFFSET, r)
    a, b = x.clone(), r.clone()
    assert head.dropout(a, 0.2, rng(), residual=r, out=a) is a and same(a, want)
    head.dropout(x, 0.2, rng(), residual=b, out=b)
    assert same(b, want)


def test_what_is_dropped_is_of_no_account():
    x, _ = inputs((30, 64), F32)
    keep, _ = R.kept(0, x.numel(), 0.5, SEED, OFFSET)
    keep = torch.from_numpy(keep).cuda().view(x.shape)
    want = head.dropout(x, 0.5, rng())
    x[~keep] = float("nan")
    assert same(head.dropout(x, 0.5, rng()), want)
    x[~keep] = float("inf")
    assert same(head.dropout(x, 0.5, rng()), want)


def test_rows_past_32_bits():
    """Strides that take offsets past 2^31 elements, and more than 2^35 elements: the
    block's number then takes a second word of the counter."""
    far = torch.zeros(3 * 0x40000000 + 64, dtype=BF, device="cuda")
    x, _ = inputs((4, 64), BF)
    view = far.as_strided((4, 64), (0x40000000, 1))
    view.copy_(x)
    assert same(head.dropout(view, 0.5, rng()), R.dropout(x, 0.5, SEED, OFFSET))
    del far, view
    H, N = 8192, (1 << 22) + 2
    big = torch.ones(N, H, dtype=BF, device="cuda")
    head.dropout(big, 0.5, rng(), out=big)
    for row in (0, 1 << 18, (1 << 22) - 1, 1 << 22, (1 << 22) + 1):
        one = torch.ones(H, dtype=BF, device="cuda")
        assert same(big[row], R.dropout(one, 0.5, SEED, OFFSET, first=row * H))


def test_a_captured_call_reads_the_seed_when_replayed():
    x, r = inputs((130, 72), BF)
    seed = rng(5, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        head.dropout(x, 0.3, seed, residual=r)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = head.dropout(x, 0.3, seed, residual=r)
        dx = head.dropout_backward(r, 0.3, seed)
        seed[1] += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert same(y, R.dropout(x, 0.3, 5, step, r)) and same(dx, R.dropout(r, 0.3, 5, step))


def test_refusals():
    x, r = inputs((10, 64), BF)
    for bad in (lambda: head.dropout(x.cpu(), 0.1, rng()), lambda: head.dropout(x, 0.1, rng().cpu()),
                lambda: head.dropout(x, 0.1, rng().int()), lambda: head.dropout(x, 0.1, rng()[:1]),
                lambda: head.dropout(x, 0.1, rng(), residual=r.float()), lambda: head.dropout(x, 0.1, rng(), residual=r[:5]),
                lambda: head.dropout(x, 0.1, rng(), out=r.float()), lambda: head.dropout(x, 0.1, rng(), out=r.t()),
                lambda: head.dropout(x.double(), 0.1, rng())):
        with pytest.raises(ValueError):
            bad()
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(D.CtcpbError):
            head.dropout(x, p, rng())
