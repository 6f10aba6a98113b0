"""Embedding rows and their gradient against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd
from gpu_helpers import ensure_built
from operators_reference import TINY, U32, UNIT, f64
from test_gpu_guard_canaries import Guarded, _check

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def unit(dtype):
    return UNIT[str(dtype).replace("torch.", "")], TINY[str(dtype).replace("torch.", "")]


def rows(shape, dtype, gen, pad=0, skip=0):
    """A matrix with `pad` elements between its rows, starting `skip` elements into its memory."""
    n, h = shape
    t = torch.zeros(skip + n * (h + pad), dtype=dtype, device="cuda")[skip:].view(n, h + pad)[:, :h]
    t.copy_(torch.randn(n, h, generator=gen, device="cuda"))
    return t


def make_ids(n, v, gen, spread=4):
    u = torch.rand(n, generator=gen, device="cuda")
    return (v * u.pow(spread)).long().clamp_max(v - 1).to(torch.int32)


def wrapped(ids, v):
    i = ids.cpu().numpy().astype(np.int64)
    i = np.where(i < 0, i + v, i)
    return i, (i >= 0) & (i < v)


def check_forward(ids, w, scale, y):
    i, ok = wrapped(ids, w.shape[0])
    want = f64(w)[np.where(ok, i, 0)] * np.float64(np.float32(scale))
    got = f64(y)
    assert np.isnan(got[~ok]).all()
    u, tiny = unit(y.dtype)     # one product in fp32, one rounding to y's type
    tol = (U32 + u + U32 * u) * np.abs(want) + tiny + TINY["float32"]
    assert (np.abs(got - want) <= tol)[ok].all()


FORWARD = [(1, 1, 1), (1, 50, 2560), (16, 1000, 2560), (5, 7, 33), (37, 101, 1111), (300, 1000, 64),
           (64, 300, 8), (9, 20, 4097), (2, 3, 70000), (1000, 77, 520)]


@pytest.mark.parametrize("n,v,h", FORWARD)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (BF16, F32),
                                       (F16, F32)])
def test_forward(n, v, h, dtype, out):
    gen = torch.Generator("cuda").manual_seed(n * 7 + h)
    for pad, skip in ((0, 0), (0, 1), (1, 3), (8, 0)):
        w = rows((v, h), dtype, gen, pad, skip)
        ids = torch.randint(-v, v, (n,), generator=gen, device="cuda").to(torch.int32)
        y = rows((n, h), out, gen, pad * 2, 2 * skip)
        lm.embedding_forward(ids, w, 1.7, out=y)
        check_forward(ids, w, 1.7, y)
    check_forward(ids, w, -0.3, lm.embedding_forward(ids, w, -0.3, out))


def test_forward_of_unknown_ids_is_nan_and_keeps_the_others():
    gen = torch.Generator("cuda").manual_seed(1)
    for dtype in (F32, BF16, F16):
        w = rows((50, 123), dtype, gen)
        ids = torch.tensor([0, 49, 50, -50, -51, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32,
                           device="cuda")
        y = lm.embedding_forward(ids, w, 2.0)
        check_forward(ids, w, 2.0, y)
        assert torch.isnan(y[[2, 4, 5, 6]]).all() and not torch.isnan(y[[0, 1, 3, 7]]).any()


def check_backward(dy, ids, v, scale, d, padding=None, before=None, parts=1):
    i, ok = wrapped(ids, v)
    if padding is not None:
        ok = ok & (i != padding % v)
    g, h = f64(dy), dy.shape[1]
    want, size = np.zeros((v, h)), np.zeros((v, h))
    np.add.at(want, i[ok], g[ok])
    np.add.at(size, i[ok], np.abs(g[ok]))
    count = np.bincount(i[ok], minlength=v)[:, None]
    s = np.float64(np.float32(scale))
    want, size = want * s, size * abs(s)
    got = f64(d)
    u, tiny = unit(d.dtype)
    # an id's n terms in n additions at most, a product, and an addition for each part onto what was there
    tol = (count + 1 + parts) * U32 * size * 1.01
    if before is not None:
        want, size = want + f64(before), size + np.abs(f64(before))
        tol = tol + parts * U32 * size * 1.01
    tol = tol + u * (np.abs(want) + tol) * (1 if u > U32 else 0) + tiny
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    if before is None:
        assert (got[np.bincount(i[ok], minlength=v) == 0] == 0).all()


BACKWARD = [(1, 1, 1), (1, 50, 64), (7, 5, 33), (8, 4, 64), (9, 3, 520), (40, 30, 1111), (333, 1000, 96),
            (2000, 90, 257), (5000, 20000, 64), (8191, 300, 40), (8192, 300, 40), (20000, 700, 72),
            (70000, 50, 24)]


@pytest.mark.parametrize("n,v,h", BACKWARD)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("out", [F32, BF16])
def test_backward(n, v, h, dtype, out):
    gen = torch.Generator("cuda").manual_seed(n + h)
    ids = make_ids(n, v, gen)
    pad, skip = ((0, 0), (8, 0), (3, 1))[(n + h) % 3]
    dy = rows((n, h), dtype, gen, pad, skip)
    d = lm.embedding_backward(dy, ids, v, 0.7, dtype=out)
    check_backward(dy, ids, v, 0.7, d)
    again = lm.embedding_backward(dy, ids, v, 0.7, dtype=out)
    assert torch.equal(d, again)


@pytest.mark.parametrize("n", [1, 31, 64, 1000, 9000, 40000])
def test_backward_of_one_id(n):
    """Every segment but the first begins inside the one id's tokens."""
    gen = torch.Generator("cuda").manual_seed(n)
    dy = rows((n, 200), BF16, gen)
    for id_ in (0, 4, 6, -1):
        ids = torch.full((n,), id_, dtype=torch.int32, device="cuda")
        check_backward(dy, ids, 7, 1.0, lm.embedding_backward(dy, ids, 7))


def test_backward_of_ids_that_fill_their_segments_exactly():
    gen = torch.Generator("cuda").manual_seed(3)
    for seg, n in ((8, 800), (32, 9600)):
        for length in (seg - 1, seg, seg + 1, 2 * seg, 3 * seg - 1):
            ids = (torch.arange(n, device="cuda") // length).to(torch.int32)
            ids = ids[torch.randperm(n, generator=gen, device="cuda")]
            v = n // length + 2
            dy = rows((n, 36), F32, gen)
            check_backward(dy, ids, v, 1.0, lm.embedding_backward(dy, ids, v))


def test_backward_padding_and_unknown_ids():
    gen = torch.Generator("cuda").manual_seed(5)
    n, v = 3000, 40
    ids = torch.randint(-v - 5, v + 5, (n,), generator=gen, device="cuda").to(torch.int32)
    dy = rows((n, 65), F32, gen)
    i, ok = wrapped(ids, v)
    dy[torch.from_numpy(~ok).cuda()] = float("nan")      # never looked at
    for padding in (None, 3, -1, 0):
        d = lm.embedding_backward(dy, ids, v, 1.3, padding_id=padding)
        check_backward(torch.nan_to_num(dy), ids, v, 1.3, d, padding)
    for only in (3, v, -v - 1):                          # no token left
        ids.fill_(only)
        d = lm.embedding_backward(dy, ids, v, padding_id=3, dtype=BF16)
        assert d.dtype is BF16 and not d.any()


@pytest.mark.parametrize("h", [64, 37])
def test_backward_adds_to_what_is_there(h):
    gen = torch.Generator("cuda").manual_seed(8)
    n, v = 9000, 500
    ids, dy = make_ids(n, v, gen), rows((n, h), BF16, gen)
    d = torch.randn(v, h, generator=gen, device="cuda")
    before = d.clone()
    assert lm.embedding_backward(dy, ids, v, 2.0, d_weight=d, accumulate=True) is d
    check_backward(dy, ids, v, 2.0, d, before=before)
    unmet = torch.ones(v, dtype=torch.bool, device="cuda")
    unmet[ids.long()] = False
    assert torch.equal(d[unmet], before[unmet])


@pytest.mark.parametrize("n", [131072, 131073, 300000])
def test_backward_of_more_tokens_than_one_sort(n):
    gen = torch.Generator("cuda").manual_seed(9)
    v, h = 3000, 16
    ids, dy = make_ids(n, v, gen), rows((n, h), F32, gen)
    parts = -(-n // 131072)
    check_backward(dy, ids, v, 1.0, lm.embedding_backward(dy, ids, v), parts=parts)
    if n > 131072:
        with pytest.raises(lm.LmheadError):
            lm.embedding_backward(dy, ids, v, dtype=BF16)


@pytest.mark.parametrize("v", [1, 2, 255, 256, 511, 512, 513, 2 ** 18 - 1, 2 ** 18, 2 ** 20 + 3])
def test_backward_of_vocabularies_around_the_sorts_digits(v):
    gen = torch.Generator("cuda").manual_seed(v)
    n, h = 1500, 4
    ids = torch.randint(0, v, (n,), generator=gen, device="cuda").to(torch.int32)
    ids[:3] = v - 1
    dy = rows((n, h), F32, gen)
    check_backward(dy, ids, v, 1.0, lm.embedding_backward(dy, ids, v))


def test_no_tokens():
    w = torch.ones(9, 16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert lm.embedding_forward(none, w).shape == (0, 16)
    d = torch.ones(9, 16, device="cuda")
    dy = torch.empty(0, 16, device="cuda")
    lm.embedding_backward(dy, none, 9, d_weight=d, accumulate=True)
    assert (d == 1).all()
    lm.embedding_backward(dy, none, 9, d_weight=d)
    assert not d.any()


def test_offsets_past_32_bits():
    """A table of more than 2^31 elements, and a gradient of one."""
    v, h = 1_100_000, 2048
    w = torch.zeros(v, h, dtype=BF16, device="cuda")
    w[-1] = 3.0
    w[0] = 2.0
    ids = torch.tensor([v - 1, 0, -1, -v], dtype=torch.int32, device="cuda")
    y = lm.embedding_forward(ids, w, 0.5)
    assert (y[0] == 1.5).all() and (y[1] == 1).all() and (y[2] == 1.5).all() and (y[3] == 1).all()
    d = lm.embedding_backward(y, ids, v, dtype=BF16)
    assert (d[-1] == 3).all() and (d[0] == 2).all() and not d[1:-1].any()


@pytest.mark.parametrize("n,v,h", [(1, 1, 1), (37, 53, 1111), (2000, 300, 64), (9000, 40, 9)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_writes_stay_inside(n, v, h, dtype):
    g = np.random.default_rng(n)
    ids = Guarded((n,), torch.int32, 61, torch.from_numpy(g.integers(-v - 1, v + 1, n).astype(np.int32)))
    w = Guarded((v, h), dtype, 62, torch.randn(v, h))
    y = Guarded((n, h), dtype, 63)
    assert lm.lmhead_embedding_fwd(ids.t, w.t, 1.5, y.t) == 0
    _check(dict(ids=ids, w=w), dict(y=y), "fwd")
    dy = Guarded((n, h), dtype, 64, torch.randn(n, h))
    for out in (F32, BF16):
        d = Guarded((v, h), out, 65)
        ws = Guarded((lm.lmhead_embedding_workspace_size(n, h),), torch.uint8, 66)
        assert lm.lmhead_embedding_bwd(dy.t, ids.t, 1.5, None, d.t, False, ws.t) == 0
        _check(dict(ids=ids, dy=dy), dict(d=d, ws=ws), "bwd")


def test_autograd_and_the_tied_table():
    gen = torch.Generator("cuda").manual_seed(12)
    n, v, h = 500, 900, 64
    w = rows((v, h), BF16, gen).requires_grad_(True)
    ids = make_ids(n, v, gen)
    y = autograd.embedding(ids, w, 8.0, padding_id=0)
    check_forward(ids, w, 8.0, y)
    g = rows((h, n), BF16, gen).t()            # a cotangent that autograd hands over transposed
    d, = torch.autograd.grad(y, w, g)
    assert d.dtype is BF16
    check_backward(g, ids, v, 8.0, d, padding=0)
    # tied: the head's gradient and the embedding's meet in one fp32 buffer
    w.main_grad = torch.zeros(v, h, device="cuda")
    y = autograd.embedding(ids, w, 8.0)
    logp, _ = autograd.lmhead_logps(y, w, ids.roll(-1))
    logp.sum().backward()
    assert w.grad is None
    tied = w.main_grad.clone()
    w.main_grad.zero_()
    rows_ = y.detach().requires_grad_(True)
    logp, _ = autograd.lmhead_logps(rows_, w, ids.roll(-1))
    logp.sum().backward()
    head = w.main_grad.clone()
    alone = lm.embedding_backward(rows_.grad, ids, v, 8.0)
    assert torch.allclose(tied, head + alone, rtol=2e-6, atol=2e-6 * float(alone.abs().max()))
    loose = w.detach().clone().requires_grad_(True)
    first, = torch.autograd.grad(autograd.embedding(ids, loose).float().square().sum(), loose,
                                 create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.sum(), loose)


def test_a_difference_along_the_gradient():
    gen = torch.Generator("cuda").manual_seed(13)
    w = torch.randn(40, 12, generator=gen, device="cuda")
    ids = make_ids(100, 40, gen)
    g = torch.randn(100, 12, generator=gen, device="cuda")
    d = lm.embedding_backward(g, ids, 40, 1.5).double()
    step = torch.randn(40, 12, generator=gen, device="cuda")
    # linear in the table: the difference is exact but for roundings
    up = (lm.embedding_forward(ids, w + step, 1.5).double() * g.double()).sum()
    down = (lm.embedding_forward(ids, w - step, 1.5).double() * g.double()).sum()
    size = float((g.abs().double() * 1.5 * (w.abs().double()[ids.long()] + 1) * 4).sum())
    moved = ((w + step).double() - (w - step).double())
    assert abs(float(up - down) - float((d * moved).sum())) <= 100 * U32 * size


def test_streams_and_graphs():
    gen = torch.Generator("cuda").manual_seed(14)
    n, v, h = 5000, 800, 72
    w, dy, ids = rows((v, h), BF16, gen), rows((n, h), BF16, gen), make_ids(n, v, gen)
    want = lm.embedding_forward(ids, w, 2.0), lm.embedding_backward(dy, ids, v, 2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        got = (lm.embedding_forward(ids, w, 2.0, stream=handle),
               lm.embedding_backward(dy, ids, v, 2.0, stream=handle))
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = (lm.embedding_forward(ids, w, 2.0), lm.embedding_backward(dy, ids, v, 2.0))
        graphs.append((graph, out))
    other = make_ids(n, v, gen, 2)
    ids.copy_(other)
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = lm.embedding_forward(ids, w, 2.0), lm.embedding_backward(dy, ids, v, 2.0)
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
