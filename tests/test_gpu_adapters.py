"""Low-rank adapters beside a shared projection against a plain 64-bit implementation."""
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


def rows(shape, dtype, gen, pad=0, skip=0, size=1.0):
    n, h = shape
    t = torch.zeros(skip + n * (h + pad), dtype=dtype, device="cuda")[skip:].view(n, h + pad)[:, :h]
    t.copy_(size * torch.randn(n, h, generator=gen, device="cuda"))
    return t


def make(T, H, V, rank, n, dtype, seed, pad=0, skip=0, runs=False, bare=0.2):
    g = torch.Generator("cuda").manual_seed(seed)
    of = torch.randint(0, n, (T,), generator=g, device="cuda")
    of = of.sort().values if runs else of
    of = torch.where(torch.rand(T, generator=g, device="cuda") < bare, -1, of).to(torch.int32)
    return dict(x=rows((T, H), BF16, g, pad, skip), of=of,
                down=(torch.randn(n, rank, H, generator=g, device="cuda") / H ** 0.5).to(BF16),
                up=torch.randn(n, rank, V, generator=g, device="cuda").to(BF16),
                scale=torch.randn(n, generator=g, device="cuda"),
                base=rows((T, V), dtype, g, pad, skip), grad=rows((T, V), dtype, g, pad, skip))


def named(t):
    return str(t.dtype).replace("torch.", "")


def groups(s):
    n = s["up"].shape[0]
    of = np.zeros(len(s["x"]), int) if s["of"] is None else s["of"].cpu().numpy()
    scale = np.ones(n) if s["scale"] is None else f64(s["scale"])
    for a in range(n):
        at = np.flatnonzero(of == a)
        yield a, at, f64(s["x"])[at], f64(s["down"])[a], f64(s["up"])[a], scale[a]


# An fp32 sum of n products of bf16 numbers is off by n roundings at most, here of up to a
# whole unit (matrix instructions may cut): n 2 U32 of the sum of magnitudes.  Three bf16
# parts hold a number to 2^-24 and products of theirs that are left out lie below 3 * 2^-24;
# two parts hold it to 2^-16.
def off(n):
    return (n + 70) * 2 * U32


def check_forward(s, out):
    want, tol = f64(s["base"]), np.zeros(s["base"].shape)
    rank = s["up"].shape[1]
    parts = 8 * U32 if s["base"].dtype is F32 else 2.0 ** -16
    for _, at, x, down, up, scale in groups(s):
        u = scale * x @ down.T
        size = abs(scale) * np.abs(x) @ np.abs(down).T
        want[at] += u @ up
        tol[at] += size @ np.abs(up) * (off(x.shape[1]) + off(3 * rank) + parts)
    unit = UNIT[named(s["base"])]
    tol = tol + U32 * np.abs(want) + (unit + U32) * (np.abs(want) + tol) + TINY[named(s["base"])]
    assert (np.abs(f64(out) - want) <= tol).all(), np.max(np.abs(f64(out) - want) / tol)


def check_backward(s, dx, d_down, d_up, dx0=None, down0=None, up0=None, extra=1):
    g_all = f64(s["grad"])
    rank = s["up"].shape[1]
    wants = [np.zeros(t.shape) if t0 is None else f64(t0)
             for t, t0 in ((dx, dx0), (d_down, down0), (d_up, up0))]
    tols = [2 * extra * U32 * np.abs(w) for w in wants]
    for a, at, x, down, up, scale in groups(s):
        g = g_all[at]
        u, u_size = scale * x @ down.T, abs(scale) * np.abs(x) @ np.abs(down).T
        du, du_size = scale * g @ up.T, abs(scale) * np.abs(g) @ np.abs(up).T
        n_u, n_du, n_t = off(x.shape[1]), off(3 * g.shape[1]), off(6 * len(at) + extra)
        wants[0][at] += du @ down
        tols[0][at] += du_size @ np.abs(down) * (n_du + off(3 * rank) + 8 * U32)
        wants[1][a] += du.T @ x
        tols[1][a] += du_size.T @ np.abs(x) * (n_du + n_t + 8 * U32)
        wants[2][a] += u.T @ g
        tols[2][a] += u_size.T @ np.abs(g) * (n_u + n_t + 8 * U32)
    for name, t, want, tol in zip(("dx", "d_down", "d_up"), (dx, d_down, d_up), wants, tols):
        assert (np.abs(f64(t) - want) <= tol + 1e-37).all(), (name, np.max(np.abs(f64(t) - want) / (tol + 1e-37)))


SIZES = [  # T, H, V, rank, adapters, rows of a request together
    (1, 64, 100, 4, 1, False), (1, 1, 1, 1, 1, False), (5, 33, 77, 3, 2, False), (64, 256, 1000, 16, 16, False),
    (65, 128, 2491, 8, 3, True), (130, 64, 256, 32, 1, True), (200, 96, 515, 17, 5, False),
    (300, 1088, 640, 33, 2, True), (40, 64, 8, 64, 40, False), (257, 72, 1111, 65, 2, True),
    (129, 40, 264, 128, 3, False), (700, 2560, 64, 9, 4, True), (3, 4001, 5003, 2, 200, False)]


@pytest.mark.parametrize("T,H,V,rank,n,runs", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_both_directions(T, H, V, rank, n, runs, dtype):
    for pad, skip in ((0, 0), (8, 8), (3, 1)):
        s = make(T, H, V, rank, n, dtype, T + V, pad, skip, runs)
        args = [s[k] for k in ("x", "down", "up", "of", "scale")]
        out = lm.adapters_forward(s["base"], *args)
        check_forward(s, out)
        bare = s["of"] < 0
        assert torch.equal(out[bare], s["base"][bare])
        grads = lm.adapters_backward(s["grad"], *args)
        check_backward(s, *grads)
        assert not grads[0][bare].any()
        # the same bits again, and in place
        assert torch.equal(out, lm.adapters_forward(s["base"], *args))
        assert all(torch.equal(a, b) for a, b in zip(grads, lm.adapters_backward(s["grad"], *args)))
        assert lm.adapters_forward(s["base"], *args, out=s["base"]) is s["base"]
        assert torch.equal(s["base"], out)


def test_one_adapter_without_ids_or_scale():
    s = make(100, 64, 300, 8, 1, F32, 1, bare=0.0)
    s["of"] = s["scale"] = None
    check_forward(s, lm.adapters_forward(s["base"], s["x"], s["down"], s["up"]))
    check_backward(s, *lm.adapters_backward(s["grad"], s["x"], s["down"], s["up"]))


def test_rows_without_an_adapter_and_adapters_without_rows():
    s = make(90, 64, 300, 8, 6, BF16, 2)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    s["of"].fill_(4)
    s["of"][::2] = -1
    s["of"][1::4] = 6
    s["of"][3] = 2 ** 31 - 1
    s["of"][7] = -2 ** 31
    s["x"][s["of"] != 4] = float("nan")       # rows that nobody looks at
    s["grad"][s["of"] != 4] = float("inf")
    out = lm.adapters_forward(s["base"], *args)
    clean = dict(s, x=torch.nan_to_num(s["x"]), grad=s["grad"].masked_fill(torch.isinf(s["grad"]), 0.0))
    check_forward(clean, out)
    grads = lm.adapters_backward(s["grad"], *args)
    check_backward(clean, *grads)
    assert not grads[1][:4].any() and not grads[1][5].any() and not grads[2][:4].any()
    s["of"].fill_(-1)                          # nobody at all
    assert torch.equal(lm.adapters_forward(s["base"], *args), s["base"])
    assert not any(t.any() for t in lm.adapters_backward(s["grad"], *args))


def test_results_that_are_added_to():
    s = make(150, 72, 333, 12, 3, F16, 3)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    g = torch.Generator("cuda").manual_seed(4)
    start = [torch.randn(t.shape, generator=g, device="cuda") for t in (s["x"], s["down"], s["up"])]
    mine = [t.clone() for t in start]
    lm.adapters_backward(s["grad"], *args, dx=mine[0], accumulate_dx=True, d_down=mine[1], d_up=mine[2],
                         accumulate=True)
    check_backward(s, *mine, *start)
    bare = s["of"] < 0
    assert torch.equal(mine[0][bare], start[0][bare])


def test_some_gradients_alone():
    s = make(150, 72, 333, 12, 3, F32, 5)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    want = lm.adapters_backward(s["grad"], *args)
    ws = torch.empty(lm.lmhead_adapters_workspace_size(150, 72, 333, 12, 3), dtype=torch.uint8, device="cuda")
    for pick in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
        got = [torch.full_like(t, 7.0) if p else None for t, p in zip(want, pick)]
        assert lm.lmhead_adapters_bwd(s["grad"], *args, got[0], False, got[1], got[2], False, ws) == 0
        for a, b in zip(got, want):
            assert a is None or torch.equal(a, b)


def test_more_rows_than_one_sort():
    T = 131072 + 700
    s = make(T, 8, 16, 2, 5, F32, 6)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    check_forward(s, lm.adapters_forward(s["base"], *args))
    check_backward(s, *lm.adapters_backward(s["grad"], *args), extra=2)


def test_no_rows():
    s = make(4, 16, 24, 2, 2, F32, 7)
    none = [s["x"][:0], s["down"], s["up"], s["of"][:0], s["scale"]]
    assert lm.adapters_forward(s["base"][:0], *none).shape == (0, 24)
    d = [torch.ones(t.shape, device="cuda") for t in (s["down"], s["up"])]
    lm.adapters_backward(s["grad"][:0], *none, d_down=d[0], d_up=d[1], accumulate=True)
    assert all((t == 1).all() for t in d)
    lm.adapters_backward(s["grad"][:0], *none, d_down=d[0], d_up=d[1])
    assert not any(t.any() for t in d)


@pytest.mark.parametrize("T,H,V,rank,n", [(1, 1, 1, 1, 1), (70, 33, 515, 5, 3), (64, 64, 512, 32, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_writes_stay_inside(T, H, V, rank, n, dtype):
    g = np.random.default_rng(T)
    gin = dict(x=Guarded((T, H), BF16, 81, torch.randn(T, H)), down=Guarded((n, rank, H), BF16, 82, torch.randn(n, rank, H)),
               up=Guarded((n, rank, V), BF16, 83, torch.randn(n, rank, V)),
               of=Guarded((T,), torch.int32, 84, torch.from_numpy(g.integers(-1, n, T).astype(np.int32))),
               scale=Guarded((n,), F32, 85, torch.randn(n)))
    t = [gin[k].t for k in ("x", "down", "up", "of", "scale")]
    ws = Guarded((lm.lmhead_adapters_workspace_size(T, H, V, rank, n),), torch.uint8, 86)
    base, out = Guarded((T, V), dtype, 87, torch.randn(T, V)), Guarded((T, V), dtype, 88)
    assert lm.lmhead_adapters_fwd(base.t, *t, out.t, ws.t) == 0
    _check(dict(gin, base=base), dict(out=out, ws=ws), "fwd")
    ws = Guarded((lm.lmhead_adapters_workspace_size(T, H, V, rank, n),), torch.uint8, 89)
    res = dict(dx=Guarded((T, H), F32, 90), d_down=Guarded((n, rank, H), F32, 91), d_up=Guarded((n, rank, V), F32, 92))
    assert lm.lmhead_adapters_bwd(base.t, *t, res["dx"].t, False, res["d_down"].t, res["d_up"].t, False, ws.t) == 0
    _check(dict(gin, base=base), dict(res, ws=ws), "bwd")


def test_offsets_past_32_bits():
    T, V = 70, 40_000_000
    base = torch.zeros(T, V, dtype=BF16, device="cuda")
    x = torch.ones(T, 8, dtype=BF16, device="cuda")
    down = torch.ones(2, 1, 8, dtype=BF16, device="cuda")
    up = torch.zeros(2, 1, V, dtype=BF16, device="cuda")
    up[1, 0, -3:] = 2.0
    of = torch.ones(T, dtype=torch.int32, device="cuda")
    lm.adapters_forward(base, x, down, up, of, out=base)
    assert (base[:, -3:] == 16).all() and not base[:, -6:-3].any() and not base[:, :4].any()
    dx, d_down, d_up = lm.adapters_backward(base, x, down, up, of)
    assert (dx == 96).all() and (d_up[1, 0, -3:] == 16 * 8 * T).all() and not d_up[0].any()
    assert (d_down[1] == 96 * T).all()


def test_autograd():
    s = make(120, 64, 200, 6, 3, BF16, 9)
    leaves = [s[k].clone().requires_grad_(True) for k in ("base", "x", "down", "up")]
    out = autograd.adapters(*leaves, s["of"], s["scale"])
    check_forward(s, out)
    g = rows((200, 120), BF16, torch.Generator("cuda").manual_seed(1)).t()     # handed over transposed
    got = torch.autograd.grad(out, leaves, g)
    assert [t.dtype for t in got] == [BF16] * 4 and torch.equal(got[0], g)
    want = lm.adapters_backward(g.contiguous(), s["x"], s["down"], s["up"], s["of"], s["scale"])
    for a, b in zip(got[1:], want):
        assert torch.equal(a, b.to(BF16))
    only, = torch.autograd.grad(autograd.adapters(s["base"], s["x"], leaves[2], s["up"], s["of"]).float().sum(),
                                leaves[2])
    assert only.shape == s["down"].shape
    first = torch.autograd.grad(autograd.adapters(*leaves, s["of"]).float().square().sum(), leaves[1],
                                create_graph=True)[0]
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.float().sum(), leaves[1])


def test_gradients_against_differences():
    """The share is linear in each factor: differences over a whole step, which bf16 holds exactly."""
    s = make(50, 32, 90, 4, 2, F32, 10)
    s["base"].zero_()
    for k in ("x", "down", "up"):                       # few bits, so that sums of two are exact
        s[k] = (torch.round(4 * s[k].float()).clamp(-8, 8) / 4).to(BF16)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    grads = lm.adapters_backward(s["grad"], *args)
    for i in range(3):
        step = torch.ones_like(args[i])
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - step, args[i] + step
        change = (lm.adapters_forward(s["base"], *hi).double() - lm.adapters_forward(s["base"], *lo).double())
        got = float((change * s["grad"].double()).sum())
        want = 2 * float(grads[i].double().sum())
        size = float((change.abs() * s["grad"].double().abs()).sum()) + 2 * float(grads[i].double().abs().sum())
        assert abs(got - want) <= off(32 + 90 + 6 * 50) * 40 * size


def test_streams_and_graphs():
    s = make(200, 128, 1000, 16, 4, BF16, 11)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    calls = (lambda **k: (lm.adapters_forward(s["base"], *args, **k),),
             lambda **k: lm.adapters_backward(s["grad"], *args, **k))
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        side.wait_stream(torch.cuda.current_stream())
        for stream in (side, side.cuda_stream):
            got = call(stream=stream)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [call() for call in calls]
        graphs.append((graph, out))
    s["of"].copy_(torch.randint(-1, 4, (200,), device="cuda"))
    s["x"].copy_(torch.randn(200, 128, device="cuda"))
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = [call() for call in calls]
    for _, out in graphs:
        assert all(torch.equal(a, b) for x, y in zip(out, want) for a, b in zip(x, y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shares", ["few", "one", "half", "none", "runs"])
def test_many_adapters_whatever_their_shares(dtype, shares):
    """Rows of far more adapters than most batches use: the multiplying kernel is chosen by what
    the batch holds."""
    for T, n, pad, skip in ((129, 17, 0, 0), (300, 64, 8, 8), (300, 200, 3, 1), (1500, 600, 0, 0)):
        s = make(T, 96, 520, 12, n, dtype, T + n, pad, skip)
        if shares == "one":
            s["of"].fill_(n // 2)
        elif shares == "half":
            s["of"][::2] = n - 1
        elif shares == "none":
            s["of"][1:] = -1
        elif shares == "runs":       # four and five rows each, around the bound of both choices
            s["of"].copy_(torch.arange(T, device="cuda") // 4 % n)
            s["of"][: T // 2] = torch.arange(T // 2, device="cuda", dtype=torch.int32) // 13 % n
        args = [s[k] for k in ("x", "down", "up", "of", "scale")]
        out = lm.adapters_forward(s["base"], *args)
        check_forward(s, out)
        bare = s["of"] < 0
        assert torch.equal(out[bare], s["base"][bare])
        grads = lm.adapters_backward(s["grad"], *args)
        check_backward(s, *grads)
        assert not grads[0][bare].any()
        assert torch.equal(lm.adapters_forward(s["base"], *args, out=s["base"]), out)


def test_more_rows_than_one_sort_of_many_adapters():
    s = make(131072 + 300, 16, 40, 3, 20000, F32, 11)
    s["of"][131072:] = 19999
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    check_forward(s, lm.adapters_forward(s["base"], *args))


def test_a_captured_call_replayed_with_other_rows():
    """What multiplies is chosen on the device, so that a captured call holds for any ids."""
    s = make(300, 96, 520, 12, 64, F32, 12)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    out = torch.empty_like(s["base"])
    ws = torch.empty(lm.lmhead_adapters_workspace_size(300, 96, 520, 12, 64), dtype=torch.uint8, device="cuda")
    lm.adapters_forward(s["base"], *args, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.adapters_forward(s["base"], *args, out=out, workspace=ws)
    for ids in (s["of"].clone(), torch.full_like(s["of"], 5), torch.full_like(s["of"], -1),
                torch.arange(300, device="cuda", dtype=torch.int32) // 9):
        s["of"].copy_(ids)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_forward(s, out)
