"""Adapters whose operands hold infinities, NaN and the largest fp32 numbers."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built
from operators_reference import U32, f64

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def rows(values, dtype, pad, skip):
    n, h = values.shape
    t = torch.zeros(skip + n * (h + pad), dtype=dtype, device="cuda")[skip:].view(n, h + pad)[:, :h]
    t.copy_(values.to("cuda"))
    return t


def make(T, H, V, rank, n, dtype, pad=0, skip=0):
    """Small multiples of powers of two: u has up to 12 bits, so more than one bf16 part of either
    sign, and every finite sum is exact in fp32 (below 2^24 of its steps)."""
    g = torch.Generator().manual_seed(T + V + rank)

    def few(shape, most, step):
        return torch.randint(-most, most + 1, shape, generator=g) * step

    of = torch.randint(-1, n, (T,), generator=g)
    return dict(x=rows(few((T, H), 3, 1.0), BF16, pad, skip), of=of.to(torch.int32).cuda(),
                down=few((n, rank, H), 15, 0.125).to(BF16).cuda(), up=few((n, rank, V), 2, 1.0).to(BF16).cuda(),
                scale=torch.tensor([0.5, -2.0, 1.0])[:n].cuda(),
                base=rows(few((T, V), 8, 1.0), dtype, pad, skip), grad=rows(few((T, V), 4, 0.25), dtype, pad, skip))


def product(a, b):
    """a [i, k] times b [k, j], every product formed (a library may pass over zeros)."""
    return np.stack([(row[:, None] * b).sum(0) for row in a]) if len(a) else np.zeros((0, b.shape[1]))


def formula(s):
    x, base, grad = (f64(s[k]) for k in ("x", "base", "grad"))
    out, dx = base.copy(), np.zeros(x.shape)
    d_down, d_up = (np.zeros(s[k].shape) for k in ("down", "up"))
    of, scale = s["of"].cpu().numpy(), f64(s["scale"])
    with np.errstate(invalid="ignore"):
        for a in range(len(d_up)):
            at = np.flatnonzero(of == a)
            if not len(at):
                continue
            down, up = f64(s["down"])[a], f64(s["up"])[a]
            u, du = scale[a] * product(x[at], down.T), scale[a] * product(grad[at], up.T)
            out[at] += product(u, up)
            dx[at] = product(du, down)
            d_down[a], d_up[a] = product(du.T, x[at]), product(u.T, grad[at])
    return out, dx, d_down, d_up


def same(name, got, want):
    want = torch.from_numpy(want).to(got.dtype).cuda()       # exact before the one rounding
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    assert torch.equal(torch.nan_to_num(got, nan=0.0, posinf=1e30, neginf=-1e30) if got.dtype is F32 else got[~got.isnan()],
                       torch.nan_to_num(want, nan=0.0, posinf=1e30, neginf=-1e30) if got.dtype is F32
                       else want[~want.isnan()]), name


def check(s):
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    want = formula(s)
    same("out", lm.adapters_forward(s["base"], *args), want[0])
    grads = lm.adapters_backward(s["grad"], *args)
    for name, t, w in zip(("dx", "d_down", "d_up"), grads, want[1:]):
        same(name, t, w)
    d_up = torch.ones_like(grads[2])
    lm.adapters_backward(s["grad"], *args, d_up=d_up, accumulate=True)
    same("d_up added", d_up, want[3] + 1.0)


SIZES = [(90, 40, 152, 5, 3), (70, 33, 151, 20, 2), (130, 64, 264, 40, 1), (60, 24, 72, 70, 2),
         (1300, 16, 40, 3, 1)]      # the last in several row splits


@pytest.mark.parametrize("T,H,V,rank,n", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_an_infinite_cotangent_goes_through_as_in_the_formula(T, H, V, rank, n, dtype):
    for pad, skip in ((0, 0), (3, 1)):
        s = make(T, H, V, rank, n, dtype, pad, skip)
        check(s)
        s["grad"][3::17, ::5] = INF
        check(s)
        s["grad"][5::19, 1::5] = -INF
        s["grad"][3, 0] = -INF               # both signs in one column
        s["grad"][7, 2] = NAN
        check(s)


@pytest.mark.parametrize("T,H,V,rank,n", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_infinite_rows_of_x_go_through_as_in_the_formula(T, H, V, rank, n, dtype):
    for pad, skip in ((0, 0), (3, 1)):
        s = make(T, H, V, rank, n, dtype, pad, skip)
        s["x"][2::23, 3] = INF
        s["x"][4, 0] = -INF
        s["x"][9, 1] = NAN
        check(s)
        s["grad"][6::29, ::7] = -INF
        check(s)


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("V", [96, 51])
def test_numbers_next_to_the_largest(T, V):
    """u and the cotangent above the largest bf16 number, which is not the largest fp32 number."""
    most = torch.finfo(F32).max
    s = make(T, 16, V, 4, 1, F32)
    s["of"].zero_()
    s["scale"].fill_(1.0)
    s["x"].zero_()
    s["x"][:, 0] = torch.finfo(BF16).max
    s["x"][:, 1] = 1.0e36                    # u = 3.3995e38: bf16 would round it to infinity
    s["down"].zero_()
    s["down"][:, :, :2] = 1.0
    s["down"][:, 1] *= -1.0
    s["up"].fill_(2.0 ** -20)
    s["base"].zero_()
    s["grad"].zero_()
    s["grad"][:, 0] = most
    s["grad"][:, 1] = -3.398e38
    s["up"][:, :, 1] = 2.0 ** -30
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    u = f64(s["x"]) @ f64(s["down"])[0].T
    assert (np.abs(u) > torch.finfo(BF16).max).all() and (np.abs(u) < most).all()
    # u and du: two products of powers of two and one rounding; three parts; sums of four
    out = f64(lm.adapters_forward(s["base"], *args))
    want = u @ f64(s["up"])[0]
    size = np.abs(u) @ np.abs(f64(s["up"])[0])
    assert (np.abs(out - want) <= 16 * U32 * size).all()
    dx, d_down, _ = lm.adapters_backward(s["grad"], *args)
    du = f64(s["grad"]) @ f64(s["up"])[0].T
    size = np.abs(f64(s["grad"])) @ np.abs(f64(s["up"])[0].T)
    assert (np.abs(f64(dx) - du @ f64(s["down"])[0]) <= 16 * U32 * size @ np.abs(f64(s["down"])[0])).all()
    s["x"].fill_(0.0)
    s["x"][:, 0] = 2.0 ** -12
    _, d_down, _ = lm.adapters_backward(s["grad"], *args)
    want = du.T @ f64(s["x"])
    assert (np.abs(f64(d_down)[0] - want) <= (16 + 2 * T) * U32 * (size.T @ np.abs(f64(s["x"])))).all()
