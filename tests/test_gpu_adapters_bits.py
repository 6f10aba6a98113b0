"""Adapters use every bit of fp32 u, du and cotangents in fp32 results.

Every sum here has one product that is not zero and one factor of it that is a power of two (or both
have all their bits, where it says so).  So nothing hides behind the magnitude of a sum: a result is
that product, rounded once where it needs more than 24 bits, and each of up to six partial products
added on the way may lose one unit in the last place (2^-23 of the result).  A number cut to two bf16
parts would be off by up to 2^-17, in most cases by more than 2^-20."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EXACT = 2.0 ** -22        # one factor a power of two: three parts, each added once
BOTH = 2.0 ** -20         # both with 24 bits: six products, and three left out below 2^-26 in all


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def powers(shape, g):
    """+-2^k, k in -3 .. 3."""
    k = torch.randint(-3, 4, shape, generator=g, device="cuda")
    return torch.ldexp(torch.randint(0, 2, shape, generator=g, device="cuda") * 2.0 - 1.0, k)


def two_parts(x):
    first = x.to(BF16).double()
    return first + (x.double() - first).to(BF16).double()


def full(shape, g):
    """Numbers of either sign with 24 bits, between 1 and 2 in size: of 16 each the one that two parts
    hold worst."""
    m = torch.randint(2 ** 23, 2 ** 24, (16, *shape), generator=g, device="cuda").double() * 2.0 ** -23
    m = m.gather(0, (two_parts(m.float()) - m).abs().argmax(0, keepdim=True))[0]
    return (m * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1)).float()


def close(got, want, tol):
    """want in 64 bits; zeros are exact."""
    assert got.dtype is F32
    assert (got.double() - want).abs().le(tol * want.abs()).all(), \
        float(((got.double() - want).abs() / want.abs().clamp_min(1e-300)).max())


def shows(x, tol):
    """The numbers are such that two parts of them would not pass."""
    x = x[x != 0]
    assert (two_parts(x) - x.double()).abs().gt(tol * x.double().abs()).float().mean() > 0.5


# T rows, an adapter each (or all the same): x_t = 2^k e_t, so that one row is one column of d_down
CASES = [(64, 64, 64, 16, 1), (50, 51, 77, 5, 1), (40, 64, 128, 33, 1), (24, 40, 104, 70, 1), (60, 64, 64, 8, 60),
         (200, 200, 264, 16, 200), (1024, 1024, 1032, 3, 1)]


@pytest.mark.parametrize("T,H,V,rank,n", CASES)
def test_u_keeps_its_bits(T, H, V, rank, n):
    """u_t = scale 2^k with 24 bits of scale, in one rank of each row."""
    g = torch.Generator("cuda").manual_seed(T + V)
    of = torch.arange(T, device="cuda", dtype=torch.int32) % n
    scale = full((n,), g)
    row = torch.arange(T, device="cuda")
    x = torch.zeros(T, H, device="cuda")
    x[row, row] = powers((T,), g)
    down = torch.zeros(n, rank, H, device="cuda")
    down[of.long(), row % rank, row] = powers((T,), g)
    up = powers((n, rank, V), g)
    args = [t.to(BF16) for t in (x, down, up)]
    u = torch.zeros(T, rank, dtype=torch.float64, device="cuda")
    u[row, row % rank] = scale.double()[of.long()] * x[row, row].double() * down[of.long(), row % rank, row].double()
    shows(u.float(), EXACT)
    zero = torch.zeros(T, V, device="cuda")
    out = lm.adapters_forward(zero, *args, of, scale)
    close(out, (u[:, :, None] * up.double()[of.long()]).sum(1), EXACT)
    for dtype in (F32, BF16, F16):          # the gradient of up, by rows whose cotangents do not meet
        grad = torch.zeros(T, V, device="cuda")
        grad[row, row % V] = powers((T,), g)
        keep = row < V
        d_up = lm.adapters_backward(grad.to(dtype)[keep], args[0][keep], *args[1:], of[keep], scale)[2]
        want = torch.zeros(n, rank, V, dtype=torch.float64, device="cuda")
        want[of.long()[keep], :, row[keep]] = u[keep] * grad[row, row % V].double()[keep, None]
        close(d_up, want, EXACT)


@pytest.mark.parametrize("T,H,V,rank,n", CASES)
def test_cotangents_and_du_keep_their_bits(T, H, V, rank, n):
    g = torch.Generator("cuda").manual_seed(T + V + 1)
    of = torch.arange(T, device="cuda", dtype=torch.int32) % n
    row = torch.arange(T, device="cuda")
    col = row * 7 % V if V % 7 else row * 5 % V
    for dtype in (F32, F16):
        grad = torch.zeros(T, V, device="cuda")
        grad[row, col] = full((T,), g)
        grad = grad.to(dtype)
        at = grad[row, col].double()
        if dtype is F32:
            shows(grad, EXACT)
        x = torch.zeros(T, H, device="cuda")
        x[row, row] = powers((T,), g)
        up, down = powers((n, rank, V), g), torch.zeros(n, rank, H, device="cuda")
        down[:, 0] = powers((n, H), g)      # one rank reaches dx
        args = [t.to(BF16) for t in (x, down, up)]
        dx, d_down, _ = lm.adapters_backward(grad, *args, of)
        du = at[:, None] * up.double()[of.long(), :, col]          # [T, rank]
        close(dx, du[:, :1] * down.double()[of.long(), 0], EXACT)
        want = torch.zeros(n, rank, H, dtype=torch.float64, device="cuda")
        want[of.long(), :, row] = du * x[row, row].double()[:, None]
        close(d_down, want, EXACT)
        scale = full((n,), g)               # du rounded once, then every bit of it
        dx = lm.adapters_backward(grad, *args, of, scale)[0]
        close(dx, scale.double()[of.long(), None] * du[:, :1] * down.double()[of.long(), 0], EXACT)


@pytest.mark.parametrize("T,H,V,rank,n", CASES)
def test_u_times_cotangent_with_all_bits_of_both(T, H, V, rank, n):
    g = torch.Generator("cuda").manual_seed(T + V + 2)
    T = min(T, V)
    of = torch.arange(T, device="cuda", dtype=torch.int32) % n
    row = torch.arange(T, device="cuda")
    x, grad = torch.zeros(T, H, device="cuda"), torch.zeros(T, V, device="cuda")
    x[row, row] = powers((T,), g)
    grad[row, row] = full((T,), g)
    down, up, scale = powers((n, rank, H), g), powers((n, rank, V), g), full((n,), g)
    d_up = lm.adapters_backward(grad, x.to(BF16), down.to(BF16), up.to(BF16), of, scale)[2]
    u = scale.double()[of.long(), None] * x[row, row].double()[:, None] * down.double()[of.long(), :, row]
    want = torch.zeros(n, rank, V, dtype=torch.float64, device="cuda")
    want[of.long(), :, row] = u * grad[row, row].double()[:, None]
    shows(u.float(), BOTH)
    shows(grad, BOTH)
    close(d_up, want, BOTH)
