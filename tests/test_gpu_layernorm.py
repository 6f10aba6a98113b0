"""Layer norm forward and backward against the 64-bit definition.

Tolerances, from the arithmetic (u = 2^-24): a sum of n terms added in chains of
at most D is off by at most D u sum|.|; every other fp32 step adds a few u of
its operands; the result is rounded once to its type (unit roundoff of the
type).  D = H / 128 + 64 covers the row sums, D = N / 8 + 64 the column sums."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd

import operators_reference as ref
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
U = ref.U32


def rows(t, pad, shift, dtype):
    """t on the GPU as dtype, rows `pad` elements further apart, `shift` elements into its buffer."""
    n, h = t.shape
    buf = torch.full((shift + n * (h + pad),), 7.0, dtype=dtype, device="cuda")
    v = buf[shift:].view(n, h + pad)[:, :h]
    v.copy_(t.to(dtype))
    return v


def inputs(n, h, x_type, p_type, seed, pad=0, shift=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, generator=g) * 2 + torch.randn(n, 1, generator=g)
    if n > 2:
        x[1] += 300.0          # the mean far above the spread
        x[2] = 3.25            # no spread at all
    w = 1 + 0.3 * torch.randn(h, generator=g)
    b = torch.randn(h, generator=g) if bias else None
    return (rows(x, pad, shift, DT[x_type]), w.to(DT[p_type]).cuda(),
            None if b is None else b.to(DT[p_type]).cuda())


def check_fwd(x, w, b, eps, y, mean, rstd):
    n, h = x.shape
    X, W, B = ref.f64(x), ref.f64(w), ref.f64(b)
    ey, em, er = ref.norm_fwd(X, W, B, eps)
    D = (h / 128 + 64) * U
    mabs = np.abs(X).mean(1) + 1e-30
    tm = D * mabs
    assert (np.abs(ref.f64(mean) - em) <= tm).all()
    # rstd: relative error of the mean square about a mean that is itself off by tm
    spread = 1 / er ** 2
    tr = er * (2 * D + 4 * U * mabs / np.sqrt(spread) + tm ** 2 / spread)
    assert (np.abs(ref.f64(rstd) - er) <= tr).all()
    xh = np.abs(X - em[:, None]) * er[:, None]
    ty = np.abs(W) * (er[:, None] * (tm[:, None] + 2 * U * np.abs(X)) + xh * (tr / er + 4 * U)[:, None])
    ty += 4 * U * (np.abs(ey) + (0 if B is None else np.abs(B)))
    name = str(y.dtype).split(".")[1]
    ty = ty * (1 + ref.UNIT[name]) + ref.UNIT[name] * np.abs(ey) + ref.TINY[name]
    assert (np.abs(ref.f64(y) - ey) <= ty).all()


def check_bwd(dy, x, w, mean, rstd, dx, dw, db, dw0=None, db0=None):
    n, h = x.shape
    X, W, G, m, r = (ref.f64(t) for t in (x, w, dy, mean, rstd))
    ex, ew, eb = ref.norm_bwd(G, X, W, m, r)
    m, r = m[:, None], r[:, None]
    D = (h / 128 + 64) * U
    H_, xh = np.abs(G * W), np.abs(X - m) * r
    exh = 2 * U * (np.abs(X) + np.abs(m)) * r + 2 * U * xh            # error of xh
    if dx is not None:
        c1, c2 = (H_ * xh).mean(1, keepdims=True), H_.mean(1, keepdims=True)
        tx = r * (4 * U * H_ + (D + 4 * U) * c2 + xh * (D + 4 * U) * c1
                  + xh * (H_ * exh).mean(1, keepdims=True) + exh * c1)
        name = str(dx.dtype).split(".")[1]
        tx = 2 * tx + ref.UNIT[name] * np.abs(ex) + ref.TINY[name]
        assert (np.abs(ref.f64(dx) - ex) <= tx).all()
    D = (n / 8 + 64) * U
    for got, want, size, start in ((dw, ew, (np.abs(G) * (D * xh + exh)).sum(0), dw0),
                                   (db, eb, D * np.abs(G).sum(0), db0)):
        if got is None:
            continue
        if start is not None:
            want = want + ref.f64(start)
            size = size + 2 * U * (np.abs(ref.f64(start)) + np.abs(want))
        assert (np.abs(ref.f64(got) - want) <= size + 2 * U * np.abs(want) + 1e-38).all()


SHAPES = [(1, 1), (1, 2560), (3, 7), (5, 1111), (33, 64), (300, 1000), (1500, 2560), (700, 4096),
          (9, 8192), (640, 8192), (640, 8200), (615, 12288), (7, 20000), (2, 70001), (1, 70008)]
TYPES = [("float32", "float32", "float32"), ("bfloat16", "bfloat16", "float32"),
         ("bfloat16", "float32", "bfloat16"), ("float16", "float16", "float16"),
         ("float32", "float32", "bfloat16"), ("float16", "float32", "float32")]


@pytest.mark.parametrize("n,h", SHAPES)
@pytest.mark.parametrize("x_type,p_type,g_type", TYPES)
def test_both_directions(n, h, x_type, p_type, g_type):
    ensure_built()
    bias = (n + h) % 2 == 0
    x, w, b = inputs(n, h, x_type, p_type, 10 * n + h, bias=bias)
    y, mean, rstd = lm.layernorm_forward(x, w, b, 1e-5)
    check_fwd(x, w, b, 1e-5, y, mean, rstd)
    dy = rows(torch.randn(n, h, generator=torch.Generator().manual_seed(5)), 0, 0, DT[g_type])
    dx, dw, db = lm.layernorm_backward(dy, x, w, mean, rstd, with_bias=bias)
    check_bwd(dy, x, w, mean, rstd, dx, dw, db)
    again = lm.layernorm_backward(dy, x, w, mean, rstd, with_bias=bias)
    for p, q in zip((dx, dw, db), again):
        assert p is None or torch.equal(p, q)          # the same bits every time


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("x_type,g_type", [("bfloat16", "float32"), ("float32", "float32"),
                                           ("float16", "float16")])
@pytest.mark.parametrize("h", [256, 1001, 2560])
def test_strides_and_alignment(pad, shift, x_type, g_type, h):
    ensure_built()
    n = 40
    x, w, b = inputs(n, h, x_type, "float32", 77, pad, shift)
    w, b = rows(w[None], 0, shift, torch.float32)[0], rows(b[None], 0, 1, torch.float32)[0]
    y = rows(torch.zeros(n, h), pad + 1, shift, DT[x_type])
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    assert lm.lmhead_layernorm_fwd(x, w, b, 1e-6, y, mean, rstd) == 0
    check_fwd(x, w, b, 1e-6, y, mean, rstd)
    dy = rows(torch.randn(n, h, generator=torch.Generator().manual_seed(6)), pad, shift, DT[g_type])
    dx = rows(torch.zeros(n, h), 2, 1, DT[x_type])
    lm.layernorm_backward(dy, x, w, mean, rstd, dx=dx)
    _, dw, db = lm.layernorm_backward(dy, x, w, mean, rstd, dx=dx)
    check_bwd(dy, x, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("h", [512, 999, 9001, 12288])
def test_accumulate_in_place_and_partial_outputs(h):
    ensure_built()
    n = 200
    x, w, b = inputs(n, h, "float32", "float32", 3)
    _, mean, rstd = lm.layernorm_forward(x, w, b)
    dy = torch.randn(n, h, device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    ws = torch.empty(lm.lmhead_layernorm_workspace_size(n, h), dtype=torch.uint8, device="cuda")
    dw0, db0 = torch.full((h,), 3.0, device="cuda"), torch.full((h,), -2.0, device="cuda")
    dw, db, dx = dw0.clone(), db0.clone(), dy.clone()
    assert lm.lmhead_layernorm_bwd(dx, x, w, mean, rstd, dx, dw, db, True, ws) == 0   # dx over dy
    check_bwd(dy, x, w, mean, rstd, dx, dw, db, dw0, db0)
    x2 = x.clone()
    assert lm.lmhead_layernorm_bwd(dy, x2, w, mean, rstd, x2, dw, None, False, ws) == 0  # dx over x
    check_bwd(dy, x, w, mean, rstd, x2, dw, None)
    only = torch.empty_like(dx)
    assert lm.lmhead_layernorm_bwd(dy, x, w, mean, rstd, only, None, None, False, None) == 0
    check_bwd(dy, x, w, mean, rstd, only, None, None)
    if h <= 4096:          # wider rows without a workspace form their sums in another order
        assert torch.equal(only, dx)
    assert lm.lmhead_layernorm_bwd(dy, x, w, mean, rstd, None, None, db, False, ws) == 0
    check_bwd(dy, x, w, mean, rstd, None, None, db)


def test_no_rows():
    ensure_built()
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = lm.layernorm_forward(x, w)
    assert y.shape == (0, 64)
    dx, dw, db = lm.layernorm_backward(x, x, w, mean, rstd)
    assert (dw == 0).all() and (db == 0).all()


def test_fp32_rows_to_bf16_and_autograd():
    ensure_built()
    n, h = 130, 320
    x, w, b = inputs(n, h, "float32", "float32", 4)
    y, mean, rstd = lm.layernorm_forward(x, w, b, 1e-5, torch.bfloat16)
    assert y.dtype == torch.bfloat16
    check_fwd(x, w, b, 1e-5, y, mean, rstd)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    out = autograd.layer_norm(*leaves, 1e-5, torch.bfloat16)
    assert torch.equal(out, y)
    g = torch.randn(n, h, device="cuda").to(torch.bfloat16)
    dx, dw, db = torch.autograd.grad(out, leaves, g)
    check_bwd(g, x, w, mean, rstd, dx, dw, db)


def test_gradient_against_differences():
    """The GPU's gradient along a direction against central differences of the 64-bit
    definition (step 1e-4: truncation and cancellation below 1e-6 of the terms' sum)."""
    ensure_built()
    n, h = 6, 200
    g = torch.Generator().manual_seed(9)
    x, w, b = inputs(n, h, "float32", "float32", 12)
    x = torch.randn(n, h, generator=g).cuda()
    dy = torch.randn(n, h, generator=g).cuda()
    _, mean, rstd = lm.layernorm_forward(x, w, b)
    dx, dw, db = lm.layernorm_backward(dy, x, w, mean, rstd)
    X, W, B, G = (ref.f64(t) for t in (x, w, b, dy))
    r = np.random.default_rng(1)
    for d, at, got in ((r.normal(size=X.shape), 0, dx), (r.normal(size=h), 1, dw),
                       (r.normal(size=h), 2, db)):
        def f(s):
            a = [X, W, B]
            a[at] = a[at] + s * d
            return (ref.norm_fwd(*a, 1e-5)[0] * G).sum()
        want = (f(1e-4) - f(-1e-4)) / 2e-4
        size = np.abs(ref.f64(got) * d).sum()
        assert abs((ref.f64(got) * d).sum() - want) <= 2e-5 * size
