"""Sizes that reach the kernels' variants and loops which ordinary sizes do not: layer norm of
many short and of many unaligned rows, logit processing of a vocabulary wider than one CTA
handles and of more rows than a grid has, the distillation loss of more rows than CTAs.
References and tolerances are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm

import operators_reference as ref
from gpu_helpers import ensure_built
from test_gpu_distill import check_logits
from test_gpu_layernorm import DT, check_bwd, check_fwd, inputs, rows
from test_gpu_process_logits import check, cu, padded, rules, sizes, wide

pytestmark = pytest.mark.gpu

F32, BF16, F16 = "float32", "bfloat16", "float16"


# ------------------------------------------------------------------ layer norm, 608 rows and more
@pytest.mark.parametrize("n,h", [(608, 8), (611, 64), (700, 512), (1001, 1000), (650, 1024), (620, 504)])
@pytest.mark.parametrize("x_type,p_type,y_type", [(F32, F32, F32), (F32, F32, BF16), (BF16, BF16, BF16),
                                                  (BF16, F32, BF16), (F16, F16, F16)])
def test_layernorm_of_many_short_rows(n, h, x_type, p_type, y_type):
    """Up to 128 packs of 16 bytes: one warp per row, four rows per CTA, the last CTA's not all
    there.  (1,024 fp32 columns are more than that.)"""
    ensure_built()
    x, w, b = inputs(n, h, x_type, p_type, 3 * n + h, bias=h % 16 == 0)
    y, mean, rstd = lm.layernorm_forward(x, w, b, 1e-5, DT[y_type])
    check_fwd(x, w, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("n,h,pad,shift", [(700, 1111, 0, 0), (608, 37, 0, 0), (640, 4095, 0, 0),
                                           (615, 1, 0, 0), (900, 512, 3, 0), (610, 2560, 0, 1),
                                           (5000, 129, 1, 3)])
@pytest.mark.parametrize("x_type,y_type", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16)])
def test_layernorm_of_many_unaligned_rows(n, h, pad, shift, x_type, y_type):
    """Odd widths, strides and starts: single elements, through the ring for fp32 rows."""
    ensure_built()
    x, w, b = inputs(n, h, x_type, F32, n + 7 * h, pad, shift, bias=n % 2 == 0)
    y = rows(torch.zeros(n, h), pad, shift, DT[y_type])
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    assert lm.lmhead_layernorm_fwd(x, w, b, 1e-5, y, mean, rstd) == 0
    check_fwd(x, w, b, 1e-5, y, mean, rstd)
    dy = rows(torch.randn(n, h, generator=torch.Generator().manual_seed(1)), pad, shift, DT[x_type])
    dx, dw, db = lm.layernorm_backward(dy, x, w, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, dx, dw, db)


# ------------------------------------------------------------------ logit processing
def process_both(R, V, n, dtype, seed, **some):
    r = np.random.default_rng(seed)
    z = padded((r.normal(size=(R, V)) * 3).astype(np.float32), 0, 0, DT[dtype])
    k = rules(R, V, n, seed + 1, **some)
    c, w, X = cu(k), wide(k), ref.f64(z)
    want, size = ref.process_fwd(X, **w), sizes(X, w)
    out = lm.process_logits(z, **c)
    check(out, want, size, dtype)
    few = [m for m in ("tokens", "spans", "repetition", "allowed", "allowed_rows") if m in k]
    g = padded(r.normal(size=(R, V)).astype(np.float32), 0, 0, DT[dtype])
    d = lm.process_logits_backward(g, z, **{m: c[m] for m in few})
    check(d, ref.process_bwd(ref.f64(g), X, **{m: w[m] for m in few}), 2 * np.abs(ref.f64(g)), dtype)
    lm.process_logits_backward(g, z, **{m: c[m] for m in few}, d_logits=g)
    lm.process_logits(z, **c, out=z)                    # in place
    assert torch.equal(out, z) and torch.equal(d, g)
    return k, c


@pytest.mark.parametrize("V,n", [(262145, 3000), (300000, 9000), (600001, 20000)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("grammar", [False, True])
def test_processing_of_a_vocabulary_in_several_ranges(V, n, dtype, grammar):
    """262,144 columns per CTA: ids and biases on both sides of every border."""
    ensure_built()
    k, _ = process_both(4, V, n, dtype, V % 1000, grammar=grammar)
    for ids in (k["tokens"], k["bias_ids"]):
        assert (ids < 262144).any()
    assert V < 300000 or (k["tokens"] >= 262144).any() and (k["bias_ids"] >= 262144).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_processing_of_ids_at_a_ranges_border(dtype):
    ensure_built()
    edge = 262144
    V = 2 * edge + 3
    tokens = np.array([edge - 1, edge, edge, 2 * edge - 1, 2 * edge, V - 1, V, 0, -1], np.int32)
    k = dict(tokens=tokens, spans=np.array([[0, 2, 9], [0, 0, 9]], np.int64),
             repetition=np.array([1.5, 1.25], np.float32), frequency=np.array([0.5, 0.25], np.float32),
             presence=np.array([1.0, 2.0], np.float32), bias_offsets=np.array([0, 3, 4], np.int64),
             bias_ids=np.array([edge, edge - 1, edge, V - 1], np.int32),
             bias_values=np.array([9.0, 3.0, 4.0, -2.0], np.float32))
    z = padded((np.random.default_rng(5).normal(size=(2, V)) * 3).astype(np.float32), 0, 0, DT[dtype])
    w, X = wide(k), ref.f64(z)
    check(lm.process_logits(z, **cu(k)), ref.process_fwd(X, **w), sizes(X, w), dtype)


@pytest.mark.parametrize("V", [96, 101])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("grammar", [False, True])
def test_processing_of_more_rows_than_the_grid(V, dtype, grammar):
    """32,768 rows are in flight at most; CTAs take a second one, histories or none."""
    ensure_built()
    process_both(33100, V, 30, dtype, V, grammar=grammar)


# ------------------------------------------------------------------ distillation, forward
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distillation_loss_of_more_rows_than_ctas(dtype):
    """2^20 CTAs at most: the first ones take a second row, some of them unscored."""
    ensure_built()
    T, V, K = (1 << 20) + 70, 8, 2
    r = np.random.default_rng(3)
    ids = r.integers(-V, V, size=(T, K)).astype(np.int32)
    a = (r.normal(size=(T, K)) * 2).astype(np.float32)
    a[r.random((T, K)) < 0.1] = -np.inf
    mask = (r.random(T) > 0.3).astype(np.uint8)
    z = padded((r.normal(size=(T, V)) * 2).astype(np.float32), 1, 0, DT[dtype])
    grad = r.normal(size=T).astype(np.float32)
    c = lambda v: torch.from_numpy(v).cuda()   # noqa: E731
    loss, lse = lm.distill_logits_forward(z, c(ids), c(a), c(mask), 0.7)
    d = lm.distill_logits_backward(z, c(ids), c(a), c(mask), 0.7, 1.0, c(grad), lse)
    for part in (slice(0, 200), slice(T - 200, T)):
        check_logits(z[part], ids[part], a[part].astype(np.float64), 0.7, 1.0, None, mask[part],
                     grad[part].astype(np.float64), loss[part], lse[part], d[part], dtype)
