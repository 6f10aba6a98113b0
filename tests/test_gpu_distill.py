"""Distillation from a teacher's top logits, on held logits and through the
head, against the 64-bit definition.

Tolerances for held logits (u = 2^-24).  lse: the exponents are off by a few u of
the scaled logits, ex2 by 2^-22 of its value, the sum of V positive terms by at
most (V / 256 + 32) u.  Loss: that, times P, and a few u of every number that
enters sum p (log p - z + lse).  Gradient: g P q and g p, q off by 2^-21 and 8 u
of its exponent's operands, then one rounding to the output type.  Through the
head the tolerances are the head's own: 1e-3 on lse, 2e-3 on the loss (times
P), 1e-2 relative Frobenius on gradients (bf16 cotangents)."""
import os

import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd

import operators_reference as ref
from gpu_helpers import LIMITS, ensure_built, rel_fro

pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
U = ref.U32


def teacher(T, V, K, seed, odd=True):
    """ids and teacher logits with absent entries, whole absent rows, repeats and negative ids."""
    r = np.random.default_rng(seed)
    ids = np.stack([r.choice(V, size=K, replace=K > V) for _ in range(T)]).astype(np.int32)
    a = (r.normal(size=(T, K)) * 2 + 5).astype(np.float32)
    a[r.random((T, K)) < 0.1] = -np.inf
    if odd:
        neg = r.random((T, K)) < 0.2
        ids[neg] -= V
        ids[np.isneginf(a)] = 2 ** 31 - 1      # never looked at
        if K > 2:
            ids[:, 2] = ids[:, 0]              # named twice; outside [-V, V) where entry 0 is absent
        a[T // 2] = -np.inf                    # the teacher says nothing
    return ids, a


def same(p, q):
    """Equal, NaN where the other is NaN."""
    return torch.allclose(p, q, rtol=0, atol=0, equal_nan=True)


def padded(z, pad, shift, dtype):
    T, V = z.shape
    buf = torch.full((shift + T * (V + pad),), float("nan"), dtype=dtype, device="cuda")
    v = buf[shift:].view(T, V + pad)[:, :V]
    v.copy_(torch.from_numpy(z).to(dtype))
    return v


def check_logits(z_t, ids, a, tau, tau_t, tlse, mask, grad, loss, lse, d, name):
    z = ref.f64(z_t) / tau
    T, V = z.shape
    K = ids.shape[1]
    el, es, _ = ref.distill_fwd(z, ids, a, tau_t, tlse, mask)
    p, logp = ref.teacher(a, tau_t, tlse)
    P = p.sum(1)
    fin = np.where(np.isfinite(z), np.abs(z), 0)
    zmax = fin.max(1)
    af = np.where(np.isfinite(a), np.abs(a), 0) / tau_t
    L = np.where(np.isfinite(a).any(1), np.abs(af).max(1) + np.log(K + 1), 0)
    if tlse is not None:
        L = np.abs(tlse)
    ts = 2.0 ** -21 + (V / 256 + 32) * U + 8 * U * zmax
    got = ref.f64(lse)
    both = np.isfinite(es)
    assert np.array_equal(np.isnan(got), np.isnan(es)) and np.array_equal(got[~both & ~np.isnan(es)], es[~both & ~np.isnan(es)])
    assert (np.abs(got - es)[both] <= ts[both]).all()
    got = ref.f64(loss)
    both = np.isfinite(el)
    assert np.array_equal(np.isnan(got), np.isnan(el)) and np.array_equal(got[~both & ~np.isnan(el)], el[~both & ~np.isnan(el)])
    lp = np.where(p > 0, np.abs(np.where(np.isfinite(logp), logp, 0)), 0)
    tl = P * ts + 16 * U * (p * (af + L[:, None] + lp + 3 * zmax[:, None] + np.abs(np.where(np.isfinite(es), es, 0))[:, None])).sum(1)
    tl += (2 * K + 64 + 16 * (af.max(1) + L)) * U * (p * (lp + 2 * zmax[:, None] + 12)).sum(1)
    assert (np.abs(got - el)[both] <= tl[both]).all()
    if d is None:
        return
    ed = ref.distill_dz(z, ref.f64(lse), ids, a, grad / tau, tau_t, tlse, mask)
    got = ref.f64(d)
    assert np.array_equal(np.isnan(got), np.isnan(ed))
    both = np.isfinite(ed)
    with np.errstate(all="ignore"):
        q = np.exp(z - ref.f64(lse)[:, None])
        taken = np.zeros_like(z)
        at = ref.wrap(ids, V)
        for t in range(T):
            np.add.at(taken[t], at[t][at[t] >= 0], p[t][at[t] >= 0])
        pe = (K + 32 + 8 * (af.max(1) + L)) * U
        lsef = np.where(np.isfinite(es), np.abs(es), 0)
        dq = 2.0 ** -21 + 8 * U * (fin + lsef[:, None])
        td = np.abs(grad / tau)[:, None] * (P[:, None] * q * (dq + pe[:, None]) + taken * pe[:, None])
    td = td * (1 + ref.UNIT[name]) + ref.UNIT[name] * np.abs(ed) + ref.TINY[name]
    off = np.abs(got - ed)[both]
    assert ((off <= td[both]) | (off == 0)).all()   # zeros of NaN rows have no q to scale by


LOGIT_SHAPES = [(1, 1, 1), (1, 2, 3), (3, 50, 50), (40, 3001, 7), (25, 3000, 64), (6, 70001, 64),
                (5, 70000, 300), (2, 151936, 20), (3, 2000, 1024), (700, 260, 5)]


@pytest.mark.parametrize("T,V,K", LOGIT_SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("own_lse", [False, True])
def test_held_logits(T, V, K, dtype, own_lse):
    ensure_built()
    r = np.random.default_rng(T + V + K)
    ids, a = teacher(T, V, K, V + K)
    pad, shift = (0, 0) if V % 8 == 0 else (5, 1)
    z = padded((r.normal(size=(T, V)) * 2).astype(np.float32), pad, shift, DT[dtype])
    tau, tau_t = (0.7, 1.5) if T % 2 else (1.0, 1.0)
    tlse = None if not own_lse else (np.array([9.0]) / tau_t + r.random(T)).astype(np.float32)
    mask = None if T < 3 else (r.random(T) > 0.25).astype(np.uint8)
    grad = r.normal(size=T).astype(np.float32)
    cu = lambda v: None if v is None else torch.from_numpy(v).cuda()   # noqa: E731
    loss, lse = lm.distill_logits_forward(z, cu(ids), cu(a), cu(mask), tau, tau_t, cu(tlse))
    d = lm.distill_logits_backward(z, cu(ids), cu(a), cu(mask), tau, tau_t, cu(grad), lse, cu(tlse))
    tl64 = None if tlse is None else tlse.astype(np.float64)
    check_logits(z, ids, a.astype(np.float64), tau, tau_t, tl64, mask, grad.astype(np.float64),
                 loss, lse, d, dtype)
    if mask is not None:
        assert (d[cu(mask) == 0] == 0).all() and (loss[cu(mask) == 0] == 0).all()
    # over the logits themselves, and into rows of another stride: the same bits
    other = padded(np.zeros((T, V), np.float32), 3, 0, DT[dtype])
    lm.distill_logits_backward(z, cu(ids), cu(a), cu(mask), tau, tau_t, cu(grad), lse, cu(tlse), other)
    assert torch.equal(other, d)
    lm.distill_logits_backward(z, cu(ids), cu(a), cu(mask), tau, tau_t, cu(grad), lse, cu(tlse), z)
    assert torch.equal(z, d)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_held_logits_more_rows_than_the_grid(dtype):
    """CTAs that take a second row, with many entries: distinct, repeated, absent, and (rows whose
    own log-sum-exp is far above) present without any mass."""
    ensure_built()
    T, V, K = 33500, 100, 80
    r = np.random.default_rng(12)
    ids = np.argsort(r.random((T, V)), axis=1)[:, :K].astype(np.int32)
    a = (r.normal(size=(T, K)) * 2 + 5).astype(np.float32)
    tlse = (9.0 + r.random(T)).astype(np.float32)
    ids[::3, 5] = ids[::3, 9]
    a[1::5] = -np.inf
    tlse[2::5] = 3000.0
    z = padded((r.normal(size=(T, V)) * 2).astype(np.float32), 4, 0, DT[dtype])
    grad = r.normal(size=T).astype(np.float32)
    cu = lambda v: torch.from_numpy(v).cuda()   # noqa: E731
    loss, lse = lm.distill_logits_forward(z, cu(ids), cu(a), None, 0.7, 1.0, cu(tlse))
    d = lm.distill_logits_backward(z, cu(ids), cu(a), None, 0.7, 1.0, cu(grad), lse, cu(tlse))
    for rows in (slice(0, 150), slice(32700, 33500)):
        check_logits(z[rows], ids[rows], a[rows].astype(np.float64), 0.7, 1.0,
                     tlse[rows].astype(np.float64), None, grad[rows].astype(np.float64),
                     loss[rows], lse[rows], d[rows], dtype)


@pytest.mark.parametrize("V", [3001, 3000, 40000])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_held_logits_not_finite(V, dtype):
    ensure_built()
    T, K = 40, 6
    r = np.random.default_rng(V)
    ids, a = teacher(T, V, K, 5)
    z = (r.normal(size=(T, V)) * 2).astype(np.float32)
    z[r.random((T, V)) < 0.05] = -np.inf
    z[3] = -np.inf
    z[4] = torch.finfo(DT[dtype]).min          # a mask of the type's lowest value
    z[5, 7] = np.nan
    z[6, 11] = np.inf
    z[7, ids[7, 1] % V] = -np.inf              # a teacher's id with no probability
    a[7, 1] = 4.0
    ids[7, 1] %= V
    a[8, 1], ids[8, 1] = 3.0, V + 4            # an invalid id
    a[9, 1] = np.nan
    a[10] = -200.0                             # every entry far below
    a[11, 0], a[11, 1] = 90.0, -90.0           # p underflows to 0
    ids[12, 0], a[12, 0] = -V, 2.0
    a[3, 0] = a[5, 0] = a[6, 0] = 1.0
    for t in (3, 5, 6):
        ids[t, 0] %= V
    zt = padded(z, 0, 0, DT[dtype])
    grad = r.normal(size=T).astype(np.float32)
    cu = lambda v: torch.from_numpy(v).cuda()   # noqa: E731
    loss, lse = lm.distill_logits_forward(zt, cu(ids), cu(a))
    d = lm.distill_logits_backward(zt, cu(ids), cu(a), None, 1.0, 1.0, cu(grad), lse)
    check_logits(zt, ids, a.astype(np.float64), 1.0, 1.0, None, None, grad.astype(np.float64), loss,
                 lse, d, dtype)
    assert torch.isinf(loss[7]) and torch.isnan(loss[8]) and torch.isnan(loss[9])
    assert (d[~torch.isfinite(zt)] == 0).all()
    assert loss[T // 2] == 0 and (d[T // 2] == 0).all()


def test_held_logits_no_tokens_and_autograd():
    ensure_built()
    e = torch.empty(0, 30, device="cuda")
    loss, lse = lm.distill_logits_forward(e, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                                          torch.empty(0, 2, device="cuda"))
    assert loss.numel() == lse.numel() == 0
    T, V, K = 20, 700, 8
    ids, a = teacher(T, V, K, 3)
    z = (torch.randn(T, V, device="cuda") * 2).to(torch.bfloat16).requires_grad_(True)
    ids, a = torch.from_numpy(ids).cuda(), torch.from_numpy(a).cuda()
    out = autograd.distill_logits(z, ids, a, None, 0.7, 1.3)
    loss, lse = lm.distill_logits_forward(z.detach(), ids, a, None, 0.7, 1.3)
    assert same(out, loss)
    g = torch.randn(T, device="cuda")
    dz, = torch.autograd.grad(out, z, g)
    assert torch.equal(dz, lm.distill_logits_backward(z.detach(), ids, a, None, 0.7, 1.3, g, lse))


def test_held_logits_gradient_against_differences():
    """Along random directions, against central differences of the 64-bit loss (step 1e-4)."""
    ensure_built()
    T, V, K = 8, 300, 5
    r = np.random.default_rng(4)
    ids, a = teacher(T, V, K, 9)
    z = (r.normal(size=(T, V)) * 2).astype(np.float32)
    g = r.normal(size=T).astype(np.float32)
    cu = lambda v: torch.from_numpy(v).cuda()   # noqa: E731
    _, lse = lm.distill_logits_forward(cu(z), cu(ids), cu(a), None, 0.8)
    d = ref.f64(lm.distill_logits_backward(cu(z), cu(ids), cu(a), None, 0.8, 1.0, cu(g), lse))
    for _ in range(3):
        way = r.normal(size=z.shape)

        def f(s):
            return (ref.distill_fwd((z + s * way) / 0.8, ids, a.astype(np.float64))[0] * g).sum()
        want = (f(1e-4) - f(-1e-4)) / 2e-4
        assert abs((d * way).sum() - want) <= 2e-5 * np.abs(d * way).sum()


# ------------------------------------------------------------------ through the head
def head_inputs(T, H, V, K, seed, mask=False):
    g = torch.Generator().manual_seed(seed)
    weight = (torch.randn(V, H, generator=g) * (2 / H ** 0.5)).to(torch.bfloat16)
    ids, a = teacher(T, V, K, seed + 1)
    hidden = torch.randn(T, H, generator=g) + 2 * weight[torch.from_numpy(ids[:, 0]).long() % V].float()
    m = (torch.rand(T, generator=g) > 0.3).to(torch.uint8) if mask else None
    grad = torch.randn(T, generator=g)
    return [t if t is None else t.cuda() for t in (hidden.to(torch.bfloat16), weight,
                                                   torch.from_numpy(ids), torch.from_numpy(a), m, grad)]


HEADS = [(1, 64, 1, 1, 1), (1, 64, 100, 3, 1), (130, 128, 2048, 16, 64), (333, 192, 3001, 7, 64),
         (700, 320, 5003, 64, 512), (257, 64, 1025, 1024, 7), (1030, 256, 9000, 33, 100)]


@pytest.mark.parametrize("T,H,V,K,chunk", HEADS)
@pytest.mark.parametrize("mask,own_lse,tau", [(False, False, 1.0), (True, True, 0.7)])
def test_through_the_head(T, H, V, K, chunk, mask, own_lse, tau):
    ensure_built()
    hidden, weight, ids, a, m, grad = head_inputs(T, H, V, K, T + V, mask)
    tlse = torch.full((T,), 8.0, device="cuda") if own_lse else None
    ws = torch.empty(max(lm.lmhead_distill_workspace_size(o, T, H, V, K, chunk) for o in (0, 1)),
                     dtype=torch.uint8, device="cuda")
    loss, lse, zt = lm.distill_forward(hidden, weight, ids, a, m, tau, 1.2, chunk, tlse, ws)
    z = ref.f64(hidden) @ ref.f64(weight).T / tau
    A, I, M, tl = ref.f64(a), ids.cpu().numpy(), None if m is None else m.cpu().numpy(), ref.f64(tlse)
    # some tokens name an id outside the vocabulary (see teacher): NaN, and a status of 6
    bad = ~np.isneginf(A) & (ref.wrap(I, V) < 0)
    status = 6 if (bad if M is None else bad[M != 0]).any() else 0
    assert lm.lmhead_read_device_status(ws) == status
    el, es, ez = ref.distill_fwd(z, I, A, 1.2, tl, M)
    P = ref.teacher(A, 1.2, tl)[0].sum(1)
    assert np.abs(ref.f64(lse) - es).max() <= LIMITS["lse"]
    assert np.array_equal(np.isnan(ref.f64(loss)), np.isnan(el))
    assert np.array_equal(np.isnan(ref.f64(zt)), np.isnan(ez))
    off = np.nan_to_num(np.abs(ref.f64(loss) - el))
    assert (off <= LIMITS["logp"] * np.maximum(P, 1e-3)).all()
    assert np.nan_to_num(np.abs(ref.f64(zt) - ez)).max() <= LIMITS["lse"]
    start = torch.ones(V, H, device="cuda")
    dh, dw = lm.distill_backward(hidden, weight, ids, a, m, tau, 1.2, chunk, grad, lse, zt, tlse,
                                 workspace=ws)
    assert lm.lmhead_read_device_status(ws) == status
    dz = ref.distill_dz(z, es, I, A, ref.f64(grad), 1.2, tl, M) / tau
    eh, ew = dz @ ref.f64(weight), dz.T @ ref.f64(hidden)
    for got, want in ((dh, eh), (dw, ew)):
        if np.abs(want).max() < 1e-6:          # one id: softmax is 1, the cotangent cancels
            assert np.abs(ref.f64(got)).max() < 1e-3
        else:
            assert rel_fro(ref.f64(got), want) <= LIMITS["d_hidden"]
    if M is not None:
        assert (dh[m == 0] == 0).all()
    # bf16 d_weight: the fp32 tiles, rounded once
    if lm.lmhead_distill_narrow_dweight(T, H, V, chunk):
        narrow = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(lm.distill_backward(hidden, weight, ids, a, m, tau, 1.2, chunk, grad, lse,
                                               zt, tlse, d_weight=narrow, workspace=ws)[0], dh)
        assert torch.equal(narrow, dw.to(torch.bfloat16))
    again = lm.distill_backward(hidden, weight, ids, a, m, tau, 1.2, chunk, grad, lse, zt, tlse,
                                d_weight=start, accumulate_dweight=True, workspace=ws)
    assert torch.equal(again[0], dh)
    assert torch.allclose(start, dw + 1.0, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("form", ["0", "2"])
def test_head_backward_forms_agree(form):
    """Two launches per block, and windows, against the persistent launch: the same bits."""
    ensure_built()
    T, H, V, K, chunk = 333, 192, 3001, 40, 64
    hidden, weight, ids, a, m, grad = head_inputs(T, H, V, K, 3, True)
    _, lse, zt = lm.distill_forward(hidden, weight, ids, a, m, 1.0, 1.0, chunk)
    want = lm.distill_backward(hidden, weight, ids, a, m, 1.0, 1.0, chunk, grad, lse, zt)
    old = os.environ.get("LMHEAD_BWD_PERSISTENT")
    try:
        os.environ["LMHEAD_BWD_PERSISTENT"] = form
        assert not lm.lmhead_distill_narrow_dweight(T, H, V, chunk)
        got = lm.distill_backward(hidden, weight, ids, a, m, 1.0, 1.0, chunk, grad, lse, zt)
    finally:
        if old is None:
            del os.environ["LMHEAD_BWD_PERSISTENT"]
        else:
            os.environ["LMHEAD_BWD_PERSISTENT"] = old
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_head_every_token_unscored_or_without_a_teacher():
    ensure_built()
    T, H, V, K = 150, 64, 500, 4
    hidden, weight, ids, a, _, grad = head_inputs(T, H, V, K, 1)
    nothing = torch.full_like(a, float("-inf"))
    for m, top in ((torch.zeros(T, dtype=torch.uint8, device="cuda"), a), (None, nothing)):
        loss, lse, zt = lm.distill_forward(hidden, weight, ids, top, m)
        assert (loss == 0).all() and (zt == 0).all()
        dh, dw = lm.distill_backward(hidden, weight, ids, top, m, 1.0, 1.0, 512, grad, lse, zt)
        assert (dh == 0).all() and (dw == 0).all()


def test_head_invalid_id_sets_the_status():
    ensure_built()
    T, H, V, K = 60, 64, 500, 4
    hidden, weight, ids, a, _, grad = head_inputs(T, H, V, K, 2)
    ids[7, 1], a[7, 1] = V, 1.0
    ws = torch.empty(max(lm.lmhead_distill_workspace_size(o, T, H, V, K, 64) for o in (0, 1)),
                     dtype=torch.uint8, device="cuda")
    loss, lse, zt = lm.distill_forward(hidden, weight, ids, a, None, 1.0, 1.0, 64, workspace=ws)
    assert lm.lmhead_read_device_status(ws) == 6
    assert torch.isnan(loss[7]) and torch.isnan(zt[7, 1])
    other = ~torch.isneginf(a) & (ids.long() >= V)           # those of teacher()
    assert torch.equal(torch.isnan(loss), other.any(1))
    dh, dw = lm.distill_backward(hidden, weight, ids, a, None, 1.0, 1.0, 64, grad, lse, zt, workspace=ws)
    assert lm.lmhead_read_device_status(ws) == 6
    A, I = ref.f64(a), ids.cpu().numpy()
    z = ref.f64(hidden) @ ref.f64(weight).T
    dz = ref.distill_dz(z, ref.log_sum_exp(z), I, A, ref.f64(grad))
    assert rel_fro(ref.f64(dh), dz @ ref.f64(weight)) <= LIMITS["d_hidden"]
    assert rel_fro(ref.f64(dw), dz.T @ ref.f64(hidden)) <= LIMITS["d_weight"]


def test_head_no_tokens():
    ensure_built()
    w = torch.ones(40, 64, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ids, a = torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, 3, device="cuda")
    loss, lse, zt = lm.distill_forward(h, w, ids, a)
    dh, dw = lm.distill_backward(h, w, ids, a, None, 1.0, 1.0, 512, loss, lse, zt)
    assert dh.shape == (0, 64) and (dw == 0).all()


def test_head_autograd_and_main_grad():
    ensure_built()
    T, H, V, K = 200, 128, 3000, 16
    hidden, weight, ids, a, m, grad = head_inputs(T, H, V, K, 6, True)
    hidden.requires_grad_(True)
    weight.requires_grad_(True)
    out = autograd.lmhead_distill(hidden, weight, ids, a, m, 0.9, 1.0, 64)
    dh, dw = torch.autograd.grad(out, (hidden, weight), grad)
    loss, lse, zt = lm.distill_forward(hidden.detach(), weight.detach(), ids, a, m, 0.9, 1.0, 64)
    eh, ew = lm.distill_backward(hidden.detach(), weight.detach(), ids, a, m, 0.9, 1.0, 64, grad, lse, zt)
    assert same(out, loss) and dh.dtype == torch.bfloat16
    assert torch.equal(dh, eh.to(torch.bfloat16)) and torch.equal(dw, ew.to(torch.bfloat16))
    main = torch.zeros(V, H, device="cuda")
    for _ in range(2):
        out = autograd.lmhead_distill(hidden, weight, ids, a, m, 0.9, 1.0, 64, main_grad=main)
        out.backward(grad)
    assert weight.grad is None and torch.allclose(main, 2 * ew, rtol=1e-5, atol=1e-7)


def test_on_another_stream_and_in_a_graph():
    ensure_built()
    T, H, V, K = 140, 64, 2000, 8
    hidden, weight, ids, a, m, grad = head_inputs(T, H, V, K, 7, True)
    z = torch.randn(T, V, device="cuda")
    want = lm.distill_forward(hidden, weight, ids, a, m) + lm.distill_logits_forward(z, ids, a, m)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = lm.distill_forward(hidden, weight, ids, a, m) + lm.distill_logits_forward(z, ids, a, m)
    side.synchronize()
    assert all(same(p, q) for p, q in zip(got, want))
    ws = torch.empty(lm.lmhead_distill_workspace_size(0, T, H, V, K, 512), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lm.distill_forward(hidden, weight, ids, a, m, workspace=ws)
        held = lm.distill_logits_forward(z, ids, a, m)
        d = lm.distill_logits_backward(z, ids, a, m, 1.0, 1.0, grad, held[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(p, q) for p, q in zip(got + held, want))
    assert torch.equal(d, lm.distill_logits_backward(z, ids, a, m, 1.0, 1.0, grad, held[1]))
