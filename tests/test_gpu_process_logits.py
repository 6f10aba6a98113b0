"""Penalties, biases and grammar masks on logits, and their gradient, against
the 64-bit definition.

Tolerance (u = 2^-24): a division or product, a fused f c + p, a subtraction and
an addition, so 4 u of the largest operand, then one rounding to the type.
Untouched logits and infinities are exact."""
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


def padded(z, pad, shift, dtype):
    R, V = z.shape
    buf = torch.full((shift + R * (V + pad),), 5.0, dtype=dtype, device="cuda")
    v = buf[shift:].view(R, V + pad)[:, :V]
    v.copy_(torch.from_numpy(z).to(dtype))
    return v


def rules(R, V, n, seed, shared=False, bias=True, grammar=True):
    r = np.random.default_rng(seed)
    tokens = (V * r.random(max(n, 1)) ** 3).astype(np.int32)
    tokens[r.random(len(tokens)) < 0.05] = -1
    tokens[r.random(len(tokens)) < 0.02] = V
    if shared:
        spans = np.stack([np.zeros(R), np.full(R, n // 2), n // 2 + np.arange(R)], 1)
    else:
        spans = np.sort(r.integers(0, n + 1, size=(R, 3)), axis=1)
        spans[0] = 0                                        # no history
        if R > 3:
            spans[1] = [-5, 1, n + 100]                     # cut to what exists
            spans[2] = [n // 2, n // 4, n // 3]             # out of order: empty
    k = dict(tokens=tokens, spans=spans.astype(np.int64),
             repetition=(1 + r.random(R)).astype(np.float32),
             frequency=r.normal(size=R).astype(np.float32),
             presence=r.normal(size=R).astype(np.float32))
    if bias:
        per = r.integers(0, 40, size=R)
        off = np.concatenate([[0], np.cumsum(per)]).astype(np.int64)
        ids = r.integers(-2, V + 2, size=off[-1]).astype(np.int32)
        if off[1] - off[0] > 1:
            ids[1] = ids[0] % V
            ids[0] = ids[1]                                 # the last entry counts
        k.update(bias_offsets=off, bias_ids=ids, bias_values=r.normal(size=off[-1]).astype(np.float32))
    if grammar:
        m = max(1, R // 2)
        words = r.integers(-2 ** 31, 2 ** 31, size=(m, (V + 31) // 32)).astype(np.int32)
        words[0] = 0                                        # allows nothing
        rows = r.integers(-1, m + 1, size=R).astype(np.int32)   # -1 and m: no mask
        rows[-1] = 0
        k.update(allowed=words, allowed_rows=rows)
    return k


def cu(k):
    return {n: torch.from_numpy(np.ascontiguousarray(v)).cuda() for n, v in k.items()}


def wide(k):
    return {n: v.astype(np.float64) if v.dtype == np.float32 else v for n, v in k.items()}


def check(got, want, size, name):
    got = ref.f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    big = np.isinf(got) & ~inf     # fp16 overflow of a finite result is an infinity of its sign
    assert np.array_equal(got[inf], want[inf])
    if name == "float16":
        assert (np.abs(want[big]) > 65000).all()
    ok = np.isfinite(want) & ~big
    tol = 4 * U * size * (1 + ref.UNIT[name]) + ref.UNIT[name] * np.abs(want) + ref.TINY[name]
    assert (np.abs(got - want)[ok] <= tol[ok]).all()


def sizes(x, k):
    """Sum of the operands' magnitudes of the forward."""
    R, V = x.shape
    _, count = ref.history(k["tokens"], k["spans"], R, V)
    s = np.where(np.isfinite(x), np.abs(x), 0) * 2.5
    s += np.abs(k["frequency"])[:, None] * count + np.abs(k["presence"])[:, None]
    b = np.abs(k["bias_values"]).max() if k.get("bias_values") is not None and len(k["bias_values"]) else 0
    return s + b


SHAPES = [(1, 1, 0), (1, 31, 5), (2, 32, 40), (5, 33, 100), (9, 3001, 500), (4, 20000, 3000),
          (3, 70000, 9000), (1, 151936, 900), (130, 1000, 700)]


@pytest.mark.parametrize("R,V,n", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_both_directions(R, V, n, dtype):
    ensure_built()
    r = np.random.default_rng(R + V)
    x = (r.normal(size=(R, V)) * 3).astype(np.float32)
    x[r.random((R, V)) < 0.02] = -np.inf
    x[0, 0] = np.nan
    if V > 5:
        x[R - 1, 4] = np.inf
        x[0, 3] = torch.finfo(DT[dtype]).min
    pad, shift = [(0, 0), (8, 0), (3, 1)][(R + V) % 3]
    z = padded(x, pad, shift, DT[dtype])
    k = rules(R, V, n, 3 * V + R)
    c, w = cu(k), wide(k)
    X = ref.f64(z)
    with np.errstate(all="ignore"):
        want = ref.process_fwd(X, **w)
    out = lm.process_logits(z, **c)
    check(out, want, sizes(X, w), dtype)
    other = padded(np.zeros((R, V), np.float32), 1, 0, DT[dtype])
    lm.process_logits(z, **c, out=other)
    assert torch.equal(out.nan_to_num(1e3), other.nan_to_num(1e3))
    g = padded(r.normal(size=(R, V)).astype(np.float32), 0, 0, DT[dtype])
    few = {n_: c[n_] for n_ in ("tokens", "spans", "repetition", "allowed", "allowed_rows")}
    d = lm.process_logits_backward(g, z, **few)
    with np.errstate(all="ignore"):
        check(d, ref.process_bwd(ref.f64(g), X, **{n_: w[n_] for n_ in few}), np.abs(ref.f64(g)) * 2, dtype)
    lm.process_logits_backward(g, z, **few, d_logits=g)            # over the cotangent
    assert torch.equal(g, d)
    lm.process_logits(z, **c, out=z)                               # over the logits
    assert torch.equal(out.nan_to_num(1e3), z.nan_to_num(1e3))


@pytest.mark.parametrize("drop", ["tokens", "bias", "allowed", "allowed_rows", "repetition",
                                  "frequency", "presence", "all"])
def test_each_rule_is_optional(drop):
    ensure_built()
    R, V, n = 6, 5000, 300
    x = (np.random.default_rng(1).normal(size=(R, V)) * 3).astype(np.float32)
    k = rules(R, V, n, 11)
    gone = {"tokens": ["tokens", "spans", "repetition", "frequency", "presence"],
            "bias": ["bias_offsets", "bias_ids", "bias_values"],
            "allowed": ["allowed", "allowed_rows"], "all": list(k)}.get(drop, [drop])
    if drop == "allowed_rows":
        k["allowed"] = np.concatenate([k["allowed"]] * 2)
    w = wide(k)
    size = sizes(x.astype(np.float64), w)
    for name in gone:
        del k[name], w[name]
    z = padded(x, 0, 0, torch.float32)
    check(lm.process_logits(z, **cu(k)), ref.process_fwd(x.astype(np.float64), **w), size, "float32")


def test_positions_of_one_sequence_share_their_tokens():
    ensure_built()
    R, V, n = 60, 9001, 400
    x = (np.random.default_rng(2).normal(size=(R, V)) * 3).astype(np.float32)
    k = rules(R, V, n, 5, shared=True, bias=False)
    z = padded(x, 0, 0, torch.float32)
    w = wide(k)
    check(lm.process_logits(z, **cu(k)), ref.process_fwd(x.astype(np.float64), **w),
          sizes(x.astype(np.float64), w), "float32")


def test_long_history():
    """One row with more outputs of one id than 16 bits count."""
    ensure_built()
    V, n = 40000, 200000
    tokens = np.random.default_rng(3).integers(0, V, size=n).astype(np.int32)
    tokens[1000:90000] = 17
    k = dict(tokens=tokens, spans=np.array([[0, 500, n]], np.int64),
             frequency=np.array([0.001], np.float32), presence=np.array([0.5], np.float32))
    x = np.random.default_rng(4).normal(size=(1, V)).astype(np.float32)
    w = wide(k)
    got = lm.process_logits(torch.from_numpy(x).cuda(), **cu(k))
    check(got, ref.process_fwd(x.astype(np.float64), **w), sizes(x.astype(np.float64), w), "float32")


def test_no_rows_and_autograd_and_side_stream():
    ensure_built()
    e = torch.empty(0, 30, device="cuda")
    assert lm.process_logits(e).shape == (0, 30)
    R, V, n = 7, 3000, 200
    k = cu(rules(R, V, n, 8))
    z = torch.randn(R, V, device="cuda", requires_grad=True)
    out = autograd.process_logits(z, **k)
    assert torch.equal(out, lm.process_logits(z.detach(), **k))
    g = torch.randn(R, V, device="cuda")
    few = {n_: k[n_] for n_ in ("tokens", "spans", "repetition", "allowed", "allowed_rows")}
    d, = torch.autograd.grad(out, z, g)
    assert torch.equal(d, lm.process_logits_backward(g, z.detach(), **few))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = lm.process_logits(z.detach(), **k)
    side.synchronize()
    assert torch.equal(again, out)


def test_processed_logits_are_scored():
    """The rows a grammar leaves nothing of, and the rest, through the scoring call: the
    log-prob of an id under the processed distribution."""
    ensure_built()
    R, V, n = 12, 4000, 300
    k = cu(rules(R, V, n, 21))
    z = torch.randn(R, V, device="cuda") * 3
    out = lm.process_logits(z, **k)
    y = torch.randint(0, V, (R,), dtype=torch.int32, device="cuda")
    logp, ent, lse = (torch.empty(R, device="cuda") for _ in range(3))
    assert lm.lmhead_score_logits_fwd(out, y, None, 1.0, logp, ent, lse) == 0
    want = torch.log_softmax(out.double(), 1).gather(1, y.long()[:, None])[:, 0]
    none = torch.isneginf(out).all(1)
    assert none.any() and torch.isnan(logp[none]).all()
    ok = ~none & torch.isfinite(want)
    assert (logp[ok].double() - want[ok]).abs().max() < 1e-4
    assert torch.isneginf(logp[~none & torch.isneginf(want)]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_empty_lists(dtype):
    """Lists without an entry (torch gives them no address) are lists all the same."""
    ensure_built()
    R, V = 3, 1000
    x = torch.randn(R, V, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(dtype)
    none = dict(dtype=torch.int32, device="cuda")
    two = torch.full((R,), 2.0, device="cuda")
    history = dict(tokens=torch.empty(0, **none),
                   spans=torch.zeros(R, 3, dtype=torch.int64, device="cuda"), repetition=two)
    grammar = dict(allowed=torch.empty(0, (V + 31) // 32, **none),
                   allowed_rows=torch.full((R,), -1, **none))
    bias = dict(bias_offsets=torch.zeros(R + 1, dtype=torch.int64, device="cuda"),
                bias_ids=torch.empty(0, **none), bias_values=torch.empty(0, device="cuda"))
    penalties = dict(frequency=two, presence=two)
    for k in (history, grammar, bias, dict(history, **grammar, **bias, **penalties)):
        assert torch.equal(lm.process_logits(x, **k), x)
    for k in (history, grammar, dict(history, **grammar)):
        assert torch.equal(lm.process_logits_backward(x, x, **k), x)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_many_rows(dtype):
    """More rows than several rounds of CTAs take at once, with histories that overlap."""
    ensure_built()
    R, V, n = 1500, 517, 120
    x = (np.random.default_rng(8).normal(size=(R, V)) * 3).astype(np.float32)
    z = padded(x, 3, 1, DT[dtype])
    k = rules(R, V, n, 6)
    w = wide(k)
    xz = ref.f64(z)
    check(lm.process_logits(z, **cu(k)), ref.process_fwd(xz, **w), sizes(xz, w), dtype)
    g = padded(np.random.default_rng(9).normal(size=(R, V)).astype(np.float32), 0, 0, DT[dtype])
    kb = {n: v for n, v in k.items() if n in ("tokens", "spans", "repetition", "allowed", "allowed_rows")}
    want = ref.process_bwd(ref.f64(g), xz, **wide(kb))
    check(lm.process_logits_backward(g, z, **cu(kb)), want, 2 * np.abs(ref.f64(g)), dtype)
