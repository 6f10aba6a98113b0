"""Rows whose element offsets pass 32 bits: the last rows of a tensor of more than
2^31 elements give the bits that the same rows give on their own."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

V = 151936
ROWS = 2 ** 31 // V + 9


def tail(t, n=7):
    return None if t is None else t[-n:].clone()


@pytest.fixture(scope="module")
def logits():
    ensure_built()
    t = torch.empty(ROWS, V, dtype=torch.bfloat16, device="cuda")
    t.normal_(0, 2, generator=torch.Generator("cuda").manual_seed(3))
    assert t.numel() > 2 ** 31
    return t


def test_distill_logits(logits):
    g = torch.Generator("cuda").manual_seed(4)
    K = 8
    ids = torch.randint(0, V, (ROWS, K), generator=g, device="cuda", dtype=torch.int32)
    top = torch.randn(ROWS, K, generator=g, device="cuda")
    grad = torch.randn(ROWS, generator=g, device="cuda")
    loss, lse = lm.distill_logits_forward(logits, ids, top)
    want = lm.distill_logits_forward(tail(logits), tail(ids), tail(top))
    # few rows are split over CTAs, so their sums may differ in the last bits
    assert torch.allclose(tail(loss), want[0], rtol=1e-5, atol=1e-5)
    assert torch.allclose(tail(lse), want[1], rtol=1e-6, atol=1e-6)
    d = lm.distill_logits_backward(logits, ids, top, None, 1.0, 1.0, grad, lse)
    w = lm.distill_logits_backward(tail(logits), tail(ids), tail(top), None, 1.0, 1.0, tail(grad),
                                   tail(lse))
    assert torch.equal(tail(d), w)


def test_process_logits(logits):
    g = torch.Generator("cuda").manual_seed(5)
    n = 40
    tokens = torch.randint(0, V, (ROWS * n,), generator=g, device="cuda", dtype=torch.int32)
    begin = torch.arange(ROWS, device="cuda") * n
    spans = torch.stack([begin, begin + n // 2, begin + n], 1)
    rep = 1 + torch.rand(ROWS, generator=g, device="cuda")
    fr = torch.rand(ROWS, generator=g, device="cuda")
    allowed = torch.randint(-2 ** 31, 2 ** 31, (ROWS, (V + 31) // 32), generator=g,
                            device="cuda").to(torch.int32)
    out = lm.process_logits(logits, tokens, spans, rep, fr, allowed=allowed)
    last = lm.process_logits(tail(logits), tokens, tail(spans), tail(rep), tail(fr),
                             allowed=tail(allowed))
    assert torch.equal(tail(out), last)


def test_layernorm():
    ensure_built()
    H = 2560
    N = 2 ** 31 // H + 11
    x = torch.empty(N, H, dtype=torch.bfloat16, device="cuda")
    x.normal_(0.5, 2, generator=torch.Generator("cuda").manual_seed(6))
    w, b = torch.rand(H, device="cuda"), torch.rand(H, device="cuda")
    y, mean, rstd = lm.layernorm_forward(x, w, b)
    few = lm.layernorm_forward(tail(x, 2000), w, b)
    assert torch.equal(y[-2000:], few[0]) and torch.equal(mean[-2000:], few[1])
    dy = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda")
    dy[-2000:].normal_(generator=torch.Generator("cuda").manual_seed(7))
    dx, dw, db = lm.layernorm_backward(dy, x, w, mean, rstd)
    want = lm.layernorm_backward(tail(dy, 2000), tail(x, 2000), w, tail(mean, 2000), tail(rstd, 2000))
    assert torch.equal(dx[-2000:], want[0])
    assert torch.allclose(dw, want[1], rtol=1e-4, atol=1e-2) and (dx[:1000] == 0).all()
