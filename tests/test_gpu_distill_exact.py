"""Distillation through the head where each logit and each cotangent can be read off: with rows or a
table of unit vectors every product has one term, so the head's sums add nothing, and what is left
is the operator's own arithmetic.

Then z is a bf16 number / temperature, z_top is that quotient rounded once, loss and lse are held
to the tolerances of held logits (the sums have chains of 16 pairs, 8 chunks and 5 shuffles at one
256-column tile per split), and each entry of the gradient is the fp32 cotangent rounded once
to bf16, the type in which both gradient products read it.  A teacher's entry that were left out
of the loss, or kept the dense cotangent, is off by its probability."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm

import operators_reference as ref
from gpu_helpers import ensure_built
from test_gpu_distill import check_logits, teacher

pytestmark = pytest.mark.gpu

TAU, TAU_T = 0.7, 1.3


def run(hidden, weight, z, K, seed, monkeypatch, form, masked, own_lse):
    """z [T, V] bf16: the logits before the temperature.  Returns (dh, dw, check of dz [T, V])."""
    ensure_built()
    monkeypatch.setenv("LMHEAD_BWD_PERSISTENT", form)
    T, V = z.shape
    r = np.random.default_rng(seed)
    ids, a = teacher(T, V, K, seed)
    mask = (r.random(T) > 0.3).astype(np.uint8) if masked else None
    tlse = (9.0 + r.random(T)).astype(np.float32) if own_lse else None
    grad = r.normal(size=T).astype(np.float32)
    cu = lambda v: None if v is None else torch.from_numpy(v).cuda()   # noqa: E731
    loss, lse, z_top = lm.distill_forward(hidden, weight, cu(ids), cu(a), cu(mask), TAU, TAU_T, 64,
                                          cu(tlse))
    at = ref.wrap(ids, V)
    want = z.float().cpu().numpy()[np.arange(T)[:, None], np.maximum(at, 0)] / np.float32(TAU)
    want = np.where(np.isneginf(a), 0, np.where(at < 0, np.nan, want))
    if masked:
        want[mask == 0] = 0
    assert np.array_equal(z_top.cpu().numpy(), want.astype(np.float32), equal_nan=True)
    dh, dw = lm.distill_backward(hidden, weight, cu(ids), cu(a), cu(mask), TAU, TAU_T, 64, cu(grad),
                                 lse, z_top, cu(tlse))

    def check(dz):
        check_logits(z, ids, a.astype(np.float64), TAU, TAU_T,
                     None if tlse is None else tlse.astype(np.float64), mask,
                     grad.astype(np.float64), loss, lse, dz, "bfloat16")
    return dh, dw, check


@pytest.mark.parametrize("form", ["", "0", "2"])
@pytest.mark.parametrize("masked,own_lse", [(False, False), (True, True)])
@pytest.mark.parametrize("T,V,K", [(300, 1025, 7), (130, 600, 64)])
def test_hidden_gradient_by_entry(T, V, K, masked, own_lse, form, monkeypatch):
    """A table of unit vectors: d_hidden is the cotangent."""
    H = (V + 63) // 64 * 64
    g = torch.Generator().manual_seed(T)
    hidden = (torch.randn(T, H, generator=g) * 2).to(torch.bfloat16).cuda()
    weight = torch.eye(V, H, dtype=torch.bfloat16, device="cuda")
    dh, _, check = run(hidden, weight, hidden[:, :V], K, V + K, monkeypatch, form, masked, own_lse)
    check(dh[:, :V])
    assert (dh[:, V:] == 0).all()


@pytest.mark.parametrize("form", ["", "0", "2"])
@pytest.mark.parametrize("masked,own_lse", [(False, False), (True, True)])
@pytest.mark.parametrize("T,V,K", [(300, 3001, 7), (257, 1300, 200)])
def test_weight_gradient_by_entry(T, V, K, masked, own_lse, form, monkeypatch):
    """Rows of unit vectors: d_weight is the cotangent."""
    H = (T + 63) // 64 * 64
    g = torch.Generator().manual_seed(V)
    hidden = torch.eye(T, H, dtype=torch.bfloat16, device="cuda")
    weight = (torch.randn(V, H, generator=g) * 2).to(torch.bfloat16).cuda()
    _, dw, check = run(hidden, weight, weight.t()[:T], K, V + K, monkeypatch, form, masked, own_lse)
    check(dw.t()[:T])
    assert (dw[:, T:] == 0).all()
