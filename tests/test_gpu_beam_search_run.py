"""The operators together: beam search of requests with adapters, step by step against plain
64-bit and indexing forms on each step's own inputs; and a training step through a tied table."""
import os
import sys

import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd
from gpu_helpers import ensure_built
from operators_reference import U32, f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_search_adapters as example  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("beams,requests,vocab", [(4, 6, 4096), (1, 3, 1001), (7, 2, 5003)])
def test_beam_search(beams, requests, vocab):
    trace = []
    model, adapter_of, history, scores = example.main(steps=10, vocab=vocab, width=128, beams=beams,
                                                      requests=requests, trace=trace)
    adapters = adapter_of.repeat_interleave(beams).cpu().numpy()
    table, down, up = f64(model["table"]), f64(model["down"]), f64(model["up"])
    for step, s in enumerate(trace):
        # the logits, head and adapter in 64 bits from the step's own rows: sums of 128 (and 8)
        # products in fp32, each off by a unit at most (a library's product in bf16 would not do:
        # it may join its partial sums in 16 bits)
        y, z = f64(s["y"]), f64(s["logits"])
        want = y @ table.T
        tol = (128 + 70) * 2 * U32 * (np.abs(y) @ np.abs(table).T)
        for r in range(len(y)):
            if adapters[r] >= 0:
                u = 0.5 * y[r] @ down[adapters[r]].T
                want[r] += u @ up[adapters[r]]
                tol[r] += (128 + 70) * 2 * U32 * (np.abs(y[r]) @ np.abs(down[adapters[r]]).T) @ np.abs(
                    up[adapters[r]])
        met = np.zeros(z.shape, bool)
        np.put_along_axis(met, s["before"].cpu().numpy()[:, :step + 1].astype(np.int64), True, 1)
        factor = np.where(met, np.where(want > 0, 1 / 1.1, 1.1), 1.0)
        assert (np.abs(z - want * factor) <= tol * 1.1 + 4 * U32 * np.abs(z) + 0.2 * met * tol).all()
        # the selection, from the logits as they were
        flat = s["old"].view(-1).double().cpu().numpy()
        ended = s["finished"].view(-1).cpu().numpy() != 0
        m = z.max(1, keepdims=True)
        total = flat[:, None] + (z - m) - np.log(np.exp(z - m).sum(1, keepdims=True))
        total[ended] = -np.inf
        total[ended, example.EOS] = flat[ended]
        total = total.reshape(requests, -1)
        for g in range(requests):
            order = np.argsort(-total[g], kind="stable")[:beams]
            best = total[g][order]
            at = (s["parents"][g].cpu().numpy() - g * beams) * vocab + s["tokens"][g].cpu().numpy()
            assert (np.abs(total[g][at] - best) <= 1e-5).all() and len(set(at.tolist())) == beams
            assert (np.abs(f64(s["scores"][g]) - best) <= 1e-5 + 4 * U32 * np.abs(best)).all()
        # the states
        parents = s["parents"].view(-1).long()
        assert torch.equal(s["history"][:, :step + 1], s["before"][parents][:, :step + 1])
        assert torch.equal(s["history"][:, step + 1], s["tokens"].view(-1))
        own = lm.embedding_forward(s["history"][:, :step + 1].reshape(-1).contiguous(), model["table"], 128 ** 0.5)
        assert torch.equal(s["cache"].reshape(-1, 128), own)
        stop = (s["finished"].view(-1)[parents] != 0) | (s["tokens"].view(-1) == example.EOS)
        assert torch.equal(s["after"].view(-1) != 0, stop)
    assert (scores[:, :-1] >= scores[:, 1:]).all() and torch.isfinite(scores).all()


def test_training_step_of_a_tied_table_with_adapters():
    """Embedding, layer norm, the head's logits with adapters, distillation on them: every gradient
    against torch's own in 64 bits from the same bf16 inputs."""
    g = torch.Generator("cuda").manual_seed(3)
    T, H, V, n, rank, K = 96, 64, 500, 3, 4, 8
    table = (torch.randn(V, H, generator=g, device="cuda") / 8).to(torch.bfloat16)
    down = (torch.randn(n, rank, H, generator=g, device="cuda") / 8).to(torch.bfloat16)
    up = torch.randn(n, rank, V, generator=g, device="cuda").to(torch.bfloat16)
    norm = torch.ones(H, device="cuda")
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    of = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    top_ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32)
    top = torch.randn(T, K, generator=g, device="cuda")

    leaves = [t.clone().requires_grad_(True) for t in (table, norm, down, up)]
    x = autograd.embedding(ids, leaves[0], 8.0, out_dtype=torch.float32)
    y = autograd.layer_norm(x, leaves[1], out_dtype=torch.bfloat16)
    logits = autograd.adapters((y.float() @ leaves[0].float().t()), y, leaves[2], leaves[3], of)
    autograd.distill_logits(logits, top_ids, top).mean().backward()

    w, wn, d, u = [t.double().requires_grad_(True) for t in (table, norm, down, up)]
    x = w[ids.long()] * 8.0
    y = torch.nn.functional.layer_norm(x, (H,), wn, None, 1e-5)
    y = y + (y.detach().to(torch.bfloat16).double() - y.detach())        # rounded as the operator rounds
    share = torch.einsum("trh,th->tr", d[of.long().clamp_min(0)], y)
    share = torch.einsum("tr,trv->tv", share, u[of.long().clamp_min(0)])
    z = y @ w.t() + torch.where(of[:, None] >= 0, share, 0.0)
    p = torch.softmax(top.double(), 1)
    loss = (p * (p.log() - torch.log_softmax(z, 1).gather(1, top_ids.long()))).sum(1)
    loss.mean().backward()
    # bf16 gradients of bf16 leaves, and y's own rounding border: two bf16 roundings and the cotangents'
    for mine, ref in zip(leaves, (w, wn, d, u)):
        a, b = mine.grad.double(), ref.grad
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -7
