"""Beam selection where different logits have one score in 64 bits."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def best(row, take):
    """Ids by falling logit, equal ones by id."""
    return np.argsort(-row.double().cpu().numpy(), kind="stable")[:take]


@pytest.mark.parametrize("R", [1, 40, 400])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V,take", [(8192, 8), (50257, 16), (3000, 128)])
def test_a_large_temperature_keeps_the_order_of_the_logits(R, dtype, V, take):
    """At 1e12 some 15 logits of every 8,192 between 0 and 1 share a score: the order is the
    logits', in however many pieces a row is read."""
    g = torch.Generator("cuda").manual_seed(V)
    ramp = torch.arange(V, device="cuda", dtype=F32) / V
    z = torch.stack([ramp[torch.randperm(V, generator=g, device="cuda")] for _ in range(min(R, 8))])
    z = z.repeat((R + 7) // 8 if R > 8 else 1, 1)[:R].to(dtype)
    scores, parents, tokens, _ = lm.beam_select(z, torch.zeros(R, device="cuda"), 1, take, 1e12)
    for r in list(range(min(R, 8))) + [R - 1]:
        assert tokens[r].tolist() == best(z[r], take).tolist()
        assert (parents[r] == r).all()
    assert torch.isfinite(scores).all()


def test_equal_scores_go_to_the_lowest_beam_first():
    """Beams of equal rows and scores (on 16-byte boundaries): all of the first beam's logits that share
    the best score come before the second's."""
    V, take = 4096, 6
    z = (torch.arange(V, device="cuda", dtype=F32).flip(0) / V * 2.0 ** -20).repeat(8, 1)
    scores, parents, tokens, _ = lm.beam_select(z, torch.zeros(8, device="cuda"), 4, take, 1e12)
    assert (scores == scores[0, 0]).all()
    assert parents.tolist() == [[0] * take, [4] * take]
    assert tokens.tolist() == [list(range(take))] * 2
    # against the order of ids: the largest logits are last now
    z = z.flip(1).contiguous()
    _, parents, tokens, _ = lm.beam_select(z, torch.zeros(8, device="cuda"), 4, take, 1e12)
    assert parents.tolist() == [[0] * take, [4] * take]
    assert tokens.tolist() == [list(range(V - 1, V - 1 - take, -1))] * 2


def test_large_scores_and_subnormal_temperatures_keep_the_order_of_the_logits():
    g = torch.Generator("cuda").manual_seed(2)
    z = torch.randn(8, 5000, generator=g, device="cuda")
    # scores whose step in 64 bits is 2^47
    _, parents, tokens, _ = lm.beam_select(z, torch.full((8,), -1e30, device="cuda"), 1, 5)
    for r in range(8):
        assert tokens[r].tolist() == best(z[r], 5).tolist() and (parents[r] == r).all()
    # log p is 0 for a row's largest logit and next to -1e40 for the others
    _, parents, tokens, _ = lm.beam_select(z, torch.zeros(8, device="cuda"), 4, 4, 1e-40)
    assert parents.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7]]
    assert tokens.view(-1).tolist() == [int(best(z[r], 1)[0]) for r in range(8)]
    _, parents, tokens, _ = lm.beam_select(z, torch.zeros(8, device="cuda"), 1, 4, 1e-40)
    for r in range(8):
        assert tokens[r].tolist() == best(z[r], 4).tolist()


@pytest.mark.parametrize("G,K,V,take", [(1, 64, 50257, 128), (3, 64, 4100, 64), (2, 16, 30011, 128), (1, 3, 151936, 100),
                                        (1, 1, 2048, 128), (5, 61, 9000, 127)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_many_continuations_of_many_beams(G, K, V, take, dtype):
    from test_gpu_beam import check, logits_of
    gen = torch.Generator("cuda").manual_seed(K + take)
    z = logits_of(G * K, V, dtype, gen)
    s = -torch.rand(G * K, generator=gen, device="cuda")
    check(z, s, K, take)
    f = (torch.rand(G * K, generator=gen, device="cuda") < 0.5).to(torch.uint8)
    check(z, s, K, take, 0.7, f, 3)
    check(z, torch.where(f != 0, -float("inf"), s), K, take)
