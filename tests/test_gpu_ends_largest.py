"""The largest sizes that embedding, adapters and beam selection take."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
MOST = 2 ** 31 - 1025


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def test_embedding_of_the_largest_vocabulary():
    table = torch.zeros(MOST, 1, dtype=BF16, device="cuda")
    where = torch.tensor([MOST - 1, 0, MOST // 2, 12345, MOST - 70000], device="cuda")
    table[where, 0] = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0], device="cuda").to(BF16)
    ids = torch.cat([where, where - MOST, where.new_tensor([MOST, -MOST - 1])]).to(torch.int32)
    y = lm.embedding_forward(ids, table, 2.0)
    assert y[:10, 0].tolist() == [2.0, 4.0, 6.0, 8.0, 10.0] * 2 and torch.isnan(y[10:]).all()
    del table
    for n, dtype in ((12, BF16), (12, F32), (3000, F32)):
        many = ids.repeat((n + 11) // 12)
        d = torch.full((MOST, 1), float("nan"), dtype=dtype, device="cuda")
        lm.embedding_backward(torch.ones(len(many), 1, device="cuda"), many, MOST, d_weight=d)
        assert (d[where, 0] == 2.0 * len(many) / 12).all()
        assert int(d.count_nonzero()) == 5 and float(d.sum(dtype=F32)) == 10.0 * len(many) / 12
        del d


@pytest.mark.parametrize("V", [MOST, MOST - 7])       # rows off and on 16-byte boundaries
def test_adapters_of_the_widest_projection(V):
    at = torch.tensor([0, 7, 8, V // 2, V - 9, V - 1], device="cuda")
    up = torch.zeros(1, 1, V, dtype=BF16, device="cuda")
    up[0, 0, at] = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0, 6.0], device="cuda").to(BF16)
    x, down = torch.ones(1, 8, dtype=BF16, device="cuda"), torch.ones(1, 1, 8, dtype=BF16, device="cuda")
    base = torch.zeros(1, V, dtype=BF16, device="cuda")
    lm.adapters_forward(base, x, down, up, out=base)
    assert (base[0, at] == 8 * up[0, 0, at]).all() and int(base.count_nonzero()) == 6
    # du = sum of 8 i^2 = 728
    dx, d_down, d_up = lm.adapters_backward(base, x, down, up)
    assert (dx == 728).all() and (d_down == 728).all()
    assert (d_up[0, 0, at] == 64 * up[0, 0, at].float()).all() and int(d_up.count_nonzero()) == 6


def test_adapters_of_the_widest_rows():
    x = torch.zeros(1, MOST, dtype=BF16, device="cuda")
    down = torch.zeros(1, 1, MOST, dtype=BF16, device="cuda")
    x[0, -3:] = 2.0
    down[0, 0, -2:] = 3.0
    up, base = torch.ones(1, 1, 8, dtype=BF16, device="cuda"), torch.zeros(1, 8, device="cuda")
    assert (lm.adapters_forward(base, x, down, up) == 12).all()
    dx, d_down, d_up = lm.adapters_backward(torch.ones(1, 8, device="cuda"), x, down, up)
    assert (dx[0, -2:] == 24).all() and int(dx.count_nonzero()) == 2
    assert (d_down[0, 0, -3:] == 16).all() and int(d_down.count_nonzero()) == 3 and (d_up == 12).all()


@pytest.mark.parametrize("R", [1, 2])
def test_selection_of_the_largest_vocabulary(R):
    V = 2 ** 30
    z = torch.zeros(R, V, dtype=BF16, device="cuda")
    z[-1, -1], z[-1, 0], z[0, V // 2 + 3] = 40.0, 39.0, 38.0
    scores, parents, tokens, lse = lm.beam_select(z, torch.zeros(R, device="cuda"), 1, 3)
    assert tokens[-1, :2].tolist() == [V - 1, 0] and tokens[0, 0] == (V - 1 if R == 1 else V // 2 + 3)
    assert tokens[-1, 2] == (V // 2 + 3 if R == 1 else 1) and (parents[:, 0].cpu() == torch.arange(R)).all()
    e = torch.tensor([40.0, 39.0, 38.0], dtype=torch.float64).exp()
    want = (e.sum() + V - 3).log() if R == 1 else (e[:2].sum() + V - 2).log()
    assert abs(float(lse[-1]) - float(want)) <= 1e-5 + 40 * 2.0 ** -23
