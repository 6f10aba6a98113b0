"""Operands and results that are neighbours in one tensor: columns beside each other, stretches end to end."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("H", [64, 33])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_embedding_beside_its_table(H, dtype):
    g = torch.Generator("cuda").manual_seed(H)
    for N, first, step in ((20, 0, 1), (50, 0, 1), (20, 1, 2), (1, 7, 1)):
        ids = torch.randint(0, 50, (N,), generator=g, device="cuda", dtype=torch.int32)
        both = torch.randn(50, 2 * H, generator=g, device="cuda").to(dtype)
        before = both.clone()
        for table, other in ((both[:, :H], both[:, H:]), (both[:, H:], both[:, :H])):
            y = other[first::step][:N]
            assert lm.embedding_forward(ids, table, out=y) is y
            assert torch.equal(y, table[ids.long()])
            kept = before[:, :H] if table.data_ptr() == both.data_ptr() else before[:, H:]
            assert torch.equal(table, kept)
            both.copy_(before)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_gradient_end_to_end_with_its_cotangent(dtype):
    g = torch.Generator("cuda").manual_seed(3)
    N, V, H = 40, 30, 24
    flat = torch.randn((N + V) * H, generator=g, device="cuda").to(dtype)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    for dy, d in ((flat[:N * H], flat[N * H:]), (flat[V * H:], flat[:V * H])):
        dy, d = dy.view(N, H), d.view(V, H)
        want = lm.embedding_backward(dy, ids, V, dtype=dtype)
        lm.embedding_backward(dy, ids, V, d_weight=d)
        assert torch.equal(d, want)
    with pytest.raises(lm.LmheadError):
        lm.embedding_backward(flat[:N * H].view(N, H), ids, V, d_weight=flat[(N - 1) * H:(N - 1 + V) * H].view(V, H))
    with pytest.raises(lm.LmheadError):
        lm.embedding_forward(ids[:5], flat[:V * H].view(V, H), out=flat[H:6 * H].view(5, H))


@pytest.mark.parametrize("V", [128, 51])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_adapters_beside_their_base(V, dtype):
    g = torch.Generator("cuda").manual_seed(V)
    T, H, rank, n = 70, 40, 5, 3
    both = torch.randn(T, 2 * V, generator=g, device="cuda").to(dtype)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    down, up = (torch.randn(n, rank, w, generator=g, device="cuda").to(BF16) for w in (H, V))
    of = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    before = both.clone()
    for base, out in ((both[:, :V], both[:, V:]), (both[:, V:], both[:, :V])):
        want = lm.adapters_forward(base.contiguous(), x, down, up, of)
        kept = base.clone()
        assert lm.adapters_forward(base, x, down, up, of, out=out) is out
        assert torch.equal(out, want) and torch.equal(base, kept)
        both.copy_(before)
    with pytest.raises(lm.LmheadError):
        lm.adapters_forward(both[:-1, :V], x[:-1], down, up, of[:-1], out=both[1:, :V])
    # every gradient and the cotangent end to end
    flat = torch.zeros(T * V + T * H + n * rank * (H + V), device="cuda")
    grad, dx, d_down, d_up = (t.view(s) for t, s in zip(flat.split([T * V, T * H, n * rank * H, n * rank * V]),
                                                      ((T, V), (T, H), (n, rank, H), (n, rank, V))))
    grad.copy_(torch.randn(T, V, generator=g, device="cuda"))
    want = lm.adapters_backward(grad.clone(), x, down, up, of)
    lm.adapters_backward(grad, x, down, up, of, dx=dx, d_down=d_down, d_up=d_up)
    assert torch.equal(dx, want[0]) and torch.equal(d_down, want[1]) and torch.equal(d_up, want[2])
    # dx beside another matrix
    wide = torch.zeros(T, 2 * H, device="cuda")
    lm.adapters_backward(grad, x, down, up, of, dx=wide[:, H:])
    assert torch.equal(wide[:, H:], want[0]) and not wide[:, :H].any()


def test_selection_out_of_one_buffer():
    """Results end to end, scores and flags in place, and scores kept behind each row of logits."""
    g = torch.Generator("cuda").manual_seed(9)
    wide = torch.randn(8, 1000 + 8, generator=g, device="cuda")
    z = wide[:, :1000]
    s = -torch.rand(8, generator=g, device="cuda")
    f = torch.tensor([0, 1, 0, 0, 0, 0, 1, 0], dtype=torch.uint8, device="cuda")
    nxt = torch.empty(2, 4, dtype=torch.uint8, device="cuda")
    want = lm.beam_select(z, s, 4, 4, 1.0, f, 5, nxt)
    flat = torch.zeros(32, device="cuda")
    mine, lse = flat[:8], flat[24:]
    mine.copy_(s)
    p, t = (flat[8 * i:8 * i + 8].view(torch.int32).view(2, 4) for i in (1, 2))
    ws = torch.empty(lm.lmhead_beam_workspace_size(8, 1000, 4), dtype=torch.uint8, device="cuda")
    assert lm.lmhead_beam_select(z, 4, 4, mine, f, 5, 1.0, mine.view(2, 4), p, t, f.view(2, 4), lse, ws) == 0
    for a, b in zip((mine.view(2, 4), p, t, lse, f.view(2, 4)), (*want, nxt)):
        assert torch.equal(a, b)
    # a result in the columns behind the logits
    out = wide[0, 1000:].view(2, 4)
    f.copy_(torch.tensor([0, 1, 0, 0, 0, 0, 1, 0]))
    assert lm.lmhead_beam_select(z, 4, 4, s, f, 5, 1.0, out, p, t, None, None, ws) == 0
    assert torch.equal(out, want[0])


def test_reorder_of_a_state_without_rows():
    parents = torch.tensor([-1, 0, -1], dtype=torch.int32, device="cuda")
    for shape, dim in (((0, 5), 0), ((2, 0, 3, 4), 1), ((2, 0, 3, 7), 1)):
        state = torch.empty(shape, device="cuda")
        full = [*shape]
        full[dim] = 3
        got = lm.beam_reorder(state, parents, dim)
        assert got.shape == tuple(full) and not got.any()
        kept = torch.ones(full, device="cuda")
        assert lm.beam_reorder(state, parents, dim, kept) is kept and (kept == 1).all()
