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
