"""The table's gradient where zeros are written beside the sort, by the summing launch, or by both."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# (tokens, vocabulary, width): tables below and above 256 MB, few and many tokens for them, odd widths
@pytest.mark.parametrize("N,V,H", [(1, 100, 8), (1024, 33000, 64), (1025, 33000, 64), (1500, 60000, 33), (16, 151936, 512),
                                   (1024, 151936, 441), (1024, 151936, 442), (4096, 151936, 2560), (1000, 900, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_row_is_written_once_or_zero(N, V, H, dtype):
    g = torch.Generator("cuda").manual_seed(N + V)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    ids[N // 2:] = V // 5                          # an id that many tokens share
    ids[N // 3] = V - 1
    dy = torch.randint(-8, 9, (N, H), generator=g, device="cuda").to(BF16)        # exact sums
    d = torch.full((V, H), float("nan"), device="cuda", dtype=dtype)
    lm.embedding_backward(dy, ids, V, d_weight=d)
    want = torch.zeros(V, H, device="cuda").index_add_(0, ids.long(), dy.float())
    assert torch.equal(d, want.to(dtype))
