"""Adapters in a workspace of exactly the size asked for, between guard bytes, where rows are split."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built
from test_gpu_adapters import BF16, F32, check_backward, check_forward, make
from test_gpu_guard_canaries import Guarded, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("T,H,V,rank,n", [(511, 64, 264, 5, 1), (1300, 64, 264, 5, 1), (2100, 33, 70, 20, 2),
                                          (1, 600, 1100, 128, 1), (131072 + 600, 16, 24, 3, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_workspace_of_the_asked_size(T, H, V, rank, n, dtype):
    s = make(T, H, V, rank, n, dtype, T)
    args = [s[k] for k in ("x", "down", "up", "of", "scale")]
    size = lm.lmhead_adapters_workspace_size(T, H, V, rank, n)
    ws = Guarded((size,), torch.uint8, 31)
    out = lm.adapters_forward(s["base"], *args, workspace=ws.t)
    _check({}, dict(ws=ws), "fwd")
    check_forward(s, out)
    ws = Guarded((size,), torch.uint8, 32)
    grads = lm.adapters_backward(s["grad"], *args, workspace=ws.t)
    _check({}, dict(ws=ws), "bwd")
    check_backward(s, *grads, extra=2)
    if T > 1:
        small = torch.empty(size - 1, dtype=torch.uint8, device="cuda")
        with pytest.raises(lm.LmheadError):
            lm.adapters_forward(s["base"], *args, workspace=small)
