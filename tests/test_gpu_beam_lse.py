"""lse of beam selection where the terms of its sum are equal, so that their roundings do not cancel."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# A term is off by the exponential's 2^-22, and by two roundings of its argument, which is below 15 here:
# (4 + 2 * 15) 2^-24.  A thread adds up to 16 terms of a tile and the sums of its tiles, of 4,096 fp32 or
# 8,192 16-bit elements; then 5 steps over lanes, 8 warps and the roundings of the join.
def tolerance(V, dtype):
    tiles = -(-V // (4096 if dtype is F32 else 8192))
    return (34 + 16 + tiles + 5 + 8 + 6) * 2.0 ** -24


@pytest.mark.parametrize("R,V", [(1000, 151936), (1000, 50257), (608, 151936), (256, 151936), (1000, 9000), (4, 151936),
                                 (150, 1 << 20)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_equal_logits_below_one(R, V, dtype):
    z = torch.full((R, V), -3.7, device="cuda") - torch.arange(R, device="cuda")[:, None] * 0.01
    z[:, 5] = 1.0
    z = z.to(dtype)
    _, _, tokens, lse = lm.beam_select(z, torch.zeros(R, device="cuda"), 1, 1)
    low = z[:, 6].double()
    want = torch.log(torch.exp(torch.tensor(1.0, dtype=torch.float64)) + (V - 1) * torch.exp(low))
    off = (lse.double() - want).abs() - 2.0 ** -24 * want.abs()
    assert (tokens == 5).all()
    assert float(off.max()) <= tolerance(V, dtype), (float(off.max()), tolerance(V, dtype))
