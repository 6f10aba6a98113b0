"""Layer norm, distillation and logit processing on rows taken out of larger tensors, and over
their own inputs: the bits of separate, packed tensors."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("B,S,V", [(4, 30, 5000), (3, 7, 3001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_last_position_of_a_batch(B, S, V, dtype):
    """What a decoding step has: logits[:, -1] of [B, S, V]."""
    ensure_built()
    every = randn(B, S, V, seed=1, dtype=dtype)
    last, packed = every[:, -1], every[:, -1].contiguous()
    g = torch.Generator("cuda").manual_seed(2)
    words = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
    tokens = torch.randint(0, V, (B * 20,), generator=g, device="cuda", dtype=torch.int32)
    begin = torch.arange(B, device="cuda") * 20
    rules = dict(tokens=tokens, spans=torch.stack([begin, begin + 5, begin + 20], 1),
                 repetition=torch.full((B,), 1.3, device="cuda"), allowed=words)
    ids = torch.randint(0, V, (B, 9), generator=g, device="cuda", dtype=torch.int32)
    top, grad = randn(B, 9, seed=3), randn(B, seed=4)

    def both(z):
        out = lm.process_logits(z, **rules)
        back = lm.process_logits_backward(z, z, **rules)
        loss, lse = lm.distill_logits_forward(z, ids, top)
        return out, back, lm.distill_logits_backward(z, ids, top, None, 1.0, 1.0, grad, lse), loss
    for name, a, b in zip(("process", "process backward", "distill backward", "loss"), both(last),
                          both(packed)):
        # (odd widths lie at another alignment packed, where a row's sums take another order)
        assert torch.equal(a, b) if V % 8 == 0 else torch.allclose(a, b, rtol=1e-2, atol=1e-6), name
        assert a.untyped_storage().nbytes() <= B * (V + 256) * a.element_size(), name


@pytest.mark.parametrize("N,H", [(40, 1001), (700, 999), (700, 1024), (9, 4500), (50, 5000), (20, 9001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("params", [False, True])
def test_layernorm_gradient_over_its_inputs(N, H, dtype, params):
    """dx over dy and over x, alone (wide rows then have no workspace for their sums) and with the
    weight's gradients."""
    ensure_built()
    x, dy = randn(N, H, seed=5, dtype=dtype), randn(N, H, seed=6, dtype=dtype)
    w = 1 + 0.1 * randn(H, seed=7)
    _, mean, rstd = lm.layernorm_forward(x, w)
    ws = torch.empty(lm.lmhead_layernorm_workspace_size(N, H), dtype=torch.uint8, device="cuda") \
        if params else None

    def call(dy, x, dx):
        dw, db = [torch.empty(H, device="cuda") if params else None for _ in range(2)]
        assert lm.lmhead_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, False, ws) == 0
        return [dx] + ([dw, db] if params else [])
    want = call(dy, x, torch.empty_like(x))
    over_dy, over_x = dy.clone(), x.clone()
    for got in (call(over_dy, x, over_dy), call(dy, over_x, over_x)):
        assert all(torch.equal(p, q) for p, q in zip(got, want))
