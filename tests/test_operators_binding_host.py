"""Host-side pieces of the binding of layer norm, distillation and logit processing (no GPU)."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,S,V", [(4, 300, 1000), (3, 50, 1001), (2, 2, 777), (5, 1, 64)])
def test_results_of_one_position_of_many_take_the_room_of_one(dtype, B, S, V):
    """logits[:, -1] of [B, S, V]: its rows lie S V apart, the result's need not."""
    logits = torch.empty(B, S, V, dtype=dtype)[:, -1]
    out = lm._rows_like(logits)
    assert out.shape == logits.shape and out.dtype == dtype and out.stride(1) == 1
    assert out.untyped_storage().nbytes() <= B * (V + 256) * dtype.itemsize
    # the kernels move 16 bytes at a time where both sides' rows have the same alignment
    assert (out.stride(0) - logits.stride(0)) * dtype.itemsize % 16 == 0


def test_results_keep_a_padded_tables_layout():
    for pad in (0, 1, 64, 256):
        logits = torch.empty(7, 1000 + pad, dtype=torch.bfloat16)[:, :1000]
        assert lm._rows_like(logits).stride() == logits.stride()


def test_workspace_sizes_are_not_remembered_without_end():
    """A trainer with packed rows asks for another length every step."""
    lm.build()
    ask = lm.lmhead_layernorm_workspace_size
    want = [ask(n, 64) for n in range(1, 3001)]
    kept = ask.cache_info().currsize if hasattr(ask, "cache_info") else 0
    assert kept <= 256
    assert want == [ask(n, 64) for n in range(1, 3001)]
