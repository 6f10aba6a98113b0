"""What the calls of embedding, adapters and beam search refuse on the host (CPU only), and with which status."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd
from test_operators_host import lib  # noqa: F401

BF16 = torch.bfloat16


def expanded(*shape):
    return torch.zeros([1] * len(shape), dtype=BF16).expand(*shape)


CALLS = [lm.adapters_forward, lm.adapters_backward, autograd.adapters]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("T,H,V,rank,n,status", [
    (4, 8, 10, 129, 2, 2), (4, 8, 10, 3, 65536, 2), (4, 8, 2 ** 31 - 1024, 3, 2, 2), (4, 2 ** 31 - 1, 8, 3, 2, 2),
    (1 << 17, 8, 1 << 30, 4, 60000, 2),        # more tiles than a grid has
    (4, 0, 10, 3, 2, 1), (4, 8, 10, 0, 2, 1), (4, 8, 10, 3, 0, 1)])
def test_sizes_that_adapters_do_not_take(lib, call, T, H, V, rank, n, status):  # noqa: F811
    base, x = expanded(T, V), expanded(T, H)
    more = {} if call is autograd.adapters else dict(
        out=base) if call is lm.adapters_forward else dict(dx=x, d_down=x, d_up=x)
    with pytest.raises(lm.LmheadError) as e:
        call(base, x, expanded(n, rank, H), expanded(n, rank, V), **more)
    assert e.value.status == status


HUGE = 2 ** 32 + 10        # cut to 32 bits it would be 10


class OnDevice(torch.Tensor):
    """A tensor that says it lies on a GPU: what follows the check of its sizes is not reached."""
    is_cuda = True

    def is_contiguous(self):
        return True


def far(*shape, dtype=BF16):
    one = torch.zeros([1] * len(shape), dtype=dtype)
    return (one.expand(*shape) if HUGE in shape else one.expand(*shape).contiguous()).as_subclass(OnDevice)


def test_sizes_past_32_bits(lib):  # noqa: F811
    one, f32, i32 = far(1, 8), torch.float32, torch.int32
    ids, scores = far(1, dtype=i32), far(1, dtype=f32)
    calls = [
        lambda: lm.lmhead_embedding_fwd(ids, far(HUGE, 8), 1.0, far(1, 8)),
        lambda: lm.lmhead_embedding_fwd(ids, far(8, HUGE), 1.0, far(1, HUGE)),
        lambda: lm.embedding_forward(ids, far(HUGE, 8)),
        lambda: lm.lmhead_embedding_bwd(one, ids, 1.0, None, far(HUGE, 8, dtype=f32), False, one),
        lambda: lm.embedding_backward(one, ids, HUGE, d_weight=far(HUGE, 8, dtype=f32), workspace=one),
        lambda: lm.adapters_forward(far(1, HUGE), one, far(2, 3, 8), far(2, 3, HUGE), out=far(1, HUGE)),
        lambda: lm.lmhead_adapters_fwd(far(1, HUGE), one, far(2, 3, 8), far(2, 3, HUGE), None, None, far(1, HUGE), one),
        lambda: lm.lmhead_adapters_bwd(one, far(1, HUGE), far(2, 3, HUGE), far(2, 3, 8), None, None, None, False,
                                       None, None, False, one),
        lambda: lm.lmhead_adapters_fwd(one, one, far(HUGE, 3, 8), far(HUGE, 3, 8), None, None, one, one),
        lambda: autograd.adapters(one, one, far(2, HUGE, 8), far(2, HUGE, 8)),
        lambda: lm.beam_select(far(1, HUGE), scores, 1),
        lambda: lm.beam_select(one, scores, 1, 2 ** 32 + 1),
        lambda: lm.lmhead_embedding_workspace_size(1, HUGE),
        lambda: lm.lmhead_adapters_workspace_size(1, 8, HUGE, 3, 2),
        lambda: lm.lmhead_beam_workspace_size(1, HUGE, 1),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(lm.LmheadError) as e:
            call()
        assert e.value.status == 2, i


def test_few_rows_need_a_small_workspace(lib):  # noqa: F811
    """Sums of row splits, which only a gradient over many rows has, are not asked for."""
    size = lm.lmhead_adapters_workspace_size
    for T, n in ((1, 1), (16, 1), (64, 16), (200, 4)):
        for H, V, rank in ((2560, 2560, 128), (64, 2560, 16), (2560, 10240, 64)):
            r = -(-rank // 16) * 16
            # places and lists of every row and adapter; u and du in three bf16 parts, and their sums of
            # at most one per 512 columns
            most = T * (8 + 32 + 2 * 6 * r + 4 * r * (-(-H // 512) + -(-V // 512))) + 36 * n + 64 + 10 * 256
            assert size(T, H, V, rank, n) <= most, (T, H, V, rank, n, size(T, H, V, rank, n), most)
