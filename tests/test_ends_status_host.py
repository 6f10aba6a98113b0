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
