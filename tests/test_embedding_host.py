"""Refusals of the embedding calls (CPU only: each is decided before anything is launched)."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd
from test_operators_host import INVALID, OK, P, SMALL, UNSUPPORTED, call, lib  # noqa: F401

FWD = dict(ids=P(), N=8, weight=P(), type=1, w_ld=64, V=100, H=64, scale=1.0, y=P(1 << 21), y_type=1,
           y_ld=64, stream=None)
BWD = dict(dy=P(), dy_type=1, dy_ld=64, ids=P(), N=8, V=100, H=64, scale=1.0,
           padding=lm.NO_PADDING, d_weight=P(1 << 21), d_type=0, accumulate=0, workspace=P(),
           bytes=1 << 30, stream=None)

CASES = [
    ("lmhead_embedding_fwd", FWD, [
        (dict(ids=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
        (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(H=0), INVALID), (dict(w_ld=63), INVALID),
        (dict(y_ld=63), INVALID), (dict(type=3), INVALID), (dict(y_type=-1), INVALID),
        (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
        (dict(y=P()), INVALID), (dict(type=1, y_type=2), UNSUPPORTED),
        (dict(type=0, y_type=2), UNSUPPORTED), (dict(type=2, y_type=1), UNSUPPORTED),
        (dict(N=(1 << 31) - 256), UNSUPPORTED), (dict(V=2 ** 31 - 1024), UNSUPPORTED),
        (dict(H=(1 << 20) + 1, w_ld=1 << 21, y_ld=1 << 21), UNSUPPORTED),
        (dict(weight=P((1 << 20) + 1)), UNSUPPORTED), (dict(y=P((1 << 21) + 1)), UNSUPPORTED),
        (dict(ids=P((1 << 20) + 2)), UNSUPPORTED), (dict(N=0, ids=None, y=None), OK)]),
    ("lmhead_embedding_bwd", BWD, [
        (dict(dy=None), INVALID), (dict(ids=None), INVALID), (dict(d_weight=None), INVALID),
        (dict(workspace=None), INVALID), (dict(dy_ld=63), INVALID), (dict(N=-1), INVALID),
        (dict(padding=100), INVALID), (dict(padding=-101), INVALID), (dict(dy_type=3), INVALID),
        (dict(scale=float("nan")), INVALID), (dict(d_weight=P()), INVALID),
        (dict(d_type=2), UNSUPPORTED), (dict(d_type=1, accumulate=1), UNSUPPORTED),
        (dict(d_type=1, N=131073), UNSUPPORTED), (dict(d_weight=P((1 << 21) + 2)), UNSUPPORTED),
        (dict(dy=P((1 << 20) + 1)), UNSUPPORTED), (dict(workspace=P((1 << 20) + 128)), UNSUPPORTED),
        (dict(V=2 ** 31 - 1024), UNSUPPORTED), (dict(bytes=1024), SMALL),
        (dict(N=0, accumulate=1, dy=None, ids=None, d_weight=None, workspace=None), OK)]),
]


@pytest.mark.parametrize("name,defaults,wrong", CASES, ids=[c[0] for c in CASES])
def test_refusals(lib, name, defaults, wrong):  # noqa: F811
    assert len(defaults) == len(lm._SIGNATURES[name][1])
    for over, status in wrong:
        assert call(getattr(lib, name), defaults, **over) == status, (name, over)


def test_workspace_sizes(lib):  # noqa: F811
    size = lm.lmhead_embedding_workspace_size
    assert size(-1, 64) == size(4, 0) == size(4, (1 << 20) + 1) == size((1 << 31) - 256, 64) == 0
    assert size(1 << 20, 64) == size(131072, 64)          # parts of 131,072 tokens in turn
    sizes = [size(n, 64) for n in (0, 1, 1000, 8191, 8192, 20000, 32768, 32769, 65536, 131072)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    for n in (1, 1000, 8191, 8192, 65536, 131072):
        segments = -(-n // (8 if n < 8192 else 32))
        assert size(n, 64) >= 256 + 8 * n + 2 * 4 * 64 * segments


def test_binding():
    ids, w = torch.zeros(4, dtype=torch.int32), torch.zeros(10, 8)
    with pytest.raises(ValueError):
        lm.embedding_forward(ids, w)                       # not on a GPU
    with pytest.raises(ValueError):
        lm.embedding_forward(ids.view(2, 2), w, out=torch.empty(2, 2, 8))
    with pytest.raises(TypeError):
        lm.embedding_forward(ids.long(), w)
    with pytest.raises(ValueError):
        lm.embedding_backward(torch.zeros(4, 8), ids, 11, d_weight=torch.zeros(10, 8),
                              workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        autograd.embedding(ids, w, main_grad=torch.zeros(9, 8))
    for padding in (10, -11, 2 ** 32 + 3):
        with pytest.raises(ValueError):
            autograd.embedding(ids, w, padding_id=padding)
