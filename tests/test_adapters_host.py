"""Refusals of the adapter calls (CPU only: each is decided before anything is launched)."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from chunked_lm_head_tcgen05_gb300 import autograd
from test_operators_host import INVALID, OK, P, SMALL, UNSUPPORTED, call, lib  # noqa: F401

OTHER = [P((1 << 20) + 4096 * (i + 1)) for i in range(6)]
FWD = dict(base=P(), type=1, base_ld=100, x=OTHER[0], x_ld=64, down=OTHER[1], up=OTHER[2], ids=P(), scale=P(),
           T=8, H=64, V=100, rank=4, n=3, out=P(), out_ld=100, workspace=P(), bytes=1 << 30, stream=None)
BWD = dict(grad=P(), type=1, ld=100, x=OTHER[0], x_ld=64, down=OTHER[1], up=OTHER[2], ids=P(), scale=P(), T=8,
           H=64, V=100, rank=4, n=3, dx=OTHER[3], dx_ld=64, accumulate_dx=0, d_down=OTHER[4], d_up=OTHER[5],
           accumulate=0, workspace=P(), bytes=1 << 30, stream=None)
BOTH = [(dict(x=None), INVALID), (dict(down=None), INVALID), (dict(up=None), INVALID),
        (dict(workspace=None), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(V=0), INVALID),
        (dict(rank=0), INVALID), (dict(n=0), INVALID), (dict(type=3), INVALID), (dict(x_ld=63), INVALID),
        (dict(rank=129), UNSUPPORTED), (dict(n=65536), UNSUPPORTED), (dict(T=(1 << 31) - 256), UNSUPPORTED),
        (dict(x=P((1 << 20) + 1)), UNSUPPORTED), (dict(down=P((1 << 20) + 1)), UNSUPPORTED),
        (dict(up=P((1 << 20) + 1)), UNSUPPORTED), (dict(ids=P((1 << 20) + 2)), UNSUPPORTED),
        (dict(scale=P((1 << 20) + 2)), UNSUPPORTED), (dict(workspace=P((1 << 20) + 128)), UNSUPPORTED),
        (dict(H=2 ** 31 - 1024, x_ld=1 << 31, dx_ld=1 << 31), UNSUPPORTED), (dict(bytes=512), SMALL)]

CASES = [
    ("lmhead_adapters_fwd", FWD, BOTH + [
        (dict(base=None), INVALID), (dict(out=None), INVALID), (dict(base_ld=99), INVALID),
        (dict(out_ld=99), INVALID), (dict(out_ld=128), INVALID), (dict(out=OTHER[0]), INVALID),
        (dict(out=OTHER[2]), INVALID), (dict(base=P((1 << 20) + 1)), UNSUPPORTED),
        (dict(V=1 << 30, base_ld=1 << 30, out_ld=1 << 30, T=1 << 17, n=60000), UNSUPPORTED),
        (dict(T=0, base=None, x=None), OK)]),
    ("lmhead_adapters_bwd", BWD, BOTH + [
        (dict(grad=None), INVALID), (dict(dx=None, d_down=None, d_up=None), INVALID), (dict(ld=99), INVALID),
        (dict(dx_ld=63), INVALID), (dict(dx=P()), INVALID), (dict(d_up=OTHER[4]), INVALID),
        (dict(dx=OTHER[5]), INVALID), (dict(d_down=OTHER[1]), INVALID),
        (dict(dx=P((1 << 20) + 2)), UNSUPPORTED), (dict(grad=P((1 << 20) + 1)), UNSUPPORTED),
        (dict(T=0, d_down=None, d_up=None), OK), (dict(T=0, accumulate=1), OK)]),
]


@pytest.mark.parametrize("name,defaults,wrong", CASES, ids=[c[0] for c in CASES])
def test_refusals(lib, name, defaults, wrong):  # noqa: F811
    assert len(defaults) == len(lm._SIGNATURES[name][1])
    for over, status in wrong:
        over = {k: v for k, v in over.items() if k in defaults}
        assert call(getattr(lib, name), defaults, **over) == status, (name, over)


def test_workspace_sizes(lib):  # noqa: F811
    size = lm.lmhead_adapters_workspace_size
    for bad in ((-1, 64, 100, 4, 3), (8, 0, 100, 4, 3), (8, 64, 0, 4, 3), (8, 64, 100, 0, 3),
                (8, 64, 100, 129, 3), (8, 64, 100, 4, 0), (8, 64, 100, 4, 65536)):
        assert size(*bad) == 0
    assert size(0, 64, 100, 4, 3) > 0
    # sorted rows, u and its gradient in three bf16 parts of 16 ranks, one sum of each at least
    for T, rank in ((1, 1), (100, 16), (5000, 33)):
        r = -(-rank // 16) * 16
        assert size(T, 64, 100, rank, 3) >= T * (8 + 2 * 6 * r + 4 * r)
    assert size(1 << 20, 64, 100, 4, 3) == size(131072, 64, 100, 4, 3)      # parts in turn


def test_binding():
    base, x = torch.zeros(4, 10), torch.zeros(4, 8, dtype=torch.bfloat16)
    down, up = (torch.zeros(2, 3, n, dtype=torch.bfloat16) for n in (8, 10))
    with pytest.raises(ValueError):
        lm.adapters_forward(base, x, down, up)            # not on a GPU
    with pytest.raises(TypeError):
        lm.adapters_forward(base, x.float(), down, up)
    with pytest.raises(lm.LmheadError):
        lm.adapters_forward(base, x, down, torch.zeros(2, 129, 10, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        autograd.adapters(base, x, down, up, None, torch.ones(2, requires_grad=True))
