"""Refusals of the beam search calls (CPU only: each is decided before anything is launched)."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from test_operators_host import INVALID, OK, P, SMALL, UNSUPPORTED, call, lib  # noqa: F401

SELECT = dict(logits=P(), type=0, ld=100, R=8, V=100, beams=4, take=8, scores=P(), finished=P(), eos=2,
              tau=1.0, out=P(1 << 22), parents=P(), tokens=P(), next=P(1 << 23), lse=P(), workspace=P(),
              bytes=1 << 30, stream=None)
A, B = 1 << 20, 1 << 24
REORDER = dict(src=P(A), so=8 * 640, sr=640, sm=320, src_rows=8, dst=P(B), do=8 * 640, dr=640, dm=320,
               parents=P(), rows=8, beams=4, outer=2, mid=2, inner=320, clear=0, stream=None)
IN_PLACE = dict(REORDER, dst=P(A))

CASES = [
    ("lmhead_beam_select", SELECT, [
        (dict(logits=None), INVALID), (dict(scores=None), INVALID), (dict(out=None), INVALID),
        (dict(parents=None), INVALID), (dict(tokens=None), INVALID), (dict(workspace=None), INVALID),
        (dict(R=-4), INVALID), (dict(R=9), INVALID), (dict(V=0), INVALID), (dict(beams=0), INVALID),
        (dict(take=0), INVALID), (dict(type=3), INVALID), (dict(ld=99), INVALID),
        (dict(tau=0.0), INVALID), (dict(tau=float("nan")), INVALID), (dict(eos=-1), INVALID),
        (dict(eos=100), INVALID), (dict(eos=-2, finished=None), INVALID),
        (dict(beams=65, R=65), UNSUPPORTED), (dict(take=129), UNSUPPORTED),
        (dict(R=(1 << 31) - 256), UNSUPPORTED), (dict(V=(1 << 30) + 1, ld=1 << 31), UNSUPPORTED),
        (dict(logits=P((1 << 20) + 2)), UNSUPPORTED), (dict(workspace=P((1 << 20) + 16)), UNSUPPORTED),
        (dict(scores=P((1 << 20) + 2)), UNSUPPORTED), (dict(lse=P((1 << 20) + 1)), UNSUPPORTED),
        (dict(out=P()), INVALID), (dict(out=P((1 << 20) + 28)), INVALID), (dict(next=P()), INVALID),
        (dict(out=P(), take=4, next=P((1 << 20) + 7)), INVALID),
        (dict(out=P(), next=P(), take=4, bytes=128), SMALL),
        (dict(bytes=128), SMALL), (dict(R=0, logits=None), OK)]),
    ("lmhead_beam_reorder", REORDER, [
        (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(parents=None), INVALID),
        (dict(rows=-1), INVALID), (dict(src_rows=-1), INVALID), (dict(outer=-1), INVALID),
        (dict(mid=-1), INVALID), (dict(inner=-1), INVALID), (dict(sr=-640), INVALID),
        (dict(do=-1), INVALID), (dict(dst=P(A + 640)), INVALID), (dict(dst=P(A + 16 * 640 - 1)), INVALID),
        (dict(dr=320), INVALID), (dict(dm=319), INVALID), (dict(do=0), INVALID),
        (dict(dr=1 << 62, rows=1 << 30), INVALID),
        (dict(parents=P((1 << 20) + 2)), UNSUPPORTED), (dict(rows=(1 << 31) - 256), UNSUPPORTED),
        (dict(rows=0, src=None), OK), (dict(inner=0, dst=None), OK), (dict(mid=0), OK),
        (dict(outer=0), OK)]),
    ("lmhead_beam_reorder", IN_PLACE, [
        (dict(sr=1280), INVALID), (dict(so=16 * 640), INVALID), (dict(src_rows=9), INVALID),
        (dict(beams=0), INVALID), (dict(beams=3), INVALID), (dict(beams=-4), INVALID),
        (dict(rows=130, src_rows=130, beams=65, so=130 * 640, do=130 * 640), UNSUPPORTED)]),
]


@pytest.mark.parametrize("name,defaults,wrong", CASES, ids=["select", "reorder", "in place"])
def test_refusals(lib, name, defaults, wrong):  # noqa: F811
    assert len(defaults) == len(lm._SIGNATURES[name][1])
    for over, status in wrong:
        assert call(getattr(lib, name), defaults, **over) == status, (name, over)


def test_workspace_sizes(lib):  # noqa: F811
    size = lm.lmhead_beam_workspace_size
    assert size(-1, 100, 4) == size(4, 0, 4) == size(4, 100, 0) == size(4, 100, 129) == 0
    assert size(4, (1 << 30) + 1, 4) == size((1 << 31) - 256, 100, 4) == 0
    assert size(0, 100, 4) > 0
    # every row's statistics and candidates, of one piece at least
    for rows, v, take in ((1, 1, 1), (4, 151936, 8), (256, 151936, 16), (64, 5000, 128), (1000, 2048, 2)):
        assert size(rows, v, take) >= rows * 8 * (1 + take)


def test_layout_of_states():
    lay = lm._state_layout
    cache = torch.empty(3, 8, 4, 50, 16, dtype=torch.bfloat16)
    out = torch.empty_like(cache)
    assert lay(cache, out, 1) == (3, 1, 4 * 50 * 32, (8 * 6400, 6400, 0), (8 * 6400, 6400, 0))
    used = cache[:, :, :, :20]
    new = torch.empty(3, 8, 4, 20, 16, dtype=torch.bfloat16)
    assert lay(used, used, 1) == (3, 4, 640, (8 * 6400, 6400, 1600), (8 * 6400, 6400, 1600))
    assert lay(used, new, 1) == (3, 4, 640, (8 * 6400, 6400, 1600), (8 * 2560, 2560, 640))
    assert lay(cache[0], out[0], 0)[:3] == (1, 1, 6400)
    every = torch.empty(8, 40)[:, ::2]
    assert lay(every, every, 0) == (1, 20, 4, (0, 160, 8), (0, 160, 8))
    with pytest.raises(ValueError):
        lay(cache[:, :, :, ::2, ::2], cache[:, :, :, ::2, ::2], 1)
    with pytest.raises(ValueError):
        lay(cache[:, :4], cache[:, :4], 2)       # layers, then rows, lie apart
    assert lay(used, used, 3)[:3] == (96, 1, 32)   # all that is before `dim` as one


def test_binding():
    z, s = torch.zeros(8, 50), torch.zeros(8)
    with pytest.raises(ValueError):
        lm.beam_select(z, s, 4)                       # not on a GPU
    with pytest.raises(ValueError):
        lm.beam_select(z, s, 0)
    with pytest.raises(ValueError):
        lm.beam_select(z, s, 4, 0)
    with pytest.raises(ValueError):
        lm.beam_select(z, s, 4, eos_id=2 ** 32 + 2)
    with pytest.raises(ValueError):
        lm.beam_reorder(z, torch.zeros(8, dtype=torch.int32))
