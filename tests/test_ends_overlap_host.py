"""Results of embedding, adapters and beam search that share memory with what the calls read, or with
one another, are refused (CPU only: decided before anything is launched)."""
import pytest

from test_operators_host import INVALID, P, call, lib  # noqa: F401
import chunked_lm_head_tcgen05_gb300 as lm

M = 1 << 20


def at(n):
    return P(M * n)


def refused(lib, name, defaults, cases):  # noqa: F811
    fn = getattr(lib, name)
    assert len(defaults) == len(lm._SIGNATURES[name][1])
    for over in cases:
        assert call(fn, defaults, **over) == INVALID, (name, over)


# table [100, 64] bf16: 12,800 bytes; eight rows of a result of 64 bf16: 1,024 bytes
EMBED_FWD = dict(ids=at(1), N=8, weight=at(2), type=1, w_ld=64, V=100, H=64, scale=1.0, y=at(3), y_type=1, y_ld=64,
                 stream=None)
EMBED_BWD = dict(dy=at(1), dy_type=1, dy_ld=64, ids=at(2), N=8, V=100, H=64, scale=1.0, padding=lm.NO_PADDING,
                 d_weight=at(3), d_type=0, accumulate=0, workspace=at(4), bytes=1 << 18, stream=None)


def test_embedding(lib):  # noqa: F811
    refused(lib, "lmhead_embedding_fwd", EMBED_FWD, [
        dict(y=at(2)), dict(y=P(2 * M + 128)), dict(y=P(2 * M + 12800 - 2)), dict(y=P(2 * M - 1024 + 2)),
        dict(y=P(2 * M + 128), N=1), dict(y=at(1)), dict(y=P(M + 28)), dict(ids=P(3 * M + 512)),
        # rows of one tensor whose columns meet
        dict(w_ld=128, y=P(2 * M + 64), y_ld=128), dict(w_ld=128, y=P(2 * M + 254), y_ld=128),
        dict(w_ld=128, y=P(2 * M - 2), y_ld=128), dict(w_ld=128, y=P(2 * M + 64), y_ld=256),
        dict(w_ld=1 << 60, y=P(2 * M + 64)), dict(w_ld=(1 << 63) - 1, y=P(2 * M + 64)),
        # a table of one row
        dict(V=1, y=P(2 * M - 900)), dict(V=1, w_ld=99, y=P(2 * M - 1022))])
    refused(lib, "lmhead_embedding_bwd", EMBED_BWD, [
        dict(d_weight=at(1)), dict(dy=P(3 * M + 256)), dict(dy=P(3 * M + 25600 - 2)), dict(d_weight=P(2 * M + 28)),
        dict(workspace=at(1)), dict(workspace=at(2)), dict(workspace=P(3 * M + 25600 - 256 * 4)),
        dict(d_type=1, d_weight=P(M + 1022))])
