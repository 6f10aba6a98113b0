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


# x [8, 64] bf16: 1,024 bytes; down [3, 4, 64]: 1,536; up [3, 4, 100]: 2,400; base and cotangent
# [8, 100] bf16: 1,600; dx [8, 64] fp32: 2,048; d_down 3,072, d_up 4,800
ADAPTERS_FWD = dict(base=at(1), type=1, base_ld=100, x=at(2), x_ld=64, down=at(3), up=at(4), ids=at(5), scale=at(6),
                    T=8, H=64, V=100, rank=4, n=3, out=at(7), out_ld=100, workspace=at(8), bytes=1 << 19, stream=None)
ADAPTERS_BWD = dict(grad=at(1), type=1, ld=100, x=at(2), x_ld=64, down=at(3), up=at(4), ids=at(5), scale=at(6), T=8,
                    H=64, V=100, rank=4, n=3, dx=at(7), dx_ld=64, accumulate_dx=0, d_down=at(8), d_up=at(9),
                    accumulate=0, workspace=at(10), bytes=1 << 19, stream=None)


def test_adapters(lib):  # noqa: F811
    inside = [P(2 * M + 1022), P(3 * M + 512), P(3 * M + 1534), P(4 * M + 2398), P(5 * M + 30), P(6 * M + 10)]
    before = [P(n * M - 1598) for n in (2, 3, 4, 5, 6)]
    refused(lib, "lmhead_adapters_fwd", ADAPTERS_FWD, [dict(out=p) for p in inside + before] + [
        dict(out=P(M + 200)), dict(out=P(M - 200)), dict(out=P(M + 1598)), dict(out=P(M + 2), T=1),
        # rows of one tensor whose columns meet
        dict(base_ld=256, out_ld=256, out=P(M + 198)), dict(base_ld=256, out_ld=256, out=P(M + 314)),
        dict(base_ld=256, out_ld=256, out=P(M - 198)),
        dict(workspace=at(1)), dict(workspace=at(2)), dict(workspace=at(3)), dict(workspace=at(4)),
        dict(workspace=at(5)), dict(workspace=at(6)), dict(workspace=at(7)), dict(base=at(8), out=at(8))])
    results = [P(M + 1596), P(2 * M + 1020), P(3 * M + 4), P(4 * M + 2396), P(5 * M + 28), P(6 * M + 8)]
    refused(lib, "lmhead_adapters_bwd", ADAPTERS_BWD,
            [{name: p} for name in ("dx", "d_down", "d_up") for p in results] + [
        dict(dx=P(8 * M + 3068)), dict(dx=P(9 * M + 4796)), dict(d_up=P(8 * M + 3068)), dict(d_down=P(9 * M - 3068)),
        dict(dx=P(8 * M - 2044)), dict(dx_ld=512, d_down=P(7 * M + 256 - 4)), dict(d_up=None, dx=P(8 * M + 4)),
        dict(dx=at(10)), dict(workspace=at(7)), dict(workspace=at(8)), dict(workspace=at(9)), dict(workspace=at(1))])


# eight rows [8, 100] fp32: 3,200 bytes; scores and lse 32, finished 8; two groups of 4: 32 a result
SELECT = dict(logits=at(1), type=0, ld=100, R=8, V=100, beams=4, take=4, scores=at(2), finished=at(3), eos=2, tau=1.0,
              out=at(4), parents=at(5), tokens=at(6), next=at(7), lse=at(8), workspace=at(9), bytes=1 << 19, stream=None)


def test_selection(lib):  # noqa: F811
    inputs = [P(M + 3196), P(M + 400), P(2 * M + 4), P(3 * M + 4), P(M - 28)]
    refused(lib, "lmhead_beam_select", SELECT,
            [{name: p} for name in ("out", "parents", "tokens", "lse") for p in inputs] + [
        dict(parents=at(2)), dict(tokens=at(2)), dict(lse=at(2)), dict(next=at(2)), dict(next=P(M + 7)),
        dict(lse=at(4)), dict(parents=at(4)), dict(tokens=at(5)), dict(tokens=P(5 * M + 28)), dict(next=P(4 * M + 31)),
        dict(next=P(8 * M + 3)), dict(lse=at(2), out=at(2)), dict(parents=at(2), out=at(2)),
        dict(ld=200, out=P(M + 384)), dict(workspace=at(1)), dict(workspace=at(2)), dict(workspace=at(8)),
        dict(workspace=at(3)), dict(workspace=at(7))])


# two times eight rows of two stretches of 320 bytes
REORDER = dict(src=at(1), so=8 * 640, sr=640, sm=320, src_rows=8, dst=at(2), do=8 * 640, dr=640, dm=320, parents=at(3),
               rows=8, beams=4, outer=2, mid=2, inner=320, clear=0, stream=None)


def test_reorder(lib):  # noqa: F811
    cases = [dict(parents=at(2)), dict(parents=P(2 * M - 28)), dict(parents=P(2 * M + 16 * 640 - 4)),
             dict(parents=P(2 * M + 5000))]
    refused(lib, "lmhead_beam_reorder", REORDER, cases)
    refused(lib, "lmhead_beam_reorder", dict(REORDER, src=at(2)), cases)     # in place
