"""Beam selection and reordering of states against plain 64-bit and indexing implementations."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built
from operators_reference import U32, f64
from test_gpu_guard_canaries import Guarded, _check

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# lse: the sum of exponentials is off by the exponential's 2^-22, three roundings of its
# argument (whose mean under the softmax is at most log V < 21) and some 50 additions, so
# by (4 + 3 * 21 + 50) 2^-24 < 1e-5 relative; a score adds its own rounding.
TOL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def log_probs(z):
    """log softmax(z), which a maximum of -3e38 must not swallow, and lse."""
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        part = np.log(np.exp(z - m).sum(1, keepdims=True))
        lse = (m + part)[:, 0]
        lse[np.isnan(z).any(1) | np.isposinf(z).any(1)] = np.nan
        return (z - m) - part, lse


def candidates(logits, scores, beams, tau, finished, eos):
    """[G, beams V] scores, -inf where there is no candidate, and lse [R]."""
    z = f64(logits) / np.float64(np.float32(tau))
    (logp, lse), s = log_probs(z), f64(scores)
    ended = np.zeros(len(s), bool) if finished is None else finished.cpu().numpy() != 0
    with np.errstate(invalid="ignore"):
        total = s[:, None] + logp
    total[~np.isfinite(s) | ~np.isfinite(lse)] = -np.inf
    total[ended] = -np.inf
    total[ended, eos] = np.where(np.isfinite(s), s, -np.inf)[ended]
    lse[ended] = 0.0
    return total.reshape(len(s) // beams, -1), lse


def check(logits, scores, beams, take, tau=1.0, finished=None, eos=-1, exactly=False, **more):
    R, V = logits.shape
    nxt = torch.full((R // beams, take), 7, dtype=torch.uint8, device="cuda")
    got = lm.beam_select(logits, scores, beams, take, tau, finished, eos, nxt, **more)
    out, parents, tokens, lse = (t.cpu().numpy() for t in got)
    want, want_lse = candidates(logits, scores, beams, tau, finished, eos)
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse))
    with np.errstate(over="ignore"):      # a row of the lowest value over tau < 1: past fp32
        want_lse = np.where(np.isinf(want_lse.astype(np.float32)), want_lse.astype(np.float32), want_lse)
    fine = np.isfinite(want_lse)
    assert np.array_equal(lse[~fine & ~np.isnan(lse)], want_lse[~fine & ~np.isnan(lse)])
    assert (np.abs(lse[fine] - want_lse[fine]) <= TOL + 2 * U32 * np.abs(want_lse[fine])).all()
    ended = np.zeros(R, bool) if finished is None else finished.cpu().numpy() != 0
    for g in range(R // beams):
        order = np.argsort(-want[g], kind="stable")[:take]
        n = int((want[g][order] > -np.inf).sum())
        assert (out[g, n:] == -np.inf).all() and (parents[g, n:] == -1).all()
        assert (tokens[g, n:] == -1).all() and not nxt[g, n:].any()
        at = (parents[g, :n].astype(np.int64) - g * beams) * V + tokens[g, :n]
        assert len(set(at.tolist())) == n and (at >= 0).all() and (at < beams * V).all()
        best, mine = want[g][order[:n]], want[g][at]
        size = TOL + 2 * U32 * np.abs(best)
        assert (np.abs(mine - best) <= size).all()
        assert (np.abs(out[g, :n] - best) <= size).all()
        if exactly:
            assert at.tolist() == order[:n].tolist()
        elif n:
            # where neighbours are further apart than the tolerance the choice is theirs
            full = np.append(np.sort(want[g])[::-1], -np.inf)[:n + 1]
            gap = np.append(np.inf, full[:-1] - full[1:])       # before and behind each
            far = (gap[:-1] > 2 * size) & (gap[1:] > 2 * size)
            assert np.array_equal(at[far], order[:n][far])
        stop = ended[parents[g, :n]] | (tokens[g, :n] == eos)
        assert np.array_equal(nxt[g, :n].cpu().numpy() != 0, stop)
    return got


def logits_of(R, V, dtype, gen, pad=0, skip=0, spread=3.0):
    t = torch.zeros(skip + R * (V + pad), dtype=dtype, device="cuda")[skip:].view(R, V + pad)[:, :V]
    t.copy_(spread * torch.randn(R, V, generator=gen, device="cuda"))
    return t


SIZES = [(1, 1, 1, 1), (1, 1, 5, 8), (3, 2, 7, 4), (1, 4, 1000, 8), (2, 3, 1111, 6), (5, 4, 2048, 9),
         (1, 1, 50257, 1), (1, 16, 30011, 32), (2, 64, 4099, 128), (40, 8, 8193, 16), (300, 1, 333, 2),
         (1, 5, 151936, 10)]


@pytest.mark.parametrize("G,K,V,N", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_select(G, K, V, N, dtype):
    gen = torch.Generator("cuda").manual_seed(G * 31 + V)
    for pad, skip, tau in ((0, 0, 1.0), (5, 3, 0.7), (8, 1, 1.9)):
        z = logits_of(G * K, V, dtype, gen, pad, skip)
        s = -8 * torch.rand(G * K, generator=gen, device="cuda")
        check(z, s, K, N, tau)


@pytest.mark.parametrize("V", [9, 3000, 40000])
def test_select_with_masks_and_ended_beams(V):
    gen = torch.Generator("cuda").manual_seed(V)
    G, K, N = 12, 4, 8
    z = logits_of(G * K, V, F32, gen)
    keep = torch.rand(G * K, V, generator=gen, device="cuda") < 0.01
    keep[:4] = False                      # a group whose masks leave nothing
    keep[4:7] = False                     # one beam of the next has its tokens left
    keep[8, :] = False
    keep[8, V // 2] = True                # a single token
    z = z.masked_fill(~keep, -float("inf"))
    z[12] = torch.finfo(F32).min          # a mask of the lowest value, everywhere
    z[13, 1:] = torch.finfo(F32).min
    s = -4 * torch.rand(G * K, generator=gen, device="cuda")
    s[17:20] = -float("inf")              # beams that do not exist yet
    s[21] = float("nan")
    s[22] = float("inf")
    f = (torch.rand(G * K, generator=gen, device="cuda") < 0.3).to(torch.uint8)
    f[:4] = 0
    f[24:28] = 1                          # a whole group has ended
    f[18] = 1                             # ended without ever existing
    z[24:28] = float("nan")               # not looked at
    check(z, s, K, N, 0.8, f, 2)
    z[30, 5] = float("nan")
    z[33, V - 1] = float("inf")
    check(z, s, K, N, 1.0, f, 2)
    check(z, s, K, N)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("R,K,V,N", [(4, 4, 20000, 8), (64, 8, 20000, 128), (1, 1, 1030, 5), (32, 16, 9000, 7)])
def test_select_among_equals(dtype, R, K, V, N):
    """Equal logits: the lowest ids, the lowest beam first; more of them than are ranked at once."""
    s = torch.zeros(R, device="cuda")
    z = torch.full((R, V), 0.5, dtype=dtype, device="cuda")
    check(z, s, K, N, exactly=True)
    z[:, V // 3:] = 2.0                               # the equals begin inside a row
    check(z, s, K, N, exactly=True)
    z[:, V - 2:] = 3.0                                # and a few are above them
    check(z, s, K, N, exactly=True)
    z[:] = -float("inf")
    z[:, 100:] = -0.0
    z[:, 101::2] = 0.0                                # one zero
    check(z, s, K, N, exactly=True)


@pytest.mark.parametrize("R,V,N", [(2, 40000, 100), (400, 9000, 8), (200, 40000, 3)])
def test_select_of_ascending_and_descending_logits(R, V, N):
    """Every tile's elements are above what was found before, or none is."""
    ramp = torch.arange(V, device="cuda", dtype=torch.float32) / 1000
    z = torch.stack([ramp, ramp.flip(0)]).repeat(R // 2, 1)
    z[:, V // 2] = torch.where(torch.arange(R, device="cuda") % 4 == 0, float("nan"), z[:, V // 2])
    s = -torch.rand(R, device="cuda")
    check(z, s, 2, N)
    check((z * 16).floor() / 16, s, 1, N)      # steps of equal logits


def test_select_with_extreme_logits_and_temperatures():
    gen = torch.Generator("cuda").manual_seed(2)
    z = logits_of(8, 5000, F32, gen)
    z[0] *= 1e30
    z[1, 7] = 3e38
    z[2, 7] = -3e38
    s = torch.zeros(8, device="cuda")
    check(z[3:], s[3:], 5, 5, 1e-3)
    check(z[3:], s[3:], 1, 5, 1e4)
    check(z[:3], s[:3], 1, 4, 1.0)
    lm.beam_select(z, s, 4, 4, 1e-40)                 # a subnormal temperature: no fault, any order
    torch.cuda.synchronize()


def test_select_of_identical_beams():
    """What a first step gives without marking the other beams: every token K times."""
    gen = torch.Generator("cuda").manual_seed(4)
    z = logits_of(2, 9000, BF16, gen).repeat_interleave(8, 0).contiguous()
    check(z, torch.zeros(16, device="cuda"), 8, 16, exactly=True)


def test_select_is_the_same_every_time_on_any_stream_and_in_graphs():
    gen = torch.Generator("cuda").manual_seed(6)
    z = logits_of(32, 30000, BF16, gen)
    s = -torch.rand(32, generator=gen, device="cuda")
    want = lm.beam_select(z, s, 4, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        got = lm.beam_select(z, s, 4, 8, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = lm.beam_select(z, s, 4, 8)
        graphs.append((graph, out))
    z.copy_(logits_of(32, 30000, BF16, gen))
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = lm.beam_select(z, s, 4, 8)
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("R,K,V,N", [(1, 1, 1, 1), (6, 3, 1111, 7), (64, 8, 20001, 16), (8, 8, 8192, 100)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_writes_stay_inside(R, K, V, N, dtype):
    gin = dict(z=Guarded((R, V), dtype, 71, torch.randn(R, V)),
               s=Guarded((R,), F32, 72, -torch.rand(R)),
               f=Guarded((R,), torch.uint8, 73, (torch.rand(R) < 0.2).to(torch.uint8)))
    shape = (R // K, N)
    out = dict(s=Guarded(shape, F32, 74), p=Guarded(shape, torch.int32, 75),
               t=Guarded(shape, torch.int32, 76), n=Guarded(shape, torch.uint8, 77),
               lse=Guarded((R,), F32, 78),
               ws=Guarded((lm.lmhead_beam_workspace_size(R, V, N),), torch.uint8, 79))
    assert lm.lmhead_beam_select(gin["z"].t, K, N, gin["s"].t, gin["f"].t, 0, 1.0, out["s"].t,
                                 out["p"].t, out["t"].t, out["n"].t, out["lse"].t, out["ws"].t) == 0
    _check(gin, out, "select")


def test_select_into_its_own_inputs():
    """A loop that keeps its scores and flags in one place."""
    gen = torch.Generator("cuda").manual_seed(21)
    z = logits_of(512, 3000, F32, gen)
    s = -torch.rand(512, generator=gen, device="cuda")
    f = (torch.rand(512, generator=gen, device="cuda") < 0.3).to(torch.uint8)
    nxt = torch.empty(128, 4, dtype=torch.uint8, device="cuda")
    want = lm.beam_select(z, s, 4, 4, 1.0, f, 5, nxt)
    ws = torch.empty(lm.lmhead_beam_workspace_size(512, 3000, 4), dtype=torch.uint8, device="cuda")
    p, t = torch.empty_like(want[1]), torch.empty_like(want[2])
    assert lm.lmhead_beam_select(z, 4, 4, s, f, 5, 1.0, s.view(128, 4), p, t, f.view(128, 4), None, ws) == 0
    assert torch.equal(s.view(128, 4), want[0]) and torch.equal(p, want[1]) and torch.equal(t, want[2])
    assert torch.equal(f.view(128, 4), nxt)


def test_select_past_32_bits():
    z = torch.zeros(17000, 151936, dtype=BF16, device="cuda")      # 2.58e9 elements
    z[-1, -1] = 5.0
    z[0, 1] = 4.0
    got = lm.beam_select(z, torch.zeros(17000, device="cuda"), 8, 1)
    assert got[1][-1, 0] == 16999 and got[2][-1, 0] == 151935
    assert got[1][0, 0] == 0 and got[2][0, 0] == 1


# ------------------------------------------------------------------ reordering
def some_parents(rows, beams, gen, none=0.0):
    p = torch.randint(0, beams, (rows,), generator=gen, device="cuda")
    p = p + torch.arange(rows, device="cuda") // beams * beams
    return torch.where(torch.rand(rows, generator=gen, device="cuda") < none, -1, p).to(torch.int32)


STATES = [((4, 30), 0), ((8, 5, 7), 0), ((3, 8, 2, 50, 16), 1), ((2, 12, 1000), 1), ((6, 4, 1), 1),
          ((1, 128, 3), 1), ((5, 64, 4, 9, 33), 1), ((2, 3, 4, 8, 10), 3), ((12,), 0), ((2, 8, 70001), 1)]


@pytest.mark.parametrize("shape,dim", STATES)
@pytest.mark.parametrize("dtype", [F32, BF16, torch.int64, torch.uint8, torch.complex128])
def test_reorder(shape, dim, dtype):
    gen = torch.Generator("cuda").manual_seed(sum(shape))
    full = (100 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)
    rows = shape[dim]
    for beams in {1, rows, next(b for b in (4, 3, 2, 1) if rows % b == 0)} & set(range(1, 65)):
        parents = some_parents(rows, beams, gen)
        want = full.index_select(dim, parents.long())
        assert torch.equal(lm.beam_reorder(full, parents, dim), want)
        mine = full.clone()
        assert lm.beam_reorder(mine, parents, dim - full.dim(), mine, beams) is mine
        assert torch.equal(mine, want)
    # any rows, more or fewer than there are, some without a parent
    parents = torch.randint(-2, rows + 2, (2 * rows + 1,), generator=gen, device="cuda").to(torch.int32)
    there = (parents >= 0) & (parents < rows)
    want = full.index_select(dim, parents.long().clamp(0, rows - 1))
    view = [1] * full.dim()
    view[dim] = -1
    want = torch.where(there.view(view), want, torch.zeros_like(want))
    assert torch.equal(lm.beam_reorder(full, parents, dim), want)
    out = torch.ones_like(want)
    lm.beam_reorder(full, parents, dim, out)
    assert torch.equal(out, torch.where(there.view(view), want, torch.ones_like(want)))


@pytest.mark.parametrize("beams", [2, 4, 7, 8, 16, 17, 32, 64])
def test_reorder_in_place_takes_every_row_before_it_is_overwritten(beams):
    """Cycles, chains and rows that stay, at alignments of 16 bytes down to one."""
    gen = torch.Generator("cuda").manual_seed(beams)
    rows = 3 * beams
    for width, skip in ((64, 0), (62, 0), (63, 0), (61, 1), (1, 3)):
        base = torch.randint(0, 255, (skip + 2 * rows * 5 * width,), generator=gen,
                             device="cuda").to(torch.uint8)
        at = torch.arange(rows, device="cuda")
        turn = (at // beams * beams + (at + 1) % beams).to(torch.int32)
        for parents in (turn, some_parents(rows, beams, gen), some_parents(rows, beams, gen, 0.4)):
            mem = base.clone()
            state = mem[skip:].view(2, rows, 5, width)
            keep = torch.where(parents < 0, at, parents.long())
            ok = keep // beams == at // beams
            want = state.index_select(1, torch.where(ok, keep, at))
            lm.beam_reorder(state, parents, 1, state, beams)
            assert torch.equal(state, want) and torch.equal(mem[:skip], base[:skip])
    # parents of another group are no parents in place
    state = torch.arange(rows, device="cuda", dtype=torch.int32)
    parents = ((at + beams) % rows).to(torch.int32)
    lm.beam_reorder(state, parents, 0, state, beams)
    assert torch.equal(state, at.to(torch.int32))


def test_reorder_of_the_used_part_leaves_the_rest():
    gen = torch.Generator("cuda").manual_seed(77)
    for dtype, dim, used in ((BF16, 64, 37), (F16, 33, 5), (torch.uint8, 33, 63)):
        cache = (50 * torch.randn(2, 8, 4, 64, dim, generator=gen, device="cuda")).to(dtype)
        before = cache.clone()
        parents = some_parents(8, 4, gen)
        view = cache[:, :, :, :used]
        lm.beam_reorder(view, parents, 1, view, 4)
        assert torch.equal(cache[:, :, :, :used], before[:, :, :, :used].index_select(1, parents.long()))
        assert torch.equal(cache[:, :, :, used:], before[:, :, :, used:])
        moved = torch.zeros_like(before)
        lm.beam_reorder(before[:, :, :, :used], parents, 1, moved[:, :, :, :used])
        assert torch.equal(moved[:, :, :, :used], cache[:, :, :, :used]) and not moved[:, :, :, used:].any()


def test_reorder_refuses_what_overlaps():
    state = torch.zeros(9, 16, device="cuda")
    parents = torch.zeros(8, dtype=torch.int32, device="cuda")
    for out in (state[1:], state[:8].view(-1).as_strided((8, 16), (8, 1)),
                torch.zeros(16, device="cuda").expand(8, 16)):
        with pytest.raises(lm.LmheadError):
            lm.beam_reorder(state[:8], parents, 0, out, 4)
    with pytest.raises(lm.LmheadError):
        lm.beam_reorder(state[:8], parents, 0, state[:8])          # in place without groups
    with pytest.raises(lm.LmheadError):
        lm.beam_reorder(state[:8], parents, 0, state[:8], 3)
    with pytest.raises(TypeError):
        lm.beam_reorder(state[:8], parents, 0, torch.zeros(8, 16, device="cuda", dtype=BF16))
    with pytest.raises(TypeError):
        lm.beam_reorder(state[:8], parents.long(), 0)
    shared = torch.randn(1, 16, device="cuda").expand(8, 16)       # a source may repeat itself
    assert torch.equal(lm.beam_reorder(shared, parents, 0), shared)


def test_reorder_past_32_bits():
    state = torch.zeros(3, 1_000_000_007, dtype=torch.uint8, device="cuda")
    state[2, -1] = 9
    parents = torch.tensor([2, 1, 0], dtype=torch.int32, device="cuda")
    lm.beam_reorder(state, parents, 0, state, 3)
    assert state[0, -1] == 9 and state[2, -1] == 0
    assert lm.beam_reorder(state, parents)[2, -1] == 9


def test_reorder_streams_and_graphs():
    gen = torch.Generator("cuda").manual_seed(5)
    state = torch.randn(2, 8, 500, generator=gen, device="cuda")
    parents = some_parents(8, 4, gen)
    want = state.index_select(1, parents.long())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lm.beam_reorder(state, parents, 1, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lm.beam_reorder(state, parents, 1)
        lm.beam_reorder(state, parents, 1, state, 4)
    parents.copy_(some_parents(8, 4, gen))
    want = state.index_select(1, parents.long())
    graph.replay()
    assert torch.equal(out, want) and torch.equal(state, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_where_tiles_differ(dtype):
    """Tiles of a long piece that add nothing, a few, some that are ranked again and more than fit, in
    turn: what one tile adds is counted before every thread has read the tile before."""
    R, V, take = 608, 60000, 5
    gen = torch.Generator("cuda").manual_seed(77)
    z = logits_of(R, V, dtype, gen, 4)
    step = torch.arange(V, device="cuda")
    for r, (width, every) in enumerate(((8192, 2), (8192, 3), (4096, 2), (2048, 5))):
        rise = (step // width + r) % every == 0          # ascending over these, and none elsewhere
        z[r::4] = torch.where(rise, step / 512.0, z[r::4].float()).to(dtype)
    s = -8 * torch.rand(R, generator=gen, device="cuda")
    first = check(z, s, 4, take)
    for _ in range(40):
        for a, b in zip(lm.beam_select(z, s, 4, take), first):
            assert torch.equal(a, b)
