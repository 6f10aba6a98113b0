"""Embedding and adapters through autograd: captured steps, threads, padded batches, operands seen twice."""
import threading

import pytest
import torch

from chunked_lm_head_tcgen05_gb300 import autograd
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def make(seed, N=300, V=520, H=64, rank=8, n=3):
    g = torch.Generator("cuda").manual_seed(seed)

    def rand(*shape, dtype=BF16, size=1.0):
        return (size * torch.randn(shape, generator=g, device="cuda")).to(dtype)

    return dict(ids=torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32),
                of=torch.randint(-1, n, (N,), generator=g, device="cuda", dtype=torch.int32),
                table=rand(V, H), head=rand(H, V, size=H ** -0.5), down=rand(n, rank, H, size=H ** -0.5),
                up=rand(n, rank, V), g=rand(N, V))


def step(s, leaves=None):
    """Embedding, a projection with adapters, and the gradients of all leaves."""
    table, down, up = leaves or [s[k].detach().clone().requires_grad_(True) for k in ("table", "down", "up")]
    x = autograd.embedding(s["ids"], table, scale=2.0, padding_id=0)
    y = autograd.adapters(x @ s["head"], x, down, up, s["of"])
    return (y.detach(), *torch.autograd.grad(y, (table, down, up), s["g"]))


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_captured_step_replayed_with_other_tokens():
    s = make(1)
    leaves = [s[k].detach().clone().requires_grad_(True) for k in ("table", "down", "up")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(s, leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s, leaves)
    for seed in (2, 3):
        other = make(seed)
        for k in ("ids", "of", "g"):
            s[k].copy_(other[k])
        s["ids"][250:] = 0              # a padded batch
        s["of"][250:] = -1
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, step(s))
        assert not out[1][0].any()       # nothing for the padding's row


@pytest.mark.parametrize("own_streams", [True, False])
def test_two_threads_at_once(own_streams):
    states = [make(10 + i, N=200 + 57 * i, rank=8 + 5 * i) for i in range(4)]
    want = [step(s) for s in states]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        stream = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            for _ in range(15):
                got = step(states[i])
                stream.synchronize()
                if not same(got, want[i]):
                    failed.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_one_tensor_in_two_places():
    """x as base of a square projection, one factor's memory as both, and the table's rows as x."""
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(50, 64, generator=g, device="cuda").to(BF16).requires_grad_(True)
    f = (0.1 * torch.randn(2, 4, 64, generator=g, device="cuda")).to(BF16).requires_grad_(True)
    of = torch.randint(0, 2, (50,), generator=g, device="cuda", dtype=torch.int32)
    y = autograd.adapters(x, x, f, f, of)
    d = torch.randn(50, 64, generator=g, device="cuda").to(BF16)
    got = torch.autograd.grad(y, (x, f), d)
    x64, f64 = (t.detach().double().requires_grad_(True) for t in (x, f))
    pick = f64[of.long()]
    u = torch.einsum("th,trh->tr", x64, pick)
    want = torch.autograd.grad(x64 + torch.einsum("tr,trh->th", u, pick), (x64, f64), d.double())
    # bf16 results of two summed gradients, each rounded to bf16 before: three roundings of 2^-8
    for a, b in zip(got, want):
        assert (a.double() - b).norm() <= 3 * 2.0 ** -8 * b.norm()
