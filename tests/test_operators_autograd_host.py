"""What the autograd functions of layer norm, distillation and logit processing keep between
forward and backward, with stand-ins for the library's calls (no GPU)."""
import contextlib
import threading
from types import SimpleNamespace

import pytest
import torch

from chunked_lm_head_tcgen05_gb300 import autograd

R, V = 3, 40


@pytest.fixture
def processing(monkeypatch):
    """Logit processing by stand-ins whose gradient depends on every rule."""
    def forward(logits, out=None, stream=None, **rules):
        return logits * 2.0 if out is None else out.copy_(logits * 2.0)

    def backward(g, logits, tokens=None, spans=None, repetition=None, allowed=None,
                 allowed_rows=None):
        scale = sum(float(t.double().sum()) for t in (tokens, spans, repetition, allowed,
                                                      allowed_rows) if t is not None)
        return g * scale

    monkeypatch.setattr(autograd, "_process_logits", forward)
    monkeypatch.setattr(autograd, "process_logits_backward", backward)
    return dict(tokens=torch.arange(9, dtype=torch.int32),
                spans=torch.tensor([[0, 1, 3], [3, 4, 6], [6, 7, 9]]),
                repetition=torch.full((R,), 1.5),
                allowed=torch.ones(R, 2, dtype=torch.int32),
                allowed_rows=torch.arange(R, dtype=torch.int32))


def test_rules_reach_the_backward(processing):
    z = torch.randn(R, V, requires_grad=True)
    some = {k: processing[k] for k in ("tokens", "spans")}
    for rules in (processing, some, {}):
        g, = torch.autograd.grad(autograd.process_logits(z, **rules), z, torch.ones(R, V))
        assert (g == sum(float(t.double().sum()) for t in rules.values())).all()


@pytest.mark.parametrize("name", ["tokens", "spans", "repetition", "allowed", "allowed_rows"])
def test_rules_changed_before_the_backward_are_noticed(processing, name):
    """A sampler that reuses one of these buffers must not get the gradient of other rules."""
    z = torch.randn(R, V, requires_grad=True)
    out = autograd.process_logits(z, **processing)
    processing[name].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out, z, torch.ones(R, V))


def test_rules_pass_through_saved_tensor_hooks(processing):
    seen = []
    z = torch.randn(R, V, requires_grad=True)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(t.shape) or t, lambda t: t):
        autograd.process_logits(z, **processing)
    assert len(seen) == 1 + len(processing)


@pytest.mark.parametrize("name", ["out", "stream"])
def test_processing_refuses_what_it_has_no_form_for(processing, name):
    """An output of the caller's could be the logits, which the backward reads."""
    z = torch.randn(R, V, requires_grad=True)
    with pytest.raises(TypeError, match=name):
        autograd.process_logits(z, **processing, **{name: z.detach() if name == "out" else 0})
    with pytest.raises(TypeError, match="no_such_rule"):
        autograd.process_logits(z, no_such_rule=None)


class Meeting:
    """A stand-in for a library call that several threads are in at once; notes the workspaces."""

    def __init__(self, threads):
        self.barrier = threading.Barrier(threads, timeout=20)
        self.workspaces = []

    def __call__(self, workspace):
        self.workspaces.append(workspace)
        self.barrier.wait()


@pytest.fixture
def cached(monkeypatch):
    """The workspace cache without a GPU: every call is on one stream, capturing as told."""
    state = SimpleNamespace(capturing=False)
    monkeypatch.setattr(autograd, "_stream_handle", lambda device: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    monkeypatch.setattr(autograd, "lmhead_layernorm_workspace_size", lambda n, h: 64 * n)
    monkeypatch.setattr(autograd, "layernorm_forward",
                        lambda x, w, b, eps, kind: (x * w, x.mean(1), x.mean(1)))
    autograd.release_workspaces()
    yield state
    autograd.release_workspaces()


def norm_backward(monkeypatch, call, rows=4):
    def backward(dy, x, w, mean, rstd, with_bias=True, workspace=None):
        call(workspace)
        return dy, torch.zeros_like(w), None
    monkeypatch.setattr(autograd, "layernorm_backward", backward)
    x, w = torch.randn(rows, 8, requires_grad=True), torch.ones(8)
    return lambda: autograd.layer_norm(x, w).backward(torch.ones(rows, 8))


def test_threads_in_one_streams_calls_do_not_share_a_workspace(cached, monkeypatch):
    """A call is several launches that pass data through its workspace, and another thread's may
    come between them on the same stream."""
    meeting = Meeting(2)
    step = norm_backward(monkeypatch, meeting)
    step_too = norm_backward(monkeypatch, meeting)
    threads = [threading.Thread(target=f) for f in (step, step_too)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(meeting.workspaces) == 2
    assert len({w.data_ptr() for w in meeting.workspaces}) == 2
    assert len(autograd._workspaces) == 1          # and one of them stays


def test_workspace_stays_between_calls_and_grows(cached, monkeypatch):
    seen = []
    for rows in (4, 4, 2, 9, 4):
        norm_backward(monkeypatch, lambda w: seen.append((w.data_ptr(), w.numel())), rows)()
    assert [n for _, n in seen] == [256, 256, 256, 576, 576]
    assert seen[0] == seen[1] == seen[2] and seen[3] == seen[4]


def test_a_captured_call_has_a_workspace_of_its_own(cached, monkeypatch):
    """A graph replays into the address it was captured with, so that memory belongs to the graph's
    pool and not to a cache that may drop it."""
    seen = []
    step = norm_backward(monkeypatch, seen.append)
    step()
    before = {k: v.data_ptr() for k, v in autograd._workspaces.items()}
    cached.capturing = True
    step()
    cached.capturing = False
    assert seen[1].data_ptr() != seen[0].data_ptr()
    assert {k: v.data_ptr() for k, v in autograd._workspaces.items()} == before


def test_a_refused_call_does_not_lose_the_workspace(cached, monkeypatch):
    seen = []

    def refuse(w):
        seen.append(w.data_ptr())
        raise ValueError("refused")
    for _ in range(2):
        with pytest.raises(ValueError, match="refused"):
            norm_backward(monkeypatch, refuse)()
    assert seen[0] == seen[1]


def first_gradients(monkeypatch):
    """(name, loss, leaf) of the four functions, by stand-ins."""
    @contextlib.contextmanager
    def no_workspace(n, device):
        yield None
    zero = torch.zeros(4)
    monkeypatch.setattr(autograd, "_stream_workspace", no_workspace)
    monkeypatch.setattr(autograd, "lmhead_layernorm_workspace_size", lambda n, h: 1)
    monkeypatch.setattr(autograd, "layernorm_forward", lambda x, w, b, eps, kind: (x * x, zero, zero))
    monkeypatch.setattr(autograd, "layernorm_backward",
                        lambda dy, x, w, *a, **k: (2 * dy * x, torch.zeros_like(w), None))
    monkeypatch.setattr(autograd, "distill_logits_forward", lambda z, *a: ((z * z).sum(1), zero))
    monkeypatch.setattr(autograd, "distill_logits_backward",
                        lambda z, ids, top, mask, t, tt, g, *a: 2 * z * g[:, None])
    monkeypatch.setattr(autograd, "lmhead_distill_workspace_size", lambda *a: 1)
    monkeypatch.setattr(autograd, "lmhead_distill_narrow_dweight", lambda *a: False)
    monkeypatch.setattr(autograd, "lmhead_distill_fwd", lambda *a: 0)
    monkeypatch.setattr(autograd, "lmhead_distill_bwd", lambda *a: 0)
    monkeypatch.setattr(autograd, "_process_logits", lambda z: z * z)
    monkeypatch.setattr(autograd, "process_logits_backward", lambda g, z, **rules: 2 * g * z)
    x = torch.randn(4, 8, requires_grad=True)
    ids, top = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    yield "layer_norm", autograd.layer_norm(x, torch.ones(8)), x
    yield "distill_logits", autograd.distill_logits(x, ids, top), x
    yield "lmhead_distill", autograd.lmhead_distill(x, torch.ones(5, 8), ids, top), x
    yield "process_logits", autograd.process_logits(x), x


def test_a_second_derivative_is_refused(monkeypatch):
    """The backward's calls are no graph of torch's: a term that needs their derivative must raise,
    not drop out of a sum in which another path carries one."""
    for name, out, x in first_gradients(monkeypatch):
        plain, = torch.autograd.grad(out.sum(), x, retain_graph=True)
        assert not plain.requires_grad
        d, = torch.autograd.grad(out.sum(), x, create_graph=True)
        if name != "lmhead_distill":           # (its stand-in writes nothing)
            assert torch.equal(d.detach(), plain), name
        (x ** 3).sum().backward()              # other paths are not concerned
        for second in (lambda p: torch.autograd.grad(p, x, retain_graph=True), torch.Tensor.backward):
            with pytest.raises(RuntimeError, match="differentiable once"):
                second(d.sum() + (x ** 3).sum())
