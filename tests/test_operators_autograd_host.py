"""What the autograd functions of layer norm, distillation and logit processing keep between
forward and backward, with stand-ins for the library's calls (no GPU)."""
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
