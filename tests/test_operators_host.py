"""Refusals of the layer norm, distillation and logit processing calls (CPU
only: every refusal is decided on the host before anything is launched)."""
import ctypes

import pytest

import chunked_lm_head_tcgen05_gb300 as lm

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    lm.build()
    return lm.library()


def P(n=1 << 20):
    return ctypes.c_void_p(n)


def call(fn, defaults, **over):
    unknown = set(over) - set(defaults)
    assert not unknown
    return fn(*{**defaults, **over}.values())


NORM_FWD = dict(x=P(), x_type=1, x_ld=64, weight=P(), bias=P(), param_type=1, N=8, H=64, eps=1e-5,
                y=P(), y_type=1, y_ld=64, mean=P(), rstd=P(), stream=None)
NORM_BWD = dict(dy=P(), dy_type=0, dy_ld=64, x=P(), x_type=1, x_ld=64, weight=P(), param_type=0,
                mean=P(), rstd=P(), N=8, H=64, dx=P(), dx_ld=64, d_weight=P(), d_bias=P(),
                accumulate=0, workspace=P(), bytes=1 << 30, stream=None)
LOGITS_FWD = dict(logits=P(), type=0, ld=100, ids=P(), top=P(), teacher_lse=None, mask=None, T=8,
                  V=100, K=4, tau=1.0, teacher_tau=1.0, loss=P(), lse=P(), stream=None)
LOGITS_BWD = dict(logits=P(), type=0, ld=100, ids=P(), top=P(), teacher_lse=None, mask=None, T=8,
                  V=100, K=4, tau=1.0, teacher_tau=1.0, grad=P(), lse=P(), d=P(), d_ld=100,
                  stream=None)
HEAD_FWD = dict(hidden=P(), weight=P(), ids=P(), top=P(), teacher_lse=None, mask=None, T=8, H=64,
                V=100, K=4, tau=1.0, teacher_tau=1.0, chunk=4, loss=P(), lse=P(), z_top=P(),
                workspace=P(), bytes=1 << 30, stream=None)
HEAD_BWD = dict(hidden=P(), weight=P(), ids=P(), top=P(), teacher_lse=None, mask=None, T=8, H=64,
                V=100, K=4, tau=1.0, teacher_tau=1.0, chunk=4, grad=P(), lse=P(), z_top=P(),
                d_hidden=P(), d_weight=P(), d_weight_type=0, accumulate=0, workspace=P(),
                bytes=1 << 30, stream=None)
PROCESS_FWD = dict(logits=P(), type=0, ld=100, R=8, V=100, tokens=P(), n_tokens=50, spans=P(),
                   repetition=P(), frequency=P(), presence=P(), offsets=P(), ids=P(), values=P(),
                   n_bias=3, allowed=P(), n_allowed=8, allowed_rows=None, out=P(), out_ld=100,
                   stream=None)
PROCESS_BWD = dict(grad=P(), grad_ld=100, logits=P(), type=0, ld=100, R=8, V=100, tokens=P(),
                   n_tokens=50, spans=P(), repetition=P(), allowed=P(), n_allowed=8,
                   allowed_rows=None, d=P(), d_ld=100, stream=None)

CASES = [
    ("lmhead_layernorm_fwd", NORM_FWD, [
        (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
        (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(x_ld=63), INVALID),
        (dict(y_ld=63), INVALID), (dict(x_type=3), INVALID), (dict(y_type=-1), INVALID),
        (dict(param_type=9), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
        (dict(N=(1 << 31) - 256), UNSUPPORTED), (dict(param_type=2), UNSUPPORTED),
        (dict(H=(1 << 20) + 1, x_ld=1 << 21, y_ld=1 << 21), UNSUPPORTED),
        (dict(y_type=0), UNSUPPORTED), (dict(x_type=2, y_type=1, param_type=0), UNSUPPORTED),
        (dict(x=P((1 << 20) + 1)), UNSUPPORTED), (dict(bias=P((1 << 20) + 1)), UNSUPPORTED),
        (dict(N=0, x=None, y=None), OK)]),
    ("lmhead_layernorm_bwd", NORM_BWD, [
        (dict(dy=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
        (dict(dx=None, d_weight=None, d_bias=None), INVALID), (dict(workspace=None), INVALID),
        (dict(dx_ld=10), INVALID), (dict(dy_ld=10), INVALID),
        (dict(dy_type=2), UNSUPPORTED), (dict(workspace=P((1 << 20) + 8)), UNSUPPORTED),
        (dict(dx=P((1 << 20) + 1)), UNSUPPORTED), (dict(bytes=16), SMALL),
        (dict(N=0, d_weight=None, d_bias=None), OK)]),
    ("lmhead_distill_logits_fwd", LOGITS_FWD, [
        (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(top=None), INVALID),
        (dict(loss=None), INVALID), (dict(lse=None), INVALID), (dict(T=-1), INVALID),
        (dict(V=0), INVALID), (dict(K=0), INVALID), (dict(ld=99), INVALID), (dict(type=3), INVALID),
        (dict(tau=0.0), INVALID), (dict(tau=float("inf")), INVALID),
        (dict(teacher_tau=-1.0), INVALID), (dict(teacher_tau=float("nan")), INVALID),
        (dict(K=1025), UNSUPPORTED), (dict(T=(1 << 31) - 256), UNSUPPORTED),
        (dict(logits=P((1 << 20) + 2)), UNSUPPORTED), (dict(T=0, logits=None, ids=None), OK)]),
    ("lmhead_distill_logits_bwd", LOGITS_BWD, [
        (dict(grad=None), INVALID), (dict(lse=None), INVALID), (dict(d=None), INVALID),
        (dict(d_ld=99), INVALID), (dict(K=1025), UNSUPPORTED),
        (dict(d=P((1 << 20) + 1)), UNSUPPORTED), (dict(T=0), OK)]),
    ("lmhead_distill_fwd", HEAD_FWD, [
        (dict(hidden=None), INVALID), (dict(ids=None), INVALID), (dict(z_top=None), INVALID),
        (dict(workspace=None), INVALID), (dict(K=0), INVALID), (dict(tau=-1.0), INVALID),
        (dict(teacher_tau=0.0), INVALID), (dict(chunk=0), INVALID), (dict(H=65), UNSUPPORTED),
        (dict(K=1025), UNSUPPORTED), (dict(hidden=P((1 << 20) + 8)), UNSUPPORTED),
        (dict(workspace=P((1 << 20) + 16)), UNSUPPORTED), (dict(bytes=256), SMALL),
        (dict(T=0, hidden=None), OK)]),
    ("lmhead_distill_bwd", HEAD_BWD, [
        (dict(hidden=None), INVALID), (dict(grad=None), INVALID), (dict(lse=None), INVALID),
        (dict(z_top=None), INVALID), (dict(d_hidden=None), INVALID), (dict(d_weight=None), INVALID),
        (dict(K=1025), UNSUPPORTED), (dict(d_weight=P((1 << 20) + 4)), UNSUPPORTED),
        (dict(d_weight_type=2), INVALID), (dict(d_weight_type=1, accumulate=1), UNSUPPORTED),
        (dict(d_weight_type=1, T=100000, H=4096, chunk=4096, V=151936), UNSUPPORTED),
        (dict(bytes=256), SMALL), (dict(T=0, accumulate=1), OK)]),
    ("lmhead_process_logits_fwd", PROCESS_FWD, [
        (dict(logits=None), INVALID), (dict(out=None), INVALID), (dict(R=-1), INVALID),
        (dict(V=0), INVALID), (dict(ld=99), INVALID), (dict(out_ld=99), INVALID),
        (dict(type=5), INVALID), (dict(spans=None), INVALID), (dict(tokens=None), INVALID),
        (dict(tokens=None, spans=None), INVALID), (dict(n_tokens=-1), INVALID),
        (dict(offsets=None), INVALID), (dict(ids=None), INVALID), (dict(values=None), INVALID),
        (dict(n_bias=-1), INVALID), (dict(allowed=None, allowed_rows=P()), INVALID),
        (dict(n_allowed=7), INVALID), (dict(n_allowed=-1), INVALID),
        (dict(R=(1 << 31) - 256), UNSUPPORTED), (dict(logits=P((1 << 20) + 2)), UNSUPPORTED),
        (dict(R=0), OK)]),
    ("lmhead_process_logits_bwd", PROCESS_BWD, [
        (dict(grad=None), INVALID), (dict(grad_ld=99), INVALID), (dict(logits=None), INVALID),
        (dict(d=None), INVALID), (dict(d_ld=99), INVALID), (dict(tokens=None), INVALID),
        (dict(grad=P((1 << 20) + 2)), UNSUPPORTED), (dict(R=0), OK)]),
]


@pytest.mark.parametrize("name,defaults,wrong", CASES, ids=[c[0] for c in CASES])
def test_refusals(lib, name, defaults, wrong):
    assert len(defaults) == len(lm._SIGNATURES[name][1])
    for over, status in wrong:
        assert call(getattr(lib, name), defaults, **over) == status, (name, over)


def test_workspace_sizes(lib):
    assert lm.lmhead_layernorm_workspace_size(-1, 64) == 0
    assert lm.lmhead_layernorm_workspace_size(4, 0) == 0
    assert lm.lmhead_layernorm_workspace_size(1 << 20, 2560) == \
        lm.lmhead_layernorm_workspace_size(1 << 30, 2560) > 0        # bounded by the GPU, not by N
    base = [lm.lmhead_workspace_size(op, 300, 64, 1000, 8) for op in (0, 1)]
    assert lm.lmhead_distill_workspace_size(0, 300, 64, 1000, 16, 8) >= base[0] + 16 * 300
    assert lm.lmhead_distill_workspace_size(1, 300, 64, 1000, 16, 8) >= base[1] + 6 * 300 * 16
    for bad in ((2, 300, 64, 1000, 16, 8), (0, 300, 65, 1000, 16, 8), (0, 300, 64, 1000, 0, 8),
                (0, 300, 64, 1000, 1025, 8), (1, -1, 64, 1000, 16, 8), (1, 300, 64, 1000, 16, 0)):
        assert lm.lmhead_distill_workspace_size(*bad) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError):
        lm.layernorm_forward(x, w)
    with pytest.raises(TypeError):
        lm.layernorm_forward(x.double(), w)
    ids, top = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        lm.distill_logits_forward(x, ids, top)
    with pytest.raises(ValueError):
        lm.process_logits(x)
    with pytest.raises(TypeError):
        lm.process_logits(x.to(torch.int32))
