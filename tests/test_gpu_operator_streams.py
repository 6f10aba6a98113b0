"""The conveniences of layer norm, distillation and logit processing on a stream of the
caller's: what they allocate belongs to that stream, and the results are the same."""
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


def calls():
    g = torch.Generator("cuda").manual_seed(11)
    T, H, V, K = 300, 128, 4096, 8
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(V, H, generator=g, device="cuda").to(torch.bfloat16)
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda", dtype=torch.int32)
    top = torch.randn(T, K, generator=g, device="cuda")
    logits = torch.randn(T, V, generator=g, device="cuda")
    dy = torch.randn(T, H, generator=g, device="cuda")
    gl = torch.randn(T, generator=g, device="cuda")
    words = torch.randint(-2 ** 31, 2 ** 31, (T, V // 32), generator=g, device="cuda").to(torch.int32)
    _, mean, rstd = lm.layernorm_forward(x, one)
    _, lse, z_top = lm.distill_forward(x, w, ids, top)
    _, lse2 = lm.distill_logits_forward(logits, ids, top)
    return {
        "layernorm_forward": lambda **k: lm.layernorm_forward(x, one, **k),
        "layernorm_backward": lambda **k: lm.layernorm_backward(dy, x, one, mean, rstd, **k),
        "layernorm_backward accumulate": lambda **k: lm.layernorm_backward(
            dy, x, one, mean, rstd, accumulate=True, **k),
        "distill_forward": lambda **k: lm.distill_forward(x, w, ids, top, **k),
        "distill_backward": lambda **k: lm.distill_backward(x, w, ids, top, None, 1.0, 1.0, 512, gl,
                                                            lse, z_top, **k),
        "distill_logits_forward": lambda **k: lm.distill_logits_forward(logits, ids, top, **k),
        "distill_logits_backward": lambda **k: lm.distill_logits_backward(
            logits, ids, top, None, 1.0, 1.0, gl, lse2, **k),
        "process_logits": lambda **k: lm.process_logits(logits, allowed=words, **k),
        "process_logits_backward": lambda **k: lm.process_logits_backward(logits, logits,
                                                                          allowed=words, **k),
    }


def tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("handle", [False, True])
def test_allocations_belong_to_the_stream(handle):
    ensure_built()
    for name, call in calls().items():
        side = torch.cuda.Stream()
        want = tensors(call())
        torch.cuda.synchronize()
        got = tensors(call(stream=side.cuda_stream if handle else side))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), name
        shapes = [(t.shape, t.dtype) for t in got]
        freed = {t.data_ptr() for t in got}
        del got, a
        # the current stream is not given what the other one's calls used
        new = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes]
        assert not freed & {t.data_ptr() for t in new}, name
