"""Out-of-bounds writes of the layer norm, distillation and logit processing
calls: guard bytes around every output, workspace and input stay as they were,
and inputs are unchanged (as test_gpu_guard_canaries does for the head)."""
import numpy as np
import pytest
import torch

import chunked_lm_head_tcgen05_gb300 as lm

from gpu_helpers import ensure_built
from test_gpu_guard_canaries import Guarded, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,h", [(1, 1), (37, 1111), (64, 2560), (5, 20001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layernorm(n, h, dtype):
    ensure_built()
    x = Guarded((n, h), dtype, 1, torch.randn(n, h))
    w = Guarded((h,), torch.float32, 2, torch.randn(h))
    b = Guarded((h,), torch.float32, 3, torch.randn(h))
    y = Guarded((n, h), dtype, 4)
    mean, rstd = Guarded((n,), torch.float32, 5), Guarded((n,), torch.float32, 6)
    gin = dict(x=x, w=w, b=b)
    assert lm.lmhead_layernorm_fwd(x.t, w.t, b.t, 1e-5, y.t, mean.t, rstd.t) == 0
    _check(gin, dict(y=y, mean=mean, rstd=rstd), "fwd")
    mean.rearm()
    rstd.rearm()
    dy = Guarded((n, h), torch.float32, 7, torch.randn(n, h))
    ws = Guarded((lm.lmhead_layernorm_workspace_size(n, h),), torch.uint8, 8)
    out = dict(dx=Guarded((n, h), dtype, 9), dw=Guarded((h,), torch.float32, 10),
               db=Guarded((h,), torch.float32, 11))
    assert lm.lmhead_layernorm_bwd(dy.t, x.t, w.t, mean.t, rstd.t, out["dx"].t, out["dw"].t,
                                   out["db"].t, False, ws.t) == 0
    _check(dict(gin, dy=dy, mean=mean, rstd=rstd), dict(out, ws=ws), "bwd")


def _teacher(T, V, K):
    ids = torch.randint(0, V, (T, K), dtype=torch.int32)
    ids[0, 0] = V - 1
    ids[-1, -1] = 0
    return (Guarded((T, K), torch.int32, 21, ids), Guarded((T, K), torch.float32, 22, torch.randn(T, K)),
            Guarded((T,), torch.uint8, 23, (torch.rand(T) > 0.3).to(torch.uint8)),
            Guarded((T,), torch.float32, 24, torch.randn(T)))


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (7, 3001, 5), (3, 70003, 64), (90, 1000, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distill_logits(T, V, K, dtype):
    ensure_built()
    ids, top, mask, grad = _teacher(T, V, K)
    z = Guarded((T, V), dtype, 25, torch.randn(T, V))
    gin = dict(ids=ids, top=top, mask=mask, grad=grad, z=z)
    out = dict(loss=Guarded((T,), torch.float32, 26), lse=Guarded((T,), torch.float32, 27))
    assert lm.lmhead_distill_logits_fwd(z.t, ids.t, top.t, None, mask.t, 0.7, 1.0, out["loss"].t,
                                        out["lse"].t) == 0
    _check(gin, out, "fwd")
    out["lse"].rearm()
    d = Guarded((T, V), dtype, 28)
    assert lm.lmhead_distill_logits_bwd(z.t, ids.t, top.t, None, mask.t, 0.7, 1.0, grad.t,
                                        out["lse"].t, d.t) == 0
    _check(dict(gin, lse=out["lse"]), dict(d=d), "bwd")


@pytest.mark.parametrize("T,H,V,K,chunk", [(1, 64, 100, 3, 1), (333, 192, 3001, 7, 64),
                                           (257, 320, 1025, 40, 7)])
def test_distill_head(T, H, V, K, chunk):
    ensure_built()
    ids, top, mask, grad = _teacher(T, V, K)
    hidden = Guarded((T, H), torch.bfloat16, 31, torch.randn(T, H))
    weight = Guarded((V, H), torch.bfloat16, 32, torch.randn(V, H) * 0.05)
    gin = dict(ids=ids, top=top, mask=mask, grad=grad, hidden=hidden, weight=weight)
    ws = Guarded((lm.lmhead_distill_workspace_size(0, T, H, V, K, chunk),), torch.uint8, 33)
    out = dict(loss=Guarded((T,), torch.float32, 34), lse=Guarded((T,), torch.float32, 35),
               z=Guarded((T, K), torch.float32, 36))
    assert lm.lmhead_distill_fwd(hidden.t, weight.t, ids.t, top.t, None, mask.t, 1.0, 1.0, chunk,
                                 out["loss"].t, out["lse"].t, out["z"].t, ws.t) == 0
    _check(gin, dict(out, ws=ws), "fwd")
    for b in out.values():
        b.rearm()
    ws = Guarded((lm.lmhead_distill_workspace_size(1, T, H, V, K, chunk),), torch.uint8, 37)
    dh, dw = Guarded((T, H), torch.float32, 38), Guarded((V, H), torch.float32, 39)
    assert lm.lmhead_distill_bwd(hidden.t, weight.t, ids.t, top.t, None, mask.t, 1.0, 1.0, chunk,
                                 grad.t, out["lse"].t, out["z"].t, dh.t, dw.t, 0, ws.t) == 0
    _check(dict(gin, **out), dict(ws=ws, dh=dh, dw=dw), "bwd")


@pytest.mark.parametrize("R,V,n", [(1, 1, 1), (5, 3001, 300), (2, 70003, 5000), (40, 96, 60)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_process_logits(R, V, n, dtype):
    ensure_built()
    g = np.random.default_rng(R + V)
    spans = torch.from_numpy(np.sort(g.integers(0, n + 1, size=(R, 3)), 1).astype(np.int64))
    spans[0] = torch.tensor([0, n // 2, n])
    tokens = torch.from_numpy(g.integers(-3, V + 3, size=n).astype(np.int32))
    gin = dict(z=Guarded((R, V), dtype, 41, torch.randn(R, V)),
               tokens=Guarded((n,), torch.int32, 42, tokens), spans=Guarded((R, 3), torch.int64, 43, spans),
               rep=Guarded((R,), torch.float32, 44, torch.rand(R) + 1),
               fr=Guarded((R,), torch.float32, 45, torch.rand(R)),
               pr=Guarded((R,), torch.float32, 46, torch.rand(R)),
               off=Guarded((R + 1,), torch.int64, 47, torch.arange(R + 1) * 3),
               ids=Guarded((3 * R,), torch.int32, 48, torch.randint(-2, V + 2, (3 * R,), dtype=torch.int32)),
               val=Guarded((3 * R,), torch.float32, 49, torch.randn(3 * R)),
               allowed=Guarded((R, (V + 31) // 32), torch.int32, 50),
               rows=Guarded((R,), torch.int32, 51, torch.randint(-1, R + 1, (R,), dtype=torch.int32)),
               grad=Guarded((R, V), dtype, 52, torch.randn(R, V)))
    t = {k: b.t for k, b in gin.items()}
    out = Guarded((R, V), dtype, 53)
    assert lm.lmhead_process_logits_fwd(t["z"], t["tokens"], t["spans"], t["rep"], t["fr"], t["pr"],
                                        t["off"], t["ids"], t["val"], t["allowed"], t["rows"],
                                        out.t) == 0
    _check(gin, dict(out=out), "fwd")
    d = Guarded((R, V), dtype, 54)
    assert lm.lmhead_process_logits_bwd(t["grad"], t["z"], t["tokens"], t["spans"], t["rep"],
                                        t["allowed"], t["rows"], d.t) == 0
    _check(gin, dict(d=d), "bwd")
