"""PyTorch autograd wrapper over the C ABI, for use inside training loops
(for instance a chunked-sequence trainer whose per-chunk loss is this head;
"Long Sequences (SeCO)" guide, section "Efficiency").

``lmhead_logps(hidden, weight, targets, ...)`` returns (logp, entropy) and
differentiates both through ``lmhead_logps_bwd``.  When the loss does not use
the entropy, its cotangent is absent and the log-prob-only backward runs
(tunix PR #2913: GRPO stops the entropy's gradient).  All computation happens
in the library's kernels; this module only allocates outputs with torch,
keeps one reusable workspace per device and stream, and moves cotangents in
and out.

Weight gradient precision.  A head called once per sequence chunk contributes
one weight gradient per call.  Returned through autograd, each is cast to the
weight's dtype (bf16) before autograd sums them, so the sum would be formed in
bf16.  Give the call an fp32 ``main_grad`` buffer [V, H] (or set
``weight.main_grad``) and the library adds every call's gradient into it in
fp32 (``accumulate_dweight = 1``) instead; ``weight.grad`` is then left
untouched, as in trainers that keep fp32 main gradients beside bf16
parameters.
"""
import functools

import torch

from . import LMHEAD_OP_BWD, LMHEAD_OP_FWD, LmheadError, distill_logits_backward, \
    distill_logits_forward, layernorm_backward, layernorm_forward, lmhead_distill_bwd, \
    lmhead_distill_narrow_dweight, lmhead_distill_fwd, lmhead_distill_workspace_size, \
    lmhead_layernorm_workspace_size, \
    lmhead_logps_bwd, lmhead_logps_fwd, lmhead_workspace_size, process_logits_backward
from . import process_logits as _process_logits

# (device index, stream handle) -> uint8 workspace, grown on demand.  Work on one
# stream runs in order, so every call on that stream can reuse one buffer; the
# backward needs nothing the forward left in it (lse and entropy are passed in).
_workspaces = {}


def _workspace(T, H, V, chunk_size, device):
    n = max(lmhead_workspace_size(LMHEAD_OP_FWD, T, H, V, chunk_size),
            lmhead_workspace_size(LMHEAD_OP_BWD, T, H, V, chunk_size))
    if n == 0:
        raise LmheadError(1, "lmhead_workspace_size")
    return _stream_workspace(n, device)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device):
    """The current stream's, without a Stream object around it where torch can say it so."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class _stream_workspace:
    """The current stream's workspace (at least n bytes), for the time a call enqueues its work.

    It leaves the cache meanwhile: a call is several launches that pass data through
    its workspace, and another thread's call on the same stream could come between
    them.  A call under graph capture gets memory of the graph's own pool, since
    replays go on using it."""

    __slots__ = "key", "buf"

    def __init__(self, n, device):
        if torch.cuda.is_current_stream_capturing():
            self.key, buf = None, None
        else:
            self.key = (device.index, _stream_handle(device))
            buf = _workspaces.pop(self.key, None)
        if buf is None or buf.numel() < n:
            # A smaller buffer replaced here may still be read by work queued on this
            # stream; torch's caching allocator gives its memory only to later work on
            # the same stream, so dropping the reference is safe.
            buf = torch.empty(n, dtype=torch.uint8, device=device)
        self.buf = buf

    def __enter__(self):
        return self.buf

    def __exit__(self, *error):
        if self.key is not None:
            kept = _workspaces.setdefault(self.key, self.buf)
            if kept is not self.buf and kept.numel() < self.buf.numel():
                _workspaces[self.key] = self.buf   # another thread's, a smaller one, came first


def release_workspaces():
    """Drops the cached workspaces (their memory returns to torch's allocator)."""
    _workspaces.clear()


class LMHeadLogps(torch.autograd.Function):
    """(hidden [T,H] bf16, weight [V,H] bf16, targets [T] int32, loss_mask [T] uint8 or
    None, temperature, chunk_size, main_grad [V,H] fp32 or None) -> (logp [T] fp32,
    entropy [T] fp32)."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, loss_mask, temperature, chunk_size, main_grad):
        T, H = hidden.shape
        V = weight.shape[0]
        dev = hidden.device
        logp = torch.empty(T, dtype=torch.float32, device=dev)
        ent = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        with _workspace(T, H, V, chunk_size, dev) as ws:
            rc = lmhead_logps_fwd(hidden, weight, targets, loss_mask, temperature, chunk_size,
                                  logp, ent, lse, ws)
        if rc:
            raise LmheadError(rc, "lmhead_logps_fwd")
        ctx.save_for_backward(hidden, weight, targets, loss_mask, lse, ent)
        ctx.temperature = temperature
        ctx.chunk_size = chunk_size
        ctx.main_grad = main_grad
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(lse)
        return logp, ent

    @staticmethod
    def backward(ctx, g_logp, g_ent):
        hidden, weight, targets, loss_mask, lse, ent = ctx.saved_tensors
        T, H = hidden.shape
        V = weight.shape[0]
        dev = hidden.device
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        main = ctx.main_grad if need_w else None
        if (g_logp is None and g_ent is None) or not (need_h or need_w):
            return (None,) * 7
        gl = None if g_logp is None else g_logp.to(torch.float32).contiguous()
        ge = None if g_ent is None else g_ent.to(torch.float32).contiguous()
        d_hidden = torch.empty((T, H), dtype=torch.float32, device=dev)
        if main is not None:
            d_weight, accumulate = main, 1
        else:
            d_weight, accumulate = torch.empty((V, H), dtype=torch.float32, device=dev), 0
        with _workspace(T, H, V, ctx.chunk_size, dev) as ws:
            rc = lmhead_logps_bwd(hidden, weight, targets, loss_mask, ctx.temperature,
                                  ctx.chunk_size, gl, ge, lse, ent if ge is not None else None,
                                  d_hidden, d_weight, accumulate, ws)
        if rc:
            raise LmheadError(rc, "lmhead_logps_bwd")
        d_w = d_weight if (need_w and main is None) else None
        return (d_hidden if need_h else None, d_w, None, None, None, None, None)


def lmhead_logps(hidden, weight, targets, loss_mask=None, temperature=1.0, chunk_size=512,
                 main_grad=None):
    """Per-token log-prob of the target and entropy, differentiable in hidden and weight.

    main_grad: an fp32 [V, H] CUDA tensor that the backward adds the weight's
    gradient to (in fp32, in place); defaults to ``weight.main_grad`` when the
    weight has one.  With it, ``weight.grad`` is not produced."""
    return LMHeadLogps.apply(hidden, weight, targets, loss_mask, float(temperature),
                             int(chunk_size), _main_grad(weight, main_grad))


def _main_grad(weight, main_grad):
    """The fp32 buffer the weight's gradient is added to: the argument, the weight's own, or
    None."""
    if main_grad is None:
        main_grad = getattr(weight, "main_grad", None)
    if main_grad is not None:
        V, H = weight.shape
        if (main_grad.dtype != torch.float32 or tuple(main_grad.shape) != (V, H)
                or not main_grad.is_contiguous() or main_grad.device != weight.device):
            raise ValueError("main_grad must be a contiguous fp32 [V, H] tensor on the "
                             "weight's device")
    return main_grad


class _Once(torch.autograd.Function):
    """(n, n gradients, what they were formed from) -> the gradients, whose own backward raises."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *cotangents):
        raise RuntimeError("this function is differentiable once: its gradient comes from the "
                           "library's kernels, whose own derivative torch does not know")


def _differentiable_once(backward):
    """A backward whose gradients refuse to be differentiated again (create_graph=True) instead of
    passing for constants.  torch's own once_differentiable looks at the cotangents only; these
    gradients depend on the saved tensors too."""
    @functools.wraps(backward)
    def first(ctx, *cotangents):
        with torch.no_grad():
            grads = backward(ctx, *cotangents)
        if not torch.is_grad_enabled():
            return grads
        at = [i for i, t in enumerate(grads) if t is not None]
        marked = _Once.apply(len(at), *(grads[i] for i in at), *cotangents, *ctx.saved_tensors)
        return tuple(marked[at.index(i)] if i in at else None for i in range(len(grads)))
    return first


class LMHeadDistill(torch.autograd.Function):
    """(hidden [T,H] bf16, weight [V,H] bf16, top_ids [T,K] int32, top_logits [T,K] fp32,
    loss_mask, temperature, teacher_temperature, chunk_size, teacher_lse [T] fp32 or None,
    main_grad) -> loss [T] fp32."""

    @staticmethod
    def forward(ctx, hidden, weight, top_ids, top_logits, loss_mask, temperature,
                teacher_temperature, chunk_size, teacher_lse, main_grad):
        T, H = hidden.shape
        V = weight.shape[0]
        K = top_ids.shape[1]
        dev = hidden.device
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        z_top = torch.empty((T, K), dtype=torch.float32, device=dev)
        sizes = [lmhead_distill_workspace_size(op, T, H, V, K, chunk_size)
                 for op in (LMHEAD_OP_FWD, LMHEAD_OP_BWD)]
        if 0 in sizes:
            raise LmheadError(1, "lmhead_distill_workspace_size")
        with _stream_workspace(max(sizes), dev) as ws:
            rc = lmhead_distill_fwd(hidden, weight, top_ids, top_logits, teacher_lse, loss_mask,
                                    temperature, teacher_temperature, chunk_size, loss, lse,
                                    z_top, ws)
        if rc:
            raise LmheadError(rc, "lmhead_distill_fwd")
        ctx.save_for_backward(hidden, weight, top_ids, top_logits, loss_mask, teacher_lse, lse,
                              z_top)
        ctx.temperatures = temperature, teacher_temperature
        ctx.chunk_size = chunk_size
        ctx.workspace_bytes = max(sizes)
        ctx.main_grad = main_grad
        return loss

    @staticmethod
    @_differentiable_once
    def backward(ctx, g_loss):
        hidden, weight, top_ids, top_logits, loss_mask, teacher_lse, lse, z_top = ctx.saved_tensors
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_h or need_w):
            return (None,) * 10
        main = ctx.main_grad if need_w else None
        T, H = hidden.shape
        V = weight.shape[0]
        dev = hidden.device
        d_hidden = torch.empty((T, H), dtype=torch.float32, device=dev)
        if main is not None:
            d_weight = main
        else:   # autograd hands the parameter its own type: bf16 at once where the library can
            kind = torch.bfloat16 if lmhead_distill_narrow_dweight(T, H, V, ctx.chunk_size) \
                else torch.float32
            d_weight = torch.empty((V, H), dtype=kind, device=dev)
        g_loss = g_loss.to(torch.float32).contiguous()
        with _stream_workspace(ctx.workspace_bytes, dev) as ws:
            rc = lmhead_distill_bwd(hidden, weight, top_ids, top_logits, teacher_lse, loss_mask,
                                    *ctx.temperatures, ctx.chunk_size, g_loss, lse, z_top,
                                    d_hidden, d_weight, main is not None, ws)
        if rc:
            raise LmheadError(rc, "lmhead_distill_bwd")
        return (d_hidden if need_h else None, d_weight if need_w and main is None else None,
                *(None,) * 8)


def lmhead_distill(hidden, weight, top_ids, top_logits, loss_mask=None, temperature=1.0,
                   teacher_temperature=1.0, chunk_size=512, teacher_lse=None, main_grad=None):
    """Per-token distillation loss from a teacher's top logits through the head (the [T, V]
    logits never exist), differentiable in hidden and weight.  main_grad as in
    ``lmhead_logps``."""
    return LMHeadDistill.apply(hidden, weight, top_ids, top_logits, loss_mask, float(temperature),
                               float(teacher_temperature), int(chunk_size), teacher_lse,
                               _main_grad(weight, main_grad))


class DistillLogits(torch.autograd.Function):
    """(logits [T,V], top_ids, top_logits, loss_mask, temperature, teacher_temperature,
    teacher_lse) -> loss [T] fp32."""

    @staticmethod
    def forward(ctx, logits, top_ids, top_logits, loss_mask, temperature, teacher_temperature,
                teacher_lse):
        loss, lse = distill_logits_forward(logits, top_ids, top_logits, loss_mask, temperature,
                                           teacher_temperature, teacher_lse)
        ctx.save_for_backward(logits, top_ids, top_logits, loss_mask, teacher_lse, lse)
        ctx.temperatures = temperature, teacher_temperature
        return loss

    @staticmethod
    @_differentiable_once
    def backward(ctx, g_loss):
        logits, top_ids, top_logits, loss_mask, teacher_lse, lse = ctx.saved_tensors
        d = distill_logits_backward(logits, top_ids, top_logits, loss_mask, *ctx.temperatures,
                                    g_loss.to(torch.float32).contiguous(), lse, teacher_lse)
        return (d, *(None,) * 6)


def distill_logits(logits, top_ids, top_logits, loss_mask=None, temperature=1.0,
                   teacher_temperature=1.0, teacher_lse=None):
    """Per-token distillation loss on held logits, differentiable in the logits."""
    return DistillLogits.apply(logits, top_ids, top_logits, loss_mask, float(temperature),
                               float(teacher_temperature), teacher_lse)


class LayerNorm(torch.autograd.Function):
    """(x [N,H], weight [H], bias [H] or None, eps, out_dtype) -> y [N,H]."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, mean, rstd = layernorm_forward(x, weight, bias, eps, out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @_differentiable_once
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        if dy.stride(1) != 1 or (dy.shape[0] > 1 and dy.stride(0) < dy.shape[1]):
            dy = dy.contiguous()
        need_b = ctx.needs_input_grad[2]
        with _stream_workspace(lmhead_layernorm_workspace_size(*x.shape), x.device) as ws:
            dx, dw, db = layernorm_backward(dy, x, weight, mean, rstd, with_bias=need_b,
                                            workspace=ws)
        return (dx, dw, db, None, None)


def layer_norm(x, weight, bias=None, eps=1e-5, out_dtype=None):
    """Layer norm of x [N, H] (fp32, bf16 or fp16; out_dtype bf16 for fp32 rows),
    differentiable in x, weight and bias."""
    return LayerNorm.apply(x, weight, bias, float(eps), out_dtype)


_RULES = {"tokens", "spans", "repetition", "frequency", "presence", "bias_offsets", "bias_ids",
          "bias_values", "allowed", "allowed_rows"}


class ProcessLogits(torch.autograd.Function):
    """(logits [R,V], rules as keyword arguments of ``process_logits``) -> processed [R,V]."""

    _BACKWARD = "tokens", "spans", "repetition", "allowed", "allowed_rows"   # rules it needs

    @staticmethod
    def forward(ctx, logits, rules):
        # saved, so that a buffer the sampler has rewritten by the time of the backward is refused
        ctx.save_for_backward(logits, *(rules.get(k) for k in ProcessLogits._BACKWARD))
        return _process_logits(logits, **rules)

    @staticmethod
    @_differentiable_once
    def backward(ctx, g):
        logits, *rules = ctx.saved_tensors
        if g.stride(1) != 1 or (g.shape[0] > 1 and g.stride(0) < g.shape[1]):
            g = g.contiguous()
        rules = dict(zip(ProcessLogits._BACKWARD, rules))
        return process_logits_backward(g, logits, **rules), None


def process_logits(logits, **rules):
    """``chunked_lm_head_tcgen05_gb300.process_logits`` (the same keyword arguments, without
    ``out`` and ``stream``), differentiable in the logits."""
    unknown = sorted(rules.keys() - _RULES)
    if unknown:
        raise TypeError("process_logits takes no %s here" % ", ".join(unknown))
    return ProcessLogits.apply(logits, rules)
