"""Chunked LM-head log-prob + entropy head for GB300 (sm_103a).

Thin Python binding over the C ABI in ``include/lmhead.h`` (``liblmhead.so``,
built by ``buildlib.py``).  The functions named ``lmhead_*`` mirror the C entry
points one to one and only marshal arguments: torch tensors supply device
memory and the CUDA stream, every step of the computation runs in the
library's kernels.  There is no CPU or PyTorch fallback: if the library is
missing or cannot load, every call raises.

``forward`` / ``backward`` are conveniences that allocate the outputs and the
workspace with torch and raise ``LmheadError`` on a non-zero status.
"""
import ctypes
import functools
import os

__all__ = [
    "LmheadError", "library", "library_path", "build",
    "LMHEAD_OP_FWD", "LMHEAD_OP_BWD", "STATUS_NAMES",
    "lmhead_workspace_size", "lmhead_logps_fwd", "lmhead_logps_bwd",
    "lmhead_read_device_status", "lmhead_read_scored_count", "lmhead_status_string",
    "lmhead_plan_info", "lmhead_profile_enable", "lmhead_profile_count",
    "lmhead_profile_record", "lmhead_launch_count", "lmhead_logps_fwd_noalloc",
    "NOALLOC_SCRATCH_BYTES", "lmhead_logps_fwd_bwd", "lmhead_fwd_bwd_keeps_logits",
    "LMHEAD_OP_FWD_BWD", "LMHEAD_STRATEGY_AUTO", "LMHEAD_STRATEGY_RECOMPUTE",
    "LMHEAD_STRATEGY_KEEP_LOGITS", "lmhead_score_logits_fwd", "lmhead_score_logits_bwd",
    "lmhead_selftest_bounded_wait", "lmhead_logps_fwd_shard", "lmhead_logps_bwd_shard",
    "lmhead_combine_shards",
    "forward", "backward",
    "LMHEAD_F32", "LMHEAD_BF16", "LMHEAD_F16",
    "lmhead_distill_workspace_size", "lmhead_distill_fwd", "lmhead_distill_bwd",
    "lmhead_distill_narrow_dweight",
    "lmhead_distill_logits_fwd", "lmhead_distill_logits_bwd",
    "lmhead_layernorm_workspace_size", "lmhead_layernorm_fwd", "lmhead_layernorm_bwd",
    "lmhead_process_logits_fwd", "lmhead_process_logits_bwd",
    "distill_forward", "distill_backward", "distill_logits_forward", "distill_logits_backward",
    "layernorm_forward", "layernorm_backward", "process_logits", "process_logits_backward",
]

LMHEAD_OP_FWD = 0
LMHEAD_OP_BWD = 1
LMHEAD_OP_FWD_BWD = 2
LMHEAD_STRATEGY_AUTO = 0
LMHEAD_STRATEGY_RECOMPUTE = 1
LMHEAD_STRATEGY_KEEP_LOGITS = 2
LMHEAD_F32 = 0
LMHEAD_BF16 = 1
LMHEAD_F16 = 2
NOALLOC_SCRATCH_BYTES = 64 << 20   # LMHEAD_NOALLOC_SCRATCH_BYTES in include/lmhead.h
STATUS_NAMES = {
    0: "LMHEAD_OK", 1: "LMHEAD_ERR_INVALID_ARG", 2: "LMHEAD_ERR_UNSUPPORTED",
    3: "LMHEAD_ERR_WORKSPACE_TOO_SMALL", 4: "LMHEAD_ERR_CUDA",
    5: "LMHEAD_ERR_DEVICE_TIMEOUT", 6: "LMHEAD_ERR_BAD_TARGET", 7: "LMHEAD_ERR_INTERNAL",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "liblmhead.so")
_lib = None

_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

# name -> (restype, argtypes), exactly the declarations of include/lmhead.h
_SIGNATURES = {
    "lmhead_workspace_size": (_SZ, [ctypes.c_int, _I64, _I32, _I32, _I32]),
    "lmhead_logps_fwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I64, _I32, _I32, ctypes.c_float,
                                        _I32, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "lmhead_logps_bwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I64, _I32, _I32, ctypes.c_float,
                                        _I32, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP,
                                        _SZ, _VP]),
    "lmhead_read_device_status": (ctypes.c_int, [_VP, _VP]),
    "lmhead_read_scored_count": (_I64, [_VP, _VP]),
    "lmhead_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "lmhead_plan_info": (ctypes.c_int, [_I64, _I32, _I32, _I32, ctypes.POINTER(_I32),
                                        ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "lmhead_profile_enable": (None, [ctypes.c_int]),
    "lmhead_profile_count": (ctypes.c_int, []),
    "lmhead_profile_record": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                             ctypes.POINTER(ctypes.c_float)]),
    "lmhead_launch_count": (ctypes.c_uint64, []),
    "lmhead_logps_fwd_noalloc": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I64, _I32, _I32,
                                                ctypes.c_float, _I32, _VP, _VP, _VP, _VP]),
    "lmhead_logps_fwd_bwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I64, _I32, _I32,
                                            ctypes.c_float, _I32, _VP, _VP, _VP, _VP, _VP, _VP,
                                            _VP, ctypes.c_int, ctypes.c_int, _VP, _SZ, _VP]),
    "lmhead_fwd_bwd_keeps_logits": (ctypes.c_int, [_I64, _I32, _I32, _I32,
                                                   ctypes.POINTER(_I32)]),
    "lmhead_selftest_bounded_wait": (ctypes.c_int, [_VP, _SZ, ctypes.c_uint32, _VP]),
    "lmhead_score_logits_fwd": (ctypes.c_int, [_VP, _VP, _VP, _I64, _I32, ctypes.c_float, _VP,
                                               _VP, _VP, _VP]),
    "lmhead_score_logits_bwd": (ctypes.c_int, [_VP, _VP, _VP, _I64, _I32, ctypes.c_float, _VP,
                                               _VP, _VP, _VP, _VP, _VP]),
    "lmhead_logps_fwd_shard": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _I32,
                                              ctypes.c_float, _I32, _VP, _VP, _SZ, _VP]),
    "lmhead_combine_shards": (ctypes.c_int, [_VP, _I32, _VP, _VP, _I64, _I32, _VP, _VP, _VP,
                                             _VP]),
    "lmhead_logps_bwd_shard": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32, _I32,
                                              ctypes.c_float, _I32, _VP, _VP, _VP, _VP, _VP, _VP,
                                              ctypes.c_int, _VP, _SZ, _VP]),
    "lmhead_distill_workspace_size": (_SZ, [ctypes.c_int, _I64, _I32, _I32, _I32, _I32]),
    "lmhead_distill_fwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32,
                                          ctypes.c_float, ctypes.c_float, _I32, _VP, _VP, _VP,
                                          _VP, _SZ, _VP]),
    "lmhead_distill_bwd": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _I32, _I32, _I32,
                                          ctypes.c_float, ctypes.c_float, _I32, _VP, _VP, _VP,
                                          _VP, _VP, ctypes.c_int, ctypes.c_int, _VP, _SZ, _VP]),
    "lmhead_distill_narrow_dweight": (ctypes.c_int, [_I64, _I32, _I32, _I32]),
    "lmhead_distill_logits_fwd": (ctypes.c_int, [_VP, ctypes.c_int, _I64, _VP, _VP, _VP, _VP, _I64,
                                                 _I32, _I32, ctypes.c_float, ctypes.c_float, _VP,
                                                 _VP, _VP]),
    "lmhead_distill_logits_bwd": (ctypes.c_int, [_VP, ctypes.c_int, _I64, _VP, _VP, _VP, _VP, _I64,
                                                 _I32, _I32, ctypes.c_float, ctypes.c_float, _VP,
                                                 _VP, _VP, _I64, _VP]),
    "lmhead_layernorm_workspace_size": (_SZ, [_I64, _I32]),
    "lmhead_layernorm_fwd": (ctypes.c_int, [_VP, ctypes.c_int, _I64, _VP, _VP, ctypes.c_int, _I64,
                                            _I32, ctypes.c_float, _VP, ctypes.c_int, _I64, _VP,
                                            _VP, _VP]),
    "lmhead_layernorm_bwd": (ctypes.c_int, [_VP, ctypes.c_int, _I64, _VP, ctypes.c_int, _I64, _VP,
                                            ctypes.c_int, _VP, _VP, _I64, _I32, _VP, _I64, _VP,
                                            _VP, ctypes.c_int, _VP, _SZ, _VP]),
    "lmhead_process_logits_fwd": (ctypes.c_int, [_VP, ctypes.c_int, _I64, _I64, _I32, _VP, _I64,
                                                 _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP,
                                                 _I64, _VP, _VP, _I64, _VP]),
    "lmhead_process_logits_bwd": (ctypes.c_int, [_VP, _I64, _VP, ctypes.c_int, _I64, _I64, _I32,
                                                 _VP, _I64, _VP, _VP, _VP, _I64, _VP, _VP, _I64,
                                                 _VP]),
}


class LmheadError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = int(status)
        super().__init__("%s%s" % (where + ": " if where else "",
                                   STATUS_NAMES.get(self.status, "status %d" % self.status)))


def build(force=False):
    """Compile liblmhead.so for sm_103a (nvcc); returns its path."""
    from . import buildlib
    return buildlib.build(force=force)


def library():
    """The loaded liblmhead.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError("liblmhead.so is not built (run chunked_lm_head_tcgen05_gb300.build())")
        lib = ctypes.CDLL(library_path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


# Bound on first use (importing this package does not import torch).
_torch = None
_types = None
_raw_stream = None


def _bind_torch():
    global _torch, _types, _raw_stream
    import torch
    _types = {torch.float32: LMHEAD_F32, torch.bfloat16: LMHEAD_BF16, torch.float16: LMHEAD_F16}
    # the handle without a Stream object around it (about 2 us a call less)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _torch = torch


def _stream(stream):
    if stream is None:
        if _torch is None:
            _bind_torch()
        if _raw_stream is not None:
            return _raw_stream(_torch.cuda.current_device())
        return _torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensor(t, name, dtype, shape, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise ValueError("%s is required" % name)
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _on_device(tensors, stream, fn):
    """Run fn() with the tensors' CUDA device current.  The library launches
    on the current device, so a call whose tensors (or stream) live on
    another device, or on several, is refused here instead of launched."""
    if _torch is None:
        _bind_torch()
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors and the stream of one call must be on one CUDA device, "
                             "got %s" % sorted({str(t.device) for t in tensors if t is not None}))
    if stream is not None and not isinstance(stream, int) and hasattr(stream, "device"):
        if dev is not None and stream.device != dev:
            raise ValueError("all tensors and the stream of one call must be on one CUDA device, "
                             "got %s" % sorted({str(dev), str(stream.device)}))
        dev = stream.device
    if dev is None or dev.index == _torch.cuda.current_device():
        return fn()
    with _torch.cuda.device(dev):
        return fn()


def _one_device(first, *others):
    """Index of the CUDA device all of these tensors are on."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors and the stream of one call must be on one CUDA device, "
                             "got %s" % sorted({str(x.device) for x in (first,) + others
                                                if x is not None}))
    return dev


def _call(fn, dev, stream, *args):
    """fn(*args, stream handle) with CUDA device `dev` current."""
    if stream is None:
        handle = (_raw_stream(dev) if _raw_stream is not None
                  else _torch.cuda.current_stream(dev).cuda_stream)
    elif isinstance(stream, int):
        handle = stream
    else:
        if stream.device.index != dev:
            raise ValueError("all tensors and the stream of one call must be on one CUDA device, "
                             "got %s" % sorted({"cuda:%d" % dev, str(stream.device)}))
        handle = stream.cuda_stream
    if dev == _torch.cuda.current_device():
        return fn(*args, handle)
    with _torch.cuda.device(dev):
        return fn(*args, handle)


def _check_workspace(ws):
    if ws is None or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")


def _check_rows(t, name, shape, dtypes=None):
    """A CUDA matrix whose rows are contiguous but may lie further apart than their
    length; returns (element type, elements between rows)."""
    if t is None:
        raise ValueError("%s is required" % name)
    if _torch is None:
        _bind_torch()
    kind = _types.get(t.dtype)
    if kind is None or (dtypes is not None and t.dtype not in dtypes):
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(
            str(d) for d in (dtypes if dtypes is not None else _types)), t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    rows, cols = shape
    ld, step = t.stride()
    if rows <= 1:
        ld = max(cols, ld)
    if (cols > 1 and step != 1) or ld < cols:
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return kind, ld


def _check_teacher(top_ids, top_logits, teacher_lse, loss_mask, T):
    if _torch is None:
        _bind_torch()
    torch = _torch
    K = top_ids.shape[1] if top_ids.dim() == 2 else -1
    _check_tensor(top_ids, "top_ids", torch.int32, (T, K))
    _check_tensor(top_logits, "top_logits", torch.float32, (T, K))
    _check_tensor(teacher_lse, "teacher_lse", torch.float32, (T,), allow_none=True)
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    return K


def lmhead_workspace_size(op, T, H, V, chunk_size):
    return int(library().lmhead_workspace_size(op, T, H, V, chunk_size))


def lmhead_logps_fwd(hidden, weight, targets, loss_mask, temperature, chunk_size, logp, entropy,
                     lse, workspace, stream=None):
    """C ``lmhead_logps_fwd`` on torch tensors; returns the status code."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight, "weight", torch.bfloat16, (V, H))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(logp, "logp", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_workspace(workspace)
    tensors = [hidden, weight, targets, loss_mask, logp, entropy, lse, workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_logps_fwd(
        _ptr(hidden), _ptr(weight), _ptr(targets), _ptr(loss_mask), T, H, V, float(temperature),
        int(chunk_size), _ptr(logp), _ptr(entropy), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))))


def lmhead_logps_bwd(hidden, weight, targets, loss_mask, temperature, chunk_size, grad_logp,
                     grad_entropy, lse, entropy, d_hidden, d_weight, accumulate_dweight, workspace,
                     stream=None):
    """C ``lmhead_logps_bwd`` on torch tensors; returns the status code."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight, "weight", torch.bfloat16, (V, H))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(grad_logp, "grad_logp", torch.float32, (T,), allow_none=True)
    _check_tensor(grad_entropy, "grad_entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(d_hidden, "d_hidden", torch.float32, (T, H))
    _check_tensor(d_weight, "d_weight", torch.float32, (V, H))
    _check_workspace(workspace)
    tensors = [hidden, weight, targets, loss_mask, grad_logp, grad_entropy, lse, entropy,
               d_hidden, d_weight, workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_logps_bwd(
        _ptr(hidden), _ptr(weight), _ptr(targets), _ptr(loss_mask), T, H, V, float(temperature),
        int(chunk_size), _ptr(grad_logp), _ptr(grad_entropy), _ptr(lse), _ptr(entropy),
        _ptr(d_hidden), _ptr(d_weight), int(bool(accumulate_dweight)), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))))


def lmhead_logps_fwd_noalloc(hidden, weight, targets, loss_mask, temperature, chunk_size, logp,
                             entropy, lse, stream=None):
    """C ``lmhead_logps_fwd_noalloc`` on torch tensors; returns the status code.

    For callers that cannot allocate device memory: no workspace argument,
    the scratch is the library's static per-GPU array (up to
    LMHEAD_NOALLOC_SCRATCH_BYTES of forward workspace)."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight, "weight", torch.bfloat16, (V, H))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(logp, "logp", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    tensors = [hidden, weight, targets, loss_mask, logp, entropy, lse]
    return _on_device(tensors, stream, lambda: int(library().lmhead_logps_fwd_noalloc(
        _ptr(hidden), _ptr(weight), _ptr(targets), _ptr(loss_mask), T, H, V, float(temperature),
        int(chunk_size), _ptr(logp), _ptr(entropy), _ptr(lse), _stream(stream))))


def lmhead_logps_fwd_bwd(hidden, weight, targets, loss_mask, temperature, chunk_size, grad_logp,
                         grad_entropy, logp, entropy, lse, d_hidden, d_weight,
                         accumulate_dweight, strategy, workspace, stream=None):
    """C ``lmhead_logps_fwd_bwd`` on torch tensors; returns the status code."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight, "weight", torch.bfloat16, (V, H))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(grad_logp, "grad_logp", torch.float32, (T,), allow_none=True)
    _check_tensor(grad_entropy, "grad_entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(logp, "logp", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_tensor(d_hidden, "d_hidden", torch.float32, (T, H))
    _check_tensor(d_weight, "d_weight", torch.float32, (V, H))
    _check_workspace(workspace)
    tensors = [hidden, weight, targets, loss_mask, grad_logp, grad_entropy, logp, entropy, lse,
               d_hidden, d_weight, workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_logps_fwd_bwd(
        _ptr(hidden), _ptr(weight), _ptr(targets), _ptr(loss_mask), T, H, V, float(temperature),
        int(chunk_size), _ptr(grad_logp), _ptr(grad_entropy), _ptr(logp), _ptr(entropy),
        _ptr(lse), _ptr(d_hidden), _ptr(d_weight), int(bool(accumulate_dweight)), int(strategy),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))))


def lmhead_fwd_bwd_keeps_logits(T, H, V, chunk_size):
    """(keeps logits under AUTO: bool, token block of the keep-logits path)."""
    tb = _I32()
    r = int(library().lmhead_fwd_bwd_keeps_logits(T, H, V, chunk_size, ctypes.byref(tb)))
    if r < 0:
        raise LmheadError(1, "lmhead_fwd_bwd_keeps_logits")
    return bool(r), tb.value


def lmhead_score_logits_fwd(logits, targets, loss_mask, temperature, logp, entropy, lse,
                            stream=None):
    """C ``lmhead_score_logits_fwd`` on torch tensors; returns the status code."""
    import torch
    T, V = logits.shape
    _check_tensor(logits, "logits", torch.float32, (T, V))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(logp, "logp", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    tensors = [logits, targets, loss_mask, logp, entropy, lse]
    return _on_device(tensors, stream, lambda: int(library().lmhead_score_logits_fwd(
        _ptr(logits), _ptr(targets), _ptr(loss_mask), T, V, float(temperature), _ptr(logp),
        _ptr(entropy), _ptr(lse), _stream(stream))))


def lmhead_score_logits_bwd(logits, targets, loss_mask, temperature, grad_logp, grad_entropy,
                            lse, entropy, d_logits, stream=None):
    """C ``lmhead_score_logits_bwd`` on torch tensors; returns the status code."""
    import torch
    T, V = logits.shape
    _check_tensor(logits, "logits", torch.float32, (T, V))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(grad_logp, "grad_logp", torch.float32, (T,), allow_none=True)
    _check_tensor(grad_entropy, "grad_entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(d_logits, "d_logits", torch.float32, (T, V))
    tensors = [logits, targets, loss_mask, grad_logp, grad_entropy, lse, entropy, d_logits]
    return _on_device(tensors, stream, lambda: int(library().lmhead_score_logits_bwd(
        _ptr(logits), _ptr(targets), _ptr(loss_mask), T, V, float(temperature), _ptr(grad_logp),
        _ptr(grad_entropy), _ptr(lse), _ptr(entropy), _ptr(d_logits), _stream(stream))))


def lmhead_logps_fwd_shard(hidden, weight_shard, targets, loss_mask, vocab_offset, vocab_total,
                           temperature, chunk_size, partials, workspace, stream=None):
    """C ``lmhead_logps_fwd_shard`` on torch tensors (partials: fp32 [T, 4]); returns
    the status code."""
    import torch
    T, H = hidden.shape
    Vs = weight_shard.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight_shard, "weight_shard", torch.bfloat16, (Vs, H))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(partials, "partials", torch.float32, (T, 4))
    _check_workspace(workspace)
    tensors = [hidden, weight_shard, targets, loss_mask, partials, workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_logps_fwd_shard(
        _ptr(hidden), _ptr(weight_shard), _ptr(targets), _ptr(loss_mask), T, H, Vs,
        int(vocab_offset), int(vocab_total), float(temperature), int(chunk_size), _ptr(partials),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))))


def lmhead_combine_shards(partials, targets, loss_mask, vocab_total, logp, entropy, lse,
                          stream=None):
    """C ``lmhead_combine_shards`` (partials: fp32 [n_shards, T, 4]); returns the status."""
    import torch
    n, T = partials.shape[0], partials.shape[1]
    _check_tensor(partials, "partials", torch.float32, (n, T, 4))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(logp, "logp", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    tensors = [partials, targets, loss_mask, logp, entropy, lse]
    return _on_device(tensors, stream, lambda: int(library().lmhead_combine_shards(
        _ptr(partials), n, _ptr(targets), _ptr(loss_mask), T, int(vocab_total), _ptr(logp),
        _ptr(entropy), _ptr(lse), _stream(stream))))


def lmhead_logps_bwd_shard(hidden, weight_shard, targets, loss_mask, vocab_offset, vocab_total,
                           temperature, chunk_size, grad_logp, grad_entropy, lse, entropy,
                           d_hidden, d_weight_shard, accumulate_dweight, workspace, stream=None):
    """C ``lmhead_logps_bwd_shard`` on torch tensors; returns the status code."""
    import torch
    T, H = hidden.shape
    Vs = weight_shard.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight_shard, "weight_shard", torch.bfloat16, (Vs, H))
    _check_tensor(targets, "targets", torch.int32, (T,))
    _check_tensor(loss_mask, "loss_mask", torch.uint8, (T,), allow_none=True)
    _check_tensor(grad_logp, "grad_logp", torch.float32, (T,), allow_none=True)
    _check_tensor(grad_entropy, "grad_entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_tensor(entropy, "entropy", torch.float32, (T,), allow_none=True)
    _check_tensor(d_hidden, "d_hidden", torch.float32, (T, H))
    _check_tensor(d_weight_shard, "d_weight_shard", torch.float32, (Vs, H))
    _check_workspace(workspace)
    tensors = [hidden, weight_shard, targets, loss_mask, grad_logp, grad_entropy, lse, entropy,
               d_hidden, d_weight_shard, workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_logps_bwd_shard(
        _ptr(hidden), _ptr(weight_shard), _ptr(targets), _ptr(loss_mask), T, H, Vs,
        int(vocab_offset), int(vocab_total), float(temperature), int(chunk_size),
        _ptr(grad_logp), _ptr(grad_entropy), _ptr(lse), _ptr(entropy), _ptr(d_hidden),
        _ptr(d_weight_shard), int(bool(accumulate_dweight)), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))))


def lmhead_distill_workspace_size(op, T, H, V, K, chunk_size):
    return int(library().lmhead_distill_workspace_size(op, T, H, V, K, chunk_size))


def lmhead_distill_narrow_dweight(T, H, V, chunk_size):
    """Whether ``lmhead_distill_bwd`` can write d_weight in bf16 for these sizes."""
    return bool(library().lmhead_distill_narrow_dweight(T, H, V, chunk_size))


def lmhead_distill_fwd(hidden, weight, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                       teacher_temperature, chunk_size, loss, lse, z_top, workspace, stream=None):
    """C ``lmhead_distill_fwd`` on torch tensors; returns the status code."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight, "weight", torch.bfloat16, (V, H))
    K = _check_teacher(top_ids, top_logits, teacher_lse, loss_mask, T)
    _check_tensor(loss, "loss", torch.float32, (T,))
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_tensor(z_top, "z_top", torch.float32, (T, K))
    _check_workspace(workspace)
    tensors = [hidden, weight, top_ids, top_logits, teacher_lse, loss_mask, loss, lse, z_top,
               workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_distill_fwd(
        _ptr(hidden), _ptr(weight), _ptr(top_ids), _ptr(top_logits), _ptr(teacher_lse),
        _ptr(loss_mask), T, H, V, K, float(temperature), float(teacher_temperature),
        int(chunk_size), _ptr(loss), _ptr(lse), _ptr(z_top), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))))


def lmhead_distill_bwd(hidden, weight, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                       teacher_temperature, chunk_size, grad_loss, lse, z_top, d_hidden, d_weight,
                       accumulate_dweight, workspace, stream=None):
    """C ``lmhead_distill_bwd`` on torch tensors (d_weight fp32, or bf16 where
    ``lmhead_distill_narrow_dweight``); returns the status code."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    _check_tensor(hidden, "hidden", torch.bfloat16, (T, H))
    _check_tensor(weight, "weight", torch.bfloat16, (V, H))
    K = _check_teacher(top_ids, top_logits, teacher_lse, loss_mask, T)
    _check_tensor(grad_loss, "grad_loss", torch.float32, (T,))
    _check_tensor(lse, "lse", torch.float32, (T,))
    _check_tensor(z_top, "z_top", torch.float32, (T, K))
    _check_tensor(d_hidden, "d_hidden", torch.float32, (T, H))
    kind = LMHEAD_BF16 if d_weight is not None and d_weight.dtype is torch.bfloat16 else LMHEAD_F32
    _check_tensor(d_weight, "d_weight", torch.bfloat16 if kind else torch.float32, (V, H))
    _check_workspace(workspace)
    tensors = [hidden, weight, top_ids, top_logits, teacher_lse, loss_mask, grad_loss, lse, z_top,
               d_hidden, d_weight, workspace]
    return _on_device(tensors, stream, lambda: int(library().lmhead_distill_bwd(
        _ptr(hidden), _ptr(weight), _ptr(top_ids), _ptr(top_logits), _ptr(teacher_lse),
        _ptr(loss_mask), T, H, V, K, float(temperature), float(teacher_temperature),
        int(chunk_size), _ptr(grad_loss), _ptr(lse), _ptr(z_top), _ptr(d_hidden),
        _ptr(d_weight), kind, int(bool(accumulate_dweight)), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))))


def _distill_logits_fwd(logits, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                        teacher_temperature, out, stream):
    T, V = logits.shape
    kind, ld = _check_rows(logits, "logits", (T, V))
    K = _check_teacher(top_ids, top_logits, teacher_lse, loss_mask, T)
    if out is None:
        new = dict(dtype=_torch.float32, device=logits.device)
        out = _torch.empty(T, **new), _torch.empty(T, **new)
        dev = _one_device(logits, top_ids, top_logits, teacher_lse, loss_mask)
    else:
        _check_tensor(out[0], "loss", _torch.float32, (T,))
        _check_tensor(out[1], "lse", _torch.float32, (T,))
        dev = _one_device(logits, top_ids, top_logits, teacher_lse, loss_mask, *out)
    rc = _call(library().lmhead_distill_logits_fwd, dev, stream, logits.data_ptr(), kind, ld,
               top_ids.data_ptr(), top_logits.data_ptr(), _ptr(teacher_lse), _ptr(loss_mask), T, V,
               K, temperature, teacher_temperature, out[0].data_ptr(), out[1].data_ptr())
    return rc, out


def lmhead_distill_logits_fwd(logits, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                              teacher_temperature, loss, lse, stream=None):
    """C ``lmhead_distill_logits_fwd`` on torch tensors; returns the status code."""
    return _distill_logits_fwd(logits, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                               teacher_temperature, (loss, lse), stream)[0]


def lmhead_distill_logits_bwd(logits, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                              teacher_temperature, grad_loss, lse, d_logits, stream=None):
    """C ``lmhead_distill_logits_bwd`` on torch tensors; returns the status code."""
    T, V = logits.shape
    kind, ld = _check_rows(logits, "logits", (T, V))
    K = _check_teacher(top_ids, top_logits, teacher_lse, loss_mask, T)
    _check_tensor(grad_loss, "grad_loss", _torch.float32, (T,))
    _check_tensor(lse, "lse", _torch.float32, (T,))
    _, d_ld = _check_rows(d_logits, "d_logits", (T, V), (logits.dtype,))
    dev = _one_device(logits, top_ids, top_logits, teacher_lse, loss_mask, grad_loss, lse, d_logits)
    return _call(library().lmhead_distill_logits_bwd, dev, stream, logits.data_ptr(), kind, ld,
                 top_ids.data_ptr(), top_logits.data_ptr(), _ptr(teacher_lse), _ptr(loss_mask), T,
                 V, K, temperature, teacher_temperature, grad_loss.data_ptr(), lse.data_ptr(),
                 d_logits.data_ptr(), d_ld)


@functools.lru_cache(maxsize=128)   # a model has few sizes; packed rows have one per length
def lmhead_layernorm_workspace_size(N, H):
    return int(library().lmhead_layernorm_workspace_size(N, H))


def _check_norm_params(x, weight, bias, H):
    if weight is None or (weight.dtype is not _torch.float32 and weight.dtype is not x.dtype):
        raise TypeError("weight must be torch.float32 or %s" % x.dtype)
    _check_tensor(weight, "weight", weight.dtype, (H,))
    _check_tensor(bias, "bias", weight.dtype, (H,), allow_none=True)
    return _types[weight.dtype]


def _layernorm_fwd(x, weight, bias, eps, out, out_dtype, stream):
    N, H = x.shape
    x_type, x_ld = _check_rows(x, "x", (N, H))
    param_type = _check_norm_params(x, weight, bias, H)
    torch = _torch
    if out is None:
        where = x.device
        y = torch.empty((N, H), dtype=x.dtype if out_dtype is None else out_dtype, device=where)
        mean = torch.empty(N, dtype=torch.float32, device=where)
        rstd = torch.empty(N, dtype=torch.float32, device=where)
        dev = _one_device(x, weight, bias)
    else:
        y, mean, rstd = out
        _check_tensor(mean, "mean", torch.float32, (N,), allow_none=True)
        _check_tensor(rstd, "rstd", torch.float32, (N,), allow_none=True)
        dev = _one_device(x, weight, bias, y, mean, rstd)
    y_type, y_ld = _check_rows(y, "y", (N, H), (x.dtype, torch.bfloat16)
                               if x_type == LMHEAD_F32 else (x.dtype,))
    rc = _call(library().lmhead_layernorm_fwd, dev, stream, x.data_ptr(), x_type, x_ld,
               weight.data_ptr(), _ptr(bias), param_type, N, H, eps, y.data_ptr(), y_type, y_ld,
               _ptr(mean), _ptr(rstd))
    return rc, (y, mean, rstd)


def lmhead_layernorm_fwd(x, weight, bias, eps, y, mean, rstd, stream=None):
    """C ``lmhead_layernorm_fwd`` on torch tensors; returns the status code."""
    return _layernorm_fwd(x, weight, bias, eps, (y, mean, rstd), None, stream)[0]


def _layernorm_bwd(dy, x, weight, mean, rstd, out, with_bias, accumulate, workspace, stream):
    """out: (dx, d_weight, d_bias), or None for new ones; then workspace may be None too."""
    N, H = x.shape
    x_type, x_ld = _check_rows(x, "x", (N, H))
    f32 = _torch.float32
    dy_type, dy_ld = _check_rows(dy, "dy", (N, H), (f32, _torch.bfloat16)
                                 if x_type == LMHEAD_F32 else (f32, x.dtype))
    param_type = _check_norm_params(x, weight, None, H)
    _check_tensor(mean, "mean", f32, (N,))
    _check_tensor(rstd, "rstd", f32, (N,))
    if out is None:
        empty, where = _torch.empty, x.device
        dx, dx_ld = empty((N, H), dtype=x.dtype, device=where), H
        d_weight = empty(H, dtype=f32, device=where)
        d_bias = empty(H, dtype=f32, device=where) if with_bias else None
        if workspace is None:
            workspace = empty(lmhead_layernorm_workspace_size(N, H), dtype=_torch.uint8,
                              device=where)
        else:
            _check_workspace(workspace)
        dev = _one_device(x, dy, weight, mean, rstd, workspace)
    else:
        dx, d_weight, d_bias = out
        dx_ld = 0 if dx is None else _check_rows(dx, "dx", (N, H), (x.dtype,))[1]
        _check_tensor(d_weight, "d_weight", f32, (H,), allow_none=True)
        _check_tensor(d_bias, "d_bias", f32, (H,), allow_none=True)
        if workspace is not None or d_weight is not None or d_bias is not None:
            _check_workspace(workspace)
        dev = _one_device(x, dy, weight, mean, rstd, dx, d_weight, d_bias, workspace)
    rc = _call(library().lmhead_layernorm_bwd, dev, stream, dy.data_ptr(), dy_type, dy_ld,
               x.data_ptr(), x_type, x_ld, weight.data_ptr(), param_type, mean.data_ptr(),
               rstd.data_ptr(), N, H, _ptr(dx), dx_ld, _ptr(d_weight), _ptr(d_bias),
               1 if accumulate else 0, _ptr(workspace),
               0 if workspace is None else workspace.nbytes)
    return rc, (dx, d_weight, d_bias)


def lmhead_layernorm_bwd(dy, x, weight, mean, rstd, dx, d_weight, d_bias, accumulate, workspace,
                         stream=None):
    """C ``lmhead_layernorm_bwd`` on torch tensors; returns the status code."""
    return _layernorm_bwd(dy, x, weight, mean, rstd, (dx, d_weight, d_bias), True, accumulate,
                          workspace, stream)[0]


def _check_rules(R, V, tokens, spans, repetition, frequency, presence, allowed, allowed_rows):
    f32, i32 = _torch.float32, _torch.int32
    if tokens is not None:
        _check_tensor(tokens, "tokens", i32, (tokens.numel(),))
    _check_tensor(spans, "spans", _torch.int64, (R, 3), allow_none=True)
    _check_tensor(repetition, "repetition", f32, (R,), allow_none=True)
    _check_tensor(frequency, "frequency", f32, (R,), allow_none=True)
    _check_tensor(presence, "presence", f32, (R,), allow_none=True)
    if allowed is not None:
        _check_tensor(allowed, "allowed", i32, (allowed.shape[0], (V + 31) // 32))
    _check_tensor(allowed_rows, "allowed_rows", i32, (R,), allow_none=True)


def lmhead_process_logits_fwd(logits, tokens, spans, repetition, frequency, presence,
                              bias_offsets, bias_ids, bias_values, allowed, allowed_rows, out,
                              stream=None):
    """C ``lmhead_process_logits_fwd`` on torch tensors; returns the status code."""
    R, V = logits.shape
    kind, ld = _check_rows(logits, "logits", (R, V))
    _check_rules(R, V, tokens, spans, repetition, frequency, presence, allowed, allowed_rows)
    _check_tensor(bias_offsets, "bias_offsets", _torch.int64, (R + 1,), allow_none=True)
    n_bias = 0 if bias_ids is None else bias_ids.numel()
    _check_tensor(bias_ids, "bias_ids", _torch.int32, (n_bias,), allow_none=bias_offsets is None)
    _check_tensor(bias_values, "bias_values", _torch.float32, (n_bias,),
                  allow_none=bias_offsets is None)
    _, out_ld = _check_rows(out, "out", (R, V), (logits.dtype,))
    dev = _one_device(logits, tokens, spans, repetition, frequency, presence, bias_offsets,
                      bias_ids, bias_values, allowed, allowed_rows, out)
    return _call(library().lmhead_process_logits_fwd, dev, stream, logits.data_ptr(), kind, ld, R,
                 V, _ptr(tokens), 0 if tokens is None else tokens.numel(), _ptr(spans),
                 _ptr(repetition), _ptr(frequency), _ptr(presence), _ptr(bias_offsets),
                 _ptr(bias_ids), _ptr(bias_values), n_bias, _ptr(allowed),
                 0 if allowed is None else allowed.shape[0], _ptr(allowed_rows), out.data_ptr(),
                 out_ld)


def lmhead_process_logits_bwd(grad_out, logits, tokens, spans, repetition, allowed, allowed_rows,
                              d_logits, stream=None):
    """C ``lmhead_process_logits_bwd`` on torch tensors; returns the status code."""
    R, V = logits.shape
    kind, ld = _check_rows(logits, "logits", (R, V))
    _, grad_ld = _check_rows(grad_out, "grad_out", (R, V), (logits.dtype,))
    _check_rules(R, V, tokens, spans, repetition, None, None, allowed, allowed_rows)
    _, d_ld = _check_rows(d_logits, "d_logits", (R, V), (logits.dtype,))
    dev = _one_device(logits, grad_out, tokens, spans, repetition, allowed, allowed_rows, d_logits)
    return _call(library().lmhead_process_logits_bwd, dev, stream, grad_out.data_ptr(), grad_ld,
                 logits.data_ptr(), kind, ld, R, V, _ptr(tokens),
                 0 if tokens is None else tokens.numel(), _ptr(spans), _ptr(repetition),
                 _ptr(allowed), 0 if allowed is None else allowed.shape[0], _ptr(allowed_rows),
                 d_logits.data_ptr(), d_ld)


def lmhead_selftest_bounded_wait(workspace, limit_ms, stream=None):
    """C ``lmhead_selftest_bounded_wait``; returns the status code of the launch."""
    _check_workspace(workspace)
    return _on_device([workspace], stream, lambda: int(library().lmhead_selftest_bounded_wait(
        _ptr(workspace), workspace.numel() * workspace.element_size(), int(limit_ms),
        _stream(stream))))


def lmhead_read_device_status(workspace, stream=None):
    _check_workspace(workspace)
    return _on_device([workspace], stream, lambda: int(
        library().lmhead_read_device_status(_ptr(workspace), _stream(stream))))


def lmhead_read_scored_count(workspace, stream=None):
    _check_workspace(workspace)
    return _on_device([workspace], stream, lambda: int(
        library().lmhead_read_scored_count(_ptr(workspace), _stream(stream))))


def lmhead_status_string(status):
    return library().lmhead_status_string(int(status)).decode()


def lmhead_plan_info(T, H, V, chunk_size):
    """(fwd_splits, bwd_tokens, bwd_vocab) for these sizes on the current device."""
    a, b, c = _I32(), _I32(), _I32()
    rc = library().lmhead_plan_info(T, H, V, chunk_size, ctypes.byref(a), ctypes.byref(b),
                                    ctypes.byref(c))
    if rc:
        raise LmheadError(rc, "lmhead_plan_info")
    return a.value, b.value, c.value


def lmhead_profile_enable(on):
    library().lmhead_profile_enable(int(bool(on)))


def lmhead_profile_count():
    return int(library().lmhead_profile_count())


def lmhead_profile_record(i):
    """(kernel name, milliseconds) of the i-th recorded launch."""
    name = ctypes.c_char_p()
    ms = ctypes.c_float()
    rc = library().lmhead_profile_record(i, ctypes.byref(name), ctypes.byref(ms))
    if rc:
        raise LmheadError(rc, "lmhead_profile_record")
    return name.value.decode(), float(ms.value)


def lmhead_launch_count():
    return int(library().lmhead_launch_count())


# ----------------------------------------------------------------- conveniences
def _workspace(op, T, H, V, chunk_size, device):
    import torch
    n = lmhead_workspace_size(op, T, H, V, chunk_size)
    if n == 0:
        raise LmheadError(1, "lmhead_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward(hidden, weight, targets, loss_mask=None, temperature=1.0, chunk_size=512,
            with_entropy=True, workspace=None, stream=None):
    """Returns (logp, entropy or None, lse) as fp32 CUDA tensors."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    logp = torch.empty(T, dtype=torch.float32, device=dev)
    ent = torch.empty(T, dtype=torch.float32, device=dev) if with_entropy else None
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(LMHEAD_OP_FWD, T, H, V, chunk_size, dev)
    rc = lmhead_logps_fwd(hidden, weight, targets, loss_mask, temperature, chunk_size, logp, ent,
                          lse, workspace, stream)
    if rc:
        raise LmheadError(rc, "lmhead_logps_fwd")
    return logp, ent, lse


def backward(hidden, weight, targets, loss_mask, temperature, chunk_size, grad_logp,
             grad_entropy, lse, entropy=None, d_weight=None, accumulate_dweight=False,
             workspace=None, stream=None):
    """Returns (d_hidden [T,H] fp32, d_weight [V,H] fp32)."""
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    d_hidden = torch.empty((T, H), dtype=torch.float32, device=dev)
    if d_weight is None:
        d_weight = torch.empty((V, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(LMHEAD_OP_BWD, T, H, V, chunk_size, dev)
    rc = lmhead_logps_bwd(hidden, weight, targets, loss_mask, temperature, chunk_size, grad_logp,
                          grad_entropy, lse, entropy, d_hidden, d_weight, accumulate_dweight,
                          workspace, stream)
    if rc:
        raise LmheadError(rc, "lmhead_logps_bwd")
    return d_hidden, d_weight


def _made_on(stream, first, fn, *args):
    """fn(*args) with `stream` current, so that what it allocates belongs to that stream: memory
    of another one could still be in use there, or be handed out again before the call is done."""
    if _torch is None:
        _bind_torch()
    cuda = _torch.cuda
    if isinstance(stream, int):
        stream = (cuda.ExternalStream(stream, device=first.device) if stream
                  else cuda.default_stream(first.device))
    if first.device != stream.device:
        raise ValueError("all tensors and the stream of one call must be on one CUDA device, "
                         "got %s" % sorted({str(first.device), str(stream.device)}))
    with cuda.stream(stream):
        return fn(*args)


def _distill_workspace(op, T, H, V, K, chunk_size, device):
    import torch
    n = lmhead_distill_workspace_size(op, T, H, V, K, chunk_size)
    if n == 0:
        raise LmheadError(1, "lmhead_distill_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def distill_forward(hidden, weight, top_ids, top_logits, loss_mask=None, temperature=1.0,
                    teacher_temperature=1.0, chunk_size=512, teacher_lse=None, workspace=None,
                    stream=None):
    """Distillation loss through the head.  Returns (loss [T], lse [T], z_top [T, K]), fp32;
    keep lse and z_top for ``distill_backward``."""
    if stream is not None:
        return _made_on(stream, hidden, distill_forward, hidden, weight, top_ids, top_logits,
                        loss_mask, temperature, teacher_temperature, chunk_size, teacher_lse,
                        workspace)
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    K = top_ids.shape[1]
    dev = hidden.device
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    z_top = torch.empty((T, K), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _distill_workspace(LMHEAD_OP_FWD, T, H, V, K, chunk_size, dev)
    rc = lmhead_distill_fwd(hidden, weight, top_ids, top_logits, teacher_lse, loss_mask,
                            temperature, teacher_temperature, chunk_size, loss, lse, z_top,
                            workspace)
    if rc:
        raise LmheadError(rc, "lmhead_distill_fwd")
    return loss, lse, z_top


def distill_backward(hidden, weight, top_ids, top_logits, loss_mask, temperature,
                     teacher_temperature, chunk_size, grad_loss, lse, z_top, teacher_lse=None,
                     d_weight=None, accumulate_dweight=False, workspace=None, stream=None):
    """Returns (d_hidden [T, H] fp32, d_weight [V, H] fp32)."""
    if stream is not None:
        return _made_on(stream, hidden, distill_backward, hidden, weight, top_ids, top_logits,
                        loss_mask, temperature, teacher_temperature, chunk_size, grad_loss, lse,
                        z_top, teacher_lse, d_weight, accumulate_dweight, workspace)
    import torch
    T, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    d_hidden = torch.empty((T, H), dtype=torch.float32, device=dev)
    if d_weight is None:
        make = torch.zeros if accumulate_dweight else torch.empty
        d_weight = make((V, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _distill_workspace(LMHEAD_OP_BWD, T, H, V, top_ids.shape[1], chunk_size, dev)
    rc = lmhead_distill_bwd(hidden, weight, top_ids, top_logits, teacher_lse, loss_mask,
                            temperature, teacher_temperature, chunk_size, grad_loss, lse, z_top,
                            d_hidden, d_weight, accumulate_dweight, workspace)
    if rc:
        raise LmheadError(rc, "lmhead_distill_bwd")
    return d_hidden, d_weight


_MOST_PADDING = 256   # elements between rows that a new result repeats


def _rows_like(t):
    """A new matrix for a result beside t: its rows as far apart as t's where those are padded (a
    table rounded up), else just far enough to have the same 16-byte alignment as t's (rows taken
    out of a larger tensor must not cost its size again)."""
    if _torch is None:
        _bind_torch()
    rows, cols = t.shape
    gap = max(t.stride(0) - cols, 0)
    if gap > _MOST_PADDING:
        gap %= 16 // t.element_size()
    return _torch.empty_strided((rows, cols), (cols + gap, 1), dtype=t.dtype, device=t.device)


def distill_logits_forward(logits, top_ids, top_logits, loss_mask=None, temperature=1.0,
                           teacher_temperature=1.0, teacher_lse=None, stream=None):
    """Distillation loss on held logits [T, V] (fp32, bf16 or fp16, rows may be padded).
    Returns (loss [T], lse [T]), fp32."""
    if stream is not None:
        return _made_on(stream, logits, distill_logits_forward, logits, top_ids, top_logits,
                        loss_mask, temperature, teacher_temperature, teacher_lse)
    rc, out = _distill_logits_fwd(logits, top_ids, top_logits, teacher_lse, loss_mask, temperature,
                                  teacher_temperature, None, None)
    if rc:
        raise LmheadError(rc, "lmhead_distill_logits_fwd")
    return out


def distill_logits_backward(logits, top_ids, top_logits, loss_mask, temperature,
                            teacher_temperature, grad_loss, lse, teacher_lse=None, d_logits=None,
                            stream=None):
    """Returns d_logits [T, V] of the logits' type, padded like the logits
    (``d_logits=logits`` overwrites them)."""
    if stream is not None:
        return _made_on(stream, logits, distill_logits_backward, logits, top_ids, top_logits,
                        loss_mask, temperature, teacher_temperature, grad_loss, lse, teacher_lse,
                        d_logits)
    if d_logits is None:
        d_logits = _rows_like(logits)
    rc = lmhead_distill_logits_bwd(logits, top_ids, top_logits, teacher_lse, loss_mask,
                                   temperature, teacher_temperature, grad_loss, lse, d_logits)
    if rc:
        raise LmheadError(rc, "lmhead_distill_logits_bwd")
    return d_logits


def layernorm_forward(x, weight, bias=None, eps=1e-5, out_dtype=None, stream=None):
    """Layer norm of x [N, H].  Returns (y [N, H] of x's type or out_dtype, mean [N] fp32,
    rstd [N] fp32)."""
    if stream is not None:
        return _made_on(stream, x, layernorm_forward, x, weight, bias, eps, out_dtype)
    rc, out = _layernorm_fwd(x, weight, bias, eps, None, out_dtype, None)
    if rc:
        raise LmheadError(rc, "lmhead_layernorm_fwd")
    return out


def layernorm_backward(dy, x, weight, mean, rstd, with_bias=True, d_weight=None, d_bias=None,
                       accumulate=False, dx=None, workspace=None, stream=None):
    """Returns (dx [N, H] of x's type, d_weight [H] fp32, d_bias [H] fp32 or None)."""
    if stream is not None:
        return _made_on(stream, dy, layernorm_backward, dy, x, weight, mean, rstd, with_bias,
                        d_weight, d_bias, accumulate, dx, workspace)
    if dx is None and d_weight is None and d_bias is None and not accumulate:
        out = None
    else:
        import torch
        N, H = x.shape
        new = dict(dtype=torch.float32, device=x.device)
        dx = torch.empty((N, H), dtype=x.dtype, device=x.device) if dx is None else dx
        make = torch.zeros if accumulate else torch.empty
        d_weight = make(H, **new) if d_weight is None else d_weight
        d_bias = make(H, **new) if d_bias is None and with_bias else d_bias
        out = dx, d_weight, d_bias
        if workspace is None:
            workspace = torch.empty(lmhead_layernorm_workspace_size(N, H), dtype=torch.uint8,
                                    device=x.device)
    rc, out = _layernorm_bwd(dy, x, weight, mean, rstd, out, with_bias, accumulate, workspace,
                             None)
    if rc:
        raise LmheadError(rc, "lmhead_layernorm_bwd")
    return out


def process_logits(logits, tokens=None, spans=None, repetition=None, frequency=None,
                   presence=None, bias_offsets=None, bias_ids=None, bias_values=None,
                   allowed=None, allowed_rows=None, out=None, stream=None):
    """Penalties, biases and a grammar mask on logits [R, V]; returns the processed logits, padded
    like the logits (``out=logits`` processes them in place)."""
    if stream is not None:
        return _made_on(stream, logits, process_logits, logits, tokens, spans, repetition,
                        frequency, presence, bias_offsets, bias_ids, bias_values, allowed,
                        allowed_rows, out)
    if out is None:
        out = _rows_like(logits)
    rc = lmhead_process_logits_fwd(logits, tokens, spans, repetition, frequency, presence,
                                   bias_offsets, bias_ids, bias_values, allowed, allowed_rows,
                                   out)
    if rc:
        raise LmheadError(rc, "lmhead_process_logits_fwd")
    return out


def process_logits_backward(grad_out, logits, tokens=None, spans=None, repetition=None,
                            allowed=None, allowed_rows=None, d_logits=None, stream=None):
    """Cotangent of the original logits, padded like grad_out (``d_logits=grad_out``
    overwrites it)."""
    if stream is not None:
        return _made_on(stream, grad_out, process_logits_backward, grad_out, logits, tokens, spans,
                        repetition, allowed, allowed_rows, d_logits)
    if d_logits is None:
        d_logits = _rows_like(grad_out)
    rc = lmhead_process_logits_bwd(grad_out, logits, tokens, spans, repetition, allowed,
                                   allowed_rows, d_logits)
    if rc:
        raise LmheadError(rc, "lmhead_process_logits_bwd")
    return d_logits
