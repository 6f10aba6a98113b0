"""64-bit definitions of layer norm, distillation and logit processing, in
plain numpy, and the rounding units the tests' tolerances are made of."""
import numpy as np

# Unit roundoff: the largest relative error of one rounding to nearest.
U32, UBF16, UF16 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
UNIT = {"float32": U32, "bfloat16": UBF16, "float16": UF16}
TINY = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -25}   # underflow


def f64(t):
    """A tensor as a 64-bit array."""
    return None if t is None else t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ layer norm
def norm_fwd(x, w, b, eps):
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def norm_bwd(dy, x, w, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    h = dy * w
    dx = (h - h.mean(1, keepdims=True) - xh * (h * xh).mean(1, keepdims=True)) * rstd[:, None]
    return dx, (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------------ distillation
def teacher(a, tau, lse):
    """p [T, K] and log p (-inf where absent)."""
    present = ~np.isneginf(a)
    z = a / tau
    if lse is None:
        with np.errstate(all="ignore"):
            m = np.max(z, axis=1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    with np.errstate(all="ignore"):
        logp = np.where(present, z - lse[:, None], -np.inf)
        return np.where(present, np.exp(logp), 0.0), logp


def log_sum_exp(z):
    with np.errstate(all="ignore"):
        m = np.max(z, axis=1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        out = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    out[np.isnan(z).any(1) | np.isposinf(z).any(1)] = np.nan
    return out


def wrap(ids, V):
    ids = np.where(ids < 0, ids + V, ids)
    return np.where((ids >= 0) & (ids < V), ids, -1)


def distill_fwd(z, ids, a, tau_t=1.0, teacher_lse=None, mask=None):
    """z is already divided by the temperature.  (loss, lse, z_top)."""
    T, V = z.shape
    p, logp = teacher(a, tau_t, teacher_lse)
    lse = log_sum_exp(z)
    at = wrap(ids, V)
    zt = np.take_along_axis(z, np.maximum(at, 0), 1)
    zt = np.where(np.isneginf(logp), 0.0, np.where(at < 0, np.nan, zt))
    with np.errstate(all="ignore"):
        term = np.where((p == 0) & ~np.isnan(zt), 0.0, p * (logp - zt + lse[:, None]))
        loss = np.where(p.sum(1) == 0, 0.0, term.sum(1))
    if mask is not None:
        on = mask != 0
        loss, lse, zt = np.where(on, loss, 0.0), np.where(on, lse, 0.0), np.where(on[:, None], zt, 0.0)
    return loss, lse, zt


def distill_dz(z, lse, ids, a, grad, tau_t=1.0, teacher_lse=None, mask=None):
    """Cotangent of z."""
    T, V = z.shape
    p, logp = teacher(a, tau_t, teacher_lse)
    P = p.sum(1)
    with np.errstate(all="ignore"):
        dz = (grad * P)[:, None] * np.exp(z - lse[:, None])
    at = wrap(ids, V)
    for t in range(T):
        for k in range(ids.shape[1]):
            if at[t, k] >= 0 and not np.isneginf(logp[t, k]):
                dz[t, at[t, k]] -= grad[t] * p[t, k]
    dz[~np.isfinite(z)] = 0.0
    dz[P == 0] = 0.0
    if mask is not None:
        dz[mask == 0] = 0.0
    return dz


# ------------------------------------------------------------------ logit processing
def history(tokens, spans, R, V):
    """met [R, V] bool and output counts [R, V]."""
    met, count = np.zeros((R, V), bool), np.zeros((R, V))
    if tokens is None:
        return met, count
    n = len(tokens)
    for r in range(R):
        b = min(max(int(spans[r, 0]), 0), n)
        m = min(max(int(spans[r, 1]), b), n)
        e = min(max(int(spans[r, 2]), m), n)
        for i in range(b, e):
            v = int(tokens[i])
            if 0 <= v < V:
                met[r, v] = True
                count[r, v] += i >= m
    return met, count


def allowed_bits(allowed, rows, R, V):
    on = np.ones((R, V), bool)
    if allowed is None:
        return on
    v = np.arange(V)
    for r in range(R):
        m = r if rows is None else int(rows[r])
        if 0 <= m < len(allowed):
            on[r] = (allowed[m].astype(np.int64)[v // 32] >> (v % 32)) & 1
    return on


def process_fwd(x, tokens=None, spans=None, repetition=None, frequency=None, presence=None,
                bias_offsets=None, bias_ids=None, bias_values=None, allowed=None,
                allowed_rows=None):
    R, V = x.shape
    met, count = history(tokens, spans, R, V)
    rho = np.ones(R) if repetition is None else repetition
    f = np.zeros(R) if frequency is None else frequency
    p = np.zeros(R) if presence is None else presence
    out = np.where(met, np.where(x > 0, x / rho[:, None], x * rho[:, None]), x)
    out = np.where(count > 0, out - (f[:, None] * count + p[:, None]), out)
    if bias_offsets is not None:
        for r in range(R):
            last = {int(bias_ids[j]): bias_values[j]
                    for j in range(int(bias_offsets[r]), int(bias_offsets[r + 1]))}
            for v, b in last.items():
                if 0 <= v < V:
                    out[r, v] += b
    return np.where(allowed_bits(allowed, allowed_rows, R, V), out, -np.inf)


def process_bwd(g, x, tokens=None, spans=None, repetition=None, allowed=None, allowed_rows=None):
    R, V = x.shape
    met, _ = history(tokens, spans, R, V)
    rho = np.ones(R) if repetition is None else repetition
    d = np.where(met, np.where(x > 0, g / rho[:, None], g * rho[:, None]), g)
    return np.where(allowed_bits(allowed, allowed_rows, R, V), d, 0.0)
