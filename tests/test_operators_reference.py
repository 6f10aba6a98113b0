"""The 64-bit gradients that the GPU tests compare with, against central
differences of the 64-bit forward definitions (CPU only).

A central difference with step h is off by h^2 f''' / 6 and by 2^-52 |f| / h;
with h = 1e-5 and values of order 10 both are below 1e-9, so 1e-7 of the
largest gradient is far above either."""
import numpy as np

import operators_reference as ref

H = 1e-5


def _differences(f, x):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += H
        down[i] -= H
        d[i] = (f(up) - f(down)) / (2 * H)
    return d


def _close(a, b):
    assert np.abs(a - b).max() <= 1e-7 * max(1.0, np.abs(b).max())


def test_norm_gradient():
    r = np.random.default_rng(1)
    x, w, b, g = r.normal(size=(3, 7)) + 0.5, r.normal(size=7), r.normal(size=7), r.normal(size=(3, 7))
    _, mean, rstd = ref.norm_fwd(x, w, b, 1e-5)
    dx, dw, db = ref.norm_bwd(g, x, w, mean, rstd)
    _close(dx, _differences(lambda v: (ref.norm_fwd(v, w, b, 1e-5)[0] * g).sum(), x))
    _close(dw, _differences(lambda v: (ref.norm_fwd(x, v, b, 1e-5)[0] * g).sum(), w))
    _close(db, _differences(lambda v: (ref.norm_fwd(x, w, v, 1e-5)[0] * g).sum(), b))


def test_distill_gradient():
    r = np.random.default_rng(2)
    z, a, g = r.normal(size=(4, 9)) * 2, r.normal(size=(4, 3)) * 2, r.normal(size=4)
    ids = np.array([[0, 3, 8], [-1, 2, 2], [5, 4, 1], [7, 6, 0]])
    a[2, 1] = -np.inf
    a[3] = -np.inf
    for lse in (None, r.normal(size=4) + 4.0):
        loss = lambda v: (ref.distill_fwd(v, ids, a, 0.7, lse)[0] * g).sum()   # noqa: E731
        dz = ref.distill_dz(z, ref.log_sum_exp(z), ids, a, g, 0.7, lse)
        _close(dz, _differences(loss, z))
        assert (dz[3] == 0).all()


def test_process_gradient():
    r = np.random.default_rng(3)
    x, g = r.normal(size=(3, 40)), r.normal(size=(3, 40))
    x[np.abs(x) < 0.01] = 0.5   # a difference must not step over the kink at 0
    rules = dict(tokens=r.integers(-1, 42, size=30), spans=np.array([[0, 5, 12], [3, 3, 30], [9, 9, 9]]),
                 repetition=np.array([1.3, 0.8, 2.0]),
                 allowed=r.integers(-2 ** 31, 2 ** 31, size=(2, 2)), allowed_rows=np.array([1, -1, 0]))

    def f(v):
        y = ref.process_fwd(v, frequency=np.full(3, 0.2), presence=np.full(3, 0.3), **rules)
        return np.where(np.isfinite(y), y * g, 0.0).sum()
    _close(ref.process_bwd(g, x, **rules), _differences(f, x))
