"""The gated linear recurrence and its gradients token by token in 64 bits (numpy), with bounds on what fp32 arithmetic
may be off.

    h_t = a_t h_{t-1} + b_t x_t

Rounding, to first order in u = 2^-24: a term of the sum h_t that entered n tokens ago has gone through n products and n
sums, in whatever order a scan groups them, and through a few more where groups are joined.  So the error is at most
E_t + 16 u M_t with E_t = |a_t| E_{t-1} + 4 u M_t, M the recurrence of the absolute values (4 where 2 would do: u_t's own
product and the second order).  The gradients' carry obeys the same from the right; products and sums over a head's
channels add theirs.
"""
import numpy as np

U = 2.0 ** -24


def widen(gate, D):
    """[T, H] or [T, H, D] gates as [T, H, D] in 64 bits."""
    g = np.asarray(gate, dtype=np.float64)
    return g if g.ndim == 3 else np.repeat(g[:, :, None], D, axis=2)


def forward(x, a, b, cu, h0=None):
    """(y, final, before, y_err, final_err, before_err): outputs, final states, the state before each token, and the bounds
    of the errors of fp32 arithmetic in each."""
    x = np.asarray(x, dtype=np.float64)
    T, H, D = x.shape
    N = len(cu) - 1
    A = widen(a, D)
    u = x if b is None else x * widen(b, D)
    y, before, ye, be = (np.zeros((T, H, D)) for _ in range(4))
    final, fe = np.zeros((N, H, D)), np.zeros((N, H, D))
    for i in range(N):
        h = np.zeros((H, D)) if h0 is None else np.asarray(h0[i], dtype=np.float64)
        m, e = np.abs(h), np.zeros((H, D))
        for t in range(cu[i], cu[i + 1]):
            before[t], be[t] = h, e + 16 * U * m
            h = A[t] * h + u[t]
            m = np.abs(A[t]) * m + np.abs(u[t])
            e = np.abs(A[t]) * e + 4 * U * m
            y[t], ye[t] = h, e + 16 * U * m
        final[i], fe[i] = h, e + (16 * U * m if cu[i + 1] > cu[i] else 0)
    return y, final, before, ye, fe, be


def backward(dy, x, a, b, cu, h0=None, d_final=None):
    """Gradients {dx, da, db, d0} and the bounds of the errors of fp32 arithmetic in each, as two dicts."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    T, H, D = x.shape
    N = len(cu) - 1
    A = widen(a, D)
    B = np.ones_like(A) if b is None else widen(b, D)
    _, _, before, _, _, be = forward(x, a, b, cu, h0)
    g, ge = np.zeros((T, H, D)), np.zeros((T, H, D))
    d0, d0e = np.zeros((N, H, D)), np.zeros((N, H, D))
    for i in range(N):
        c = np.zeros((H, D)) if d_final is None else np.asarray(d_final[i], dtype=np.float64)
        m, e = np.abs(c), np.zeros((H, D))
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            g[t] = dy[t] + c
            mg = np.abs(dy[t]) + m
            ge[t] = e + 20 * U * mg
            c = A[t] * g[t]
            m = np.abs(A[t]) * mg
            e = np.abs(A[t]) * e + 4 * U * m
        d0[i], d0e[i] = c, e + (16 * U * m if cu[i + 1] > cu[i] else 0)
    val = {"dx": B * g, "da": g * before, "db": g * x, "d0": d0}
    err = {"dx": np.abs(B) * ge + U * np.abs(B * g), "da": ge * np.abs(before) + np.abs(g) * be + ge * be + U * np.abs(g * before),
           "db": ge * np.abs(x) + U * np.abs(g * x), "d0": d0e}
    if np.ndim(a) == 2:
        for k in ("da", "db"):
            err[k] = err[k].sum(2) + D * U * np.abs(val[k]).sum(2)
            val[k] = val[k].sum(2)
    if b is None:
        val["db"] = err["db"] = None
    return val, err
