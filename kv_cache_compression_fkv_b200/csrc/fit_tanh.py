"""Fits the two forms of tanh in the bf16 kernels' capped scores (paged_common.cuh).

tanh_parts: tanh(y) = y P(u) / Q(u), u = y^2, P of degree 4 and Q of degree 3, minimising the
maximum relative error on |y| <= 8 by differential correction: with the last
quotient's error t and denominator Q_k, the linear program

    minimise d  s.t.  |P - f Q| - t f Q <= d f Q_k,   f = tanh(y) / y

on Chebyshev points, until t no longer falls.  tanh_small: tanh(y) = y (1 + u S(u)),
S of degree 3, the same on |y| <= 1/2, one linear program.

    python kv_cache_compression_fkv_b200/csrc/fit_tanh.py

prints the coefficients (float32) and the error, in units of 2^-24, of both evaluated
in float32.
"""
import numpy as np
from numpy.polynomial import Chebyshev, Polynomial
from numpy.polynomial.chebyshev import chebvander
from scipy.optimize import linprog

LIMIT, DEG_P, DEG_Q = 8.0, 4, 3
SMALL, TERMS = 0.5, 4


def fit(limit=LIMIT, m=DEG_P, n=DEG_Q, points=1500):
    y = limit * (1 + np.cos(np.pi * (np.arange(points) + 0.5) / points)) / 2
    y = y[y > 1e-3]
    u, f = y * y, np.tanh(y) / y
    V = chebvander(2 * u / limit ** 2 - 1, max(m, n))
    VP, VQ = V[:, :m + 1], V[:, :n + 1]
    qk, t, best = 1 + 0.4 * u, 1.0, None
    for step in range(25):
        A = np.vstack([np.hstack([VP / f[:, None], -VQ * (1 + t), -qk[:, None]]) / qk[:, None],
                       np.hstack([-VP / f[:, None], VQ * (1 - t), -qk[:, None]]) / qk[:, None]])
        res = linprog(np.r_[np.zeros(m + n + 2), 1.0], A_ub=A, b_ub=np.zeros(len(A)),
                      bounds=[(None, None)] * (m + 1) + [(-1, 1)] * (n + 1) + [(None, None)], method="highs")
        if res.status != 0:
            break
        p, q = VP @ res.x[:m + 1], VQ @ res.x[m + 1:m + n + 2]
        e = np.max(np.abs(p / q / f - 1))
        if best is None or e < best[0]:
            best = (e, res.x[:m + 1], res.x[m + 1:m + n + 2])
        if step > 3 and e >= 0.999 * t:
            break
        t, qk = e, q
    e, p, q = best
    P, Q = (Chebyshev(c, domain=[0, limit ** 2]).convert(kind=Polynomial).coef for c in (p, q))
    return P / Q[0], Q / Q[0], e


def fit_small(limit=SMALL, terms=TERMS, grid=8001):
    x = np.linspace(0.0, 1.0, grid)[1:]  # u / limit^2
    y = limit * np.sqrt(x)
    f = np.tanh(y) / y
    # unknowns: scaled c1 .. c_terms, 1e6 t; minimise t s.t. |(1 + sum c_k x^k) / f - 1| <= t
    A = 1e6 * np.stack([x ** k / f for k in range(1, terms + 1)], axis=1)
    b = 1e6 * (1.0 - 1.0 / f)
    ones = np.ones((len(x), 1))
    res = linprog(np.r_[np.zeros(terms), 1.0], A_ub=np.vstack([np.hstack([A, -ones]), np.hstack([-A, -ones])]),
                  b_ub=np.r_[b, -b], bounds=[(None, None)] * (terms + 1), method="highs")
    return res.x[:terms] / limit ** (2.0 * np.arange(1, terms + 1)), res.x[-1] / 1e6


def horner32(c, u):
    r = np.full_like(u, np.float32(c[-1]))
    for k in c[-2::-1]:
        r = (r.astype(np.float64) * u + np.float32(k)).astype(np.float32)
    return r


def tanh32(P, Q, y, limit=LIMIT):
    """The quotient as the kernels form it: float32, fused products and sums."""
    y = np.clip(y.astype(np.float32), np.float32(-limit), np.float32(limit))
    u = y * y
    return (y * horner32(P, u)) / horner32(Q, u)


def small32(S, y):
    y = y.astype(np.float32)
    u = y * y
    return ((y * u).astype(np.float64) * horner32(S, u) + y).astype(np.float32)


if __name__ == "__main__":
    P, Q, e = fit()
    print("P:", ", ".join(f"{float(c):.9e}f" for c in P.astype(np.float32)))
    print("Q:", ", ".join(f"{float(c):.9e}f" for c in Q.astype(np.float32)))
    y = np.concatenate([np.logspace(-9, -1, 20000), np.linspace(0.1, 12, 400000)]).astype(np.float32)
    err = np.max(np.abs(tanh32(P, Q, y) / np.tanh(y.astype(np.float64)) - 1))
    print(f"error of the fit {e:.2e}, in float32 {err * 2 ** 24:.1f} of 2^-24")
    S, e = fit_small()
    print("S:", ", ".join(f"{float(c):.9e}f" for c in S.astype(np.float32)))
    y = y[y <= SMALL]
    err = np.max(np.abs(small32(S, y) / np.tanh(y.astype(np.float64)) - 1))
    print(f"error of the fit {e:.2e}, in float32 {err * 2 ** 24:.1f} of 2^-24")
