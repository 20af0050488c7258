"""How far the row losses may be off, from the arithmetic of a float32 kernel.

u = 2^-24 is half a step of float32.  For a column with x = |y - max y|:

  exponential   its argument is rounded where it is formed (x u, and x u for
                the rounded log2(e) factor), the hardware's exp2 is good to one
                step (2 u): relative (2 x + 4) u
  sum Z         float32 within a thread, at most C / 64 terms each, then joined
                over 10 levels: relative (C / 64 + 16) u beyond the terms' own
                errors, which count by their share
  logp, lse     the sum's relative error, plus rounding to float32 at the end
  gradient      the coefficient's and the probability's errors, then one
                rounding to the output type: half a step, eps / 2, and half the
                smallest number for float16

Everything below is these figures applied to the values of a case.
"""

import numpy as np
import torch

U = 2.0 ** -24
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}


def row_bounds(z, scale):
    """(q, logq, relative error of q per column, error of ln Z per row)."""
    y = np.asarray(z, dtype=np.float64) * scale
    with np.errstate(invalid="ignore"):
        x = y.max(1, keepdims=True) - y
    q = np.exp(-x)
    total = q.sum(1, keepdims=True)
    q = q / total
    logq = -x - np.log(total)
    x = np.where(np.isfinite(x), np.minimum(x, 200.0), 200.0)
    ln_z = U * (2 * (q * x).sum(1) + 4 + z.shape[1] / 64 + 16)
    return q, logq, U * (2 * x + 6) + ln_z[:, None], ln_z


def logp_bound(logp, ln_z, x_t):
    return ln_z + U * (2 * np.abs(logp) + 2 * x_t + 4)


def rounded(g, tol, dtype):
    """Error of a value near g, off by tol, after its rounding to dtype."""
    half = torch.finfo(dtype).eps / 2
    return tol + half * (np.abs(g) + tol) + TINY[dtype]


def grad_bound(coef, coef_off, onehot, q, q_rel, dtype):
    """Bound for coef (onehot - q); coef [R], its absolute error coef_off [R]."""
    k, dk = np.abs(coef)[:, None], coef_off[:, None]
    g = np.abs(coef)[:, None] * np.abs(onehot - q)
    # the target's entry is formed as k - k q, so q's error and two roundings of k
    tol = k * q * (q_rel + 4 * U) + dk * np.abs(onehot - q) + k * onehot * 3 * U
    return rounded(g, tol, dtype)
