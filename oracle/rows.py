"""Float64 CPU oracle for the losses over rows of logits.

TEST INFRASTRUCTURE ONLY (see the package docstring): imported by tests, never
by the library.

A row is C logits z; y = s z, q = softmax(y), logp = y_t - logsumexp(y).  A row
is left out (outputs and gradient 0) when its target is negative or its weight
is 0.  Everything is float64; sums of exponentials are taken relative to the
row's maximum.
"""

from __future__ import annotations

import numpy as np

SIGMOID, HINGE, SQUARE = 0, 1, 2


def _softmax(y):
    """(q, log q, log-sum-exp) of one row; columns of -inf have probability 0.
    log q is taken relative to the maximum, which may dwarf the rest."""
    m = y.max()
    e = np.exp(y - m)
    ln_sum = np.log(e.sum())
    return e / e.sum(), y - m - ln_sum, m + ln_sum


def _weights(w, n):
    return np.full(n, 1.0 / n) if w is None else np.asarray(w, dtype=np.float64)


def logprob_rows(z, targets, scale=1.0):
    """(logp [R], lse [R])."""
    z = np.asarray(z, dtype=np.float64)
    logp, lse = np.zeros(len(z)), np.zeros(len(z))
    for r, t in enumerate(targets):
        if t < 0:
            continue
        _, logq, lse[r] = _softmax(scale * z[r])
        logp[r] = logq[t] if t < z.shape[1] else np.nan
    return logp, lse


def logprob_rows_bwd(z, targets, grad_logp, scale=1.0):
    """Gradient of sum_r grad_logp[r] logp[r]."""
    z = np.asarray(z, dtype=np.float64)
    grad = np.zeros_like(z)
    for r, t in enumerate(targets):
        if t < 0 or grad_logp[r] == 0:
            continue
        grad[r] = -_softmax(scale * z[r])[0]
        if t < z.shape[1]:
            grad[r, t] += 1.0
            grad[r] *= grad_logp[r] * scale
        else:
            grad[r] = np.nan
    return grad


def distill_rows(z, idx, val, teacher_lse=None, scale=1.0, weight=None):
    """(loss, row losses [R], grad [R, C]) of the divergence from a teacher's
    listed logits."""
    z = np.asarray(z, dtype=np.float64)
    R, C = z.shape
    w = _weights(weight, R)
    losses, grad = np.zeros(R), np.zeros((R, C))
    for r in range(R):
        if w[r] == 0:
            continue
        if np.any(np.asarray(idx[r]) >= C):
            losses[r], grad[r] = np.nan, np.nan
            continue
        entries = [(int(j), scale * float(v)) for j, v in zip(idx[r], val[r]) if j >= 0]
        live = [(j, v) for j, v in entries if v > -np.inf]
        if teacher_lse is None:
            if not live:
                continue
            top = max(v for _, v in live)
            lt = top + np.log(sum(np.exp(v - top) for _, v in live))
        else:
            lt = float(teacher_lse[r])
        q, logq, _ = _softmax(scale * z[r])
        p_col = np.zeros(C)
        mass = 0.0
        for j, v in live:
            p = np.exp(v - lt)
            losses[r] += p * (v - lt - logq[j])
            p_col[j] += p
            mass += p
        rest = np.ones(C, dtype=bool)
        rest[[j for j, _ in entries]] = False
        if teacher_lse is not None and rest.any():
            p_rest, q_rest = max(0.0, 1.0 - mass), q[rest].sum()
            if p_rest > 0:
                losses[r] += p_rest * (np.log(p_rest) - np.log(q_rest))
            grad[r] = (mass + p_rest) * q - p_col - np.where(rest, p_rest * q / q_rest, 0.0)
        else:
            grad[r] = mass * q - p_col
        grad[r] *= w[r] * scale
    on = w != 0
    return float(np.sum(w[on] * losses[on])), losses, grad


def policy_rows(z, targets, old, adv, ref=None, scale=1.0, clip_low=0.2, clip_high=0.2, kl=0.0,
                weight=None):
    """(loss, row losses [R], logp [R], grad [R, C], slopes dl/dlogp [R])."""
    z = np.asarray(z, dtype=np.float64)
    R = len(z)
    w = _weights(weight, R)
    t = np.where(w == 0, -1, np.asarray(targets))
    logp, _ = logprob_rows(z, t, scale)
    losses, slopes = np.zeros(R), np.zeros(R)
    for r in range(R):
        if t[r] < 0:
            continue
        rho, a = np.exp(logp[r] - old[r]), float(adv[r])
        clipped = min(max(rho, 1 - clip_low), 1 + clip_high)
        losses[r] = -min(rho * a, clipped * a)
        inside = rho <= 1 + clip_high if a >= 0 else rho >= 1 - clip_low
        slopes[r] = -rho * a if inside or np.isnan(rho) else 0.0
        if np.isnan(rho):
            losses[r] = np.nan
        if ref is not None:
            d = ref[r] - logp[r]
            losses[r] += kl * (np.expm1(d) - d)
            slopes[r] -= kl * np.expm1(d)
    grad = logprob_rows_bwd(z, t, np.where(t >= 0, w * slopes, 0.0), scale)
    on = w != 0
    return float(np.sum(w[on] * losses[on])), losses, logp, grad, slopes


def preference_rows(z, targets, offsets, chosen, rejected, ref=None, kind=SIGMOID, beta=0.1,
                    margin=0.0, smoothing=0.0, mean=False, scale=1.0, weight=None):
    """(loss, pair losses [P], sequence log-probabilities [S], grad [R, C],
    d loss / d row log-probability [R])."""
    z = np.asarray(z, dtype=np.float64)
    R, S, P = len(z), len(offsets) - 1, len(chosen)
    t = np.asarray(targets).copy()
    t[:offsets[0]] = -1
    t[offsets[-1]:] = -1
    w = _weights(weight, P) if P else np.zeros(0)
    logp, _ = logprob_rows(z, t, scale)
    seq, count = np.zeros(S), np.ones(S)
    for s in range(S):
        part = slice(offsets[s], offsets[s + 1])
        if mean:
            count[s] = max(1, int(np.sum(t[part] >= 0)))
        seq[s] = logp[part].sum() / count[s]
    off = seq if ref is None else seq - np.asarray(ref, dtype=np.float64)
    losses, d_seq = np.zeros(P), np.zeros(S)
    for i, (c, r) in enumerate(zip(chosen, rejected)):
        if not (0 <= c < S and 0 <= r < S):
            losses[i] = np.nan
            continue
        d = off[c] - off[r]
        h = beta * d - margin
        if kind == SIGMOID:
            losses[i] = (1 - smoothing) * np.logaddexp(0, -h) + smoothing * np.logaddexp(0, h)
            up = np.exp(-np.logaddexp(0, h))           # sigmoid(-h)
            slope = beta * (smoothing * (1 - up) - (1 - smoothing) * up)
        elif kind == HINGE:
            losses[i] = 0.0 if h >= 1 else 1 - h
            slope = -beta if h < 1 else (h if np.isnan(h) else 0.0)
        else:
            losses[i] = (d - 0.5 / beta) ** 2
            slope = 2 * (d - 0.5 / beta)
        if w[i] != 0 and (c != r or np.isnan(slope)):
            d_seq[c] += w[i] * slope
            d_seq[r] -= w[i] * slope
    d_row = np.zeros(R)
    for s in range(S):
        part = slice(offsets[s], offsets[s + 1])
        d_row[part] = np.where(t[part] >= 0, d_seq[s] / count[s], 0.0)
    on = w != 0
    return (float(np.sum(w[on] * losses[on])), losses, seq,
            logprob_rows_bwd(z, t, d_row, scale), d_row)
