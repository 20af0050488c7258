"""Float64 CPU oracle for the paged cache in 8 bits.

TEST INFRASTRUCTURE ONLY (see the package docstring): imported by tests, never
by the library.

Codes are e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities,
0x7f and 0xff no numbers.  A number is its code times the scale of its block
and head.  Caches are lists of arrays: k codes [N, heads, block_size, dim],
v codes [N, heads, dim, block_size], scales [N, heads].
"""

from __future__ import annotations

import math

import numpy as np

SCALE_MIN, SCALE_MAX = 2.0 ** -40, 2.0 ** 40


def code_values():
    """The number of every code, 256 of them."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = -x if c & 128 else x
    out[[0x7f, 0xff]] = np.nan
    return out


VALUES = code_values()
_UP = VALUES[:127]                       # 0 .. 448, rising


def encode(x):
    """Nearest codes, ties to the even one, at most 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_UP, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up = _UP[hi] - a, a - _UP[lo]
    code = np.where(up[0] < up[1], hi, np.where(up[0] > up[1], lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(_UP[hi] == a, hi, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax):
    """The smallest power of two with amax <= 448 times it."""
    s = SCALE_MIN
    while s < SCALE_MAX and amax > 448 * s:
        s *= 2
    return s


def _scale(s):
    return s if math.isnan(s) else min(max(s, SCALE_MIN), SCALE_MAX)


def append_part(x, slots, codes, scales):
    """One of the two caches, codes [N, heads, block_size, dim] (a view of v's is
    transposed): writes x [T, heads, dim] in place."""
    N, heads, bs, _ = codes.shape
    runs = []
    for t, slot in enumerate(slots):
        b = slot // bs if 0 <= slot < N * bs else -1
        if b >= 0 and runs and runs[-1][0] == b and runs[-1][1][-1] == t - 1:
            runs[-1][1].append(t)
        elif b >= 0:
            runs.append((b, [t]))
    for b, tokens in runs:
        fresh = any(slots[t] % bs == 0 for t in tokens)
        for h in range(heads):
            new = np.asarray(x, dtype=np.float64)[tokens, h]
            was = _scale(float(scales[b, h]))
            if not np.isfinite(new).all():
                now = math.nan
            else:
                now = scale_for(np.abs(new).max())
                if not fresh:
                    now = was if math.isnan(was) else max(now, 2.0 ** math.ceil(math.log2(was)))
            if not fresh and now == now and now != scales[b, h]:
                codes[b, h] = encode(VALUES[codes[b, h]] * (was / now))
            for t in tokens:
                if now == now:
                    codes[b, h, slots[t] % bs] = encode(np.asarray(x[t, h], dtype=np.float64) / now)
                else:
                    codes[b, h, slots[t] % bs] = 0
            scales[b, h] = now


def tables(old_len, new_len, table, ring, state, block_size, tokens):
    """Changes table, ring and state in place; (granted, token_offsets, slots)."""
    S, width = table.shape
    N = len(ring)
    head, free = int(state[0]), int(state[1])
    asked = given = taken = at = 0
    granted, offsets, slots = [], [0], []
    back = []
    for s in range(S):
        old = min(max(int(old_len[s]), 0), width * block_size)
        new = max(int(new_len[s]), 0)
        have, need = -(-old // block_size), -(-new // block_size)
        fits = need <= width
        ask = max(0, need - have) if fits else 0
        ok = fits and (ask == 0 or asked + ask <= free)
        if ok:
            for i in range(have, need):
                table[s, i] = ring[(head + asked + i - have) % N]
                taken += 1
            for i in range(need, have):
                back.append((given + i - need, int(table[s, i])))
                table[s, i] = -1
        if fits:
            given += max(0, have - need)
        asked += ask
        granted.append(new if ok else old)
        for p in range(old, min(new, old + max(0, tokens - len(slots)))):
            b = int(table[s, p // block_size]) if ok else -1
            slots.append(b * block_size + p % block_size if 0 <= b < N else -1)
        at += max(0, new - old)
        offsets.append(min(at, 2 ** 31 - 1))
    for i, b in back:
        ring[(head + free + i) % N] = b
    if N:
        state[0], state[1] = (head + taken) % N, min(N, free - taken + len(back))
    slots = (slots + [-1] * tokens)[:tokens]
    return np.array(granted, dtype=np.int64), np.array(offsets), np.array(slots, dtype=np.int64)


def attention(q, q_offsets, kv_len, table, k_codes, v_codes, k_scale, v_scale, scale, bounds=False):
    """(out [T, q_heads, dim], lse [T, q_heads]); with bounds also what the error
    of a kernel goes by: sum_j w_j |v_j| / sum w (the size of what is summed),
    the largest sum |scale q_i k_i| of a row, and the largest |v| scale's 448."""
    q = np.asarray(q, dtype=np.float64)
    T, hq, dim = q.shape
    N, hkv, bs, _ = k_codes.shape
    S, width = table.shape
    out, lse = np.zeros((T, hq, dim)), np.full((T, hq), -np.inf)
    size, dots, top, count = np.zeros((T, hq, dim)), np.zeros((T, hq)), np.zeros((T, hq)), np.zeros((T, hq))
    for s in range(S):
        lo, hi = (min(max(int(q_offsets[i]), 0), T) for i in (s, s + 1))
        n = hi - lo
        length = min(max(int(kv_len[s]), 0), width * bs)
        at = np.arange(length)
        block = table[s][at // bs] if length else np.zeros(0, dtype=int)
        real = (block >= 0) & (block < N)
        at, block = at[real], block[real]
        for g in range(hkv):
            ks = np.array([_scale(float(x)) for x in k_scale[:, g]])[block][:, None]
            vs = np.array([_scale(float(x)) for x in v_scale[:, g]])[block][:, None]
            k = VALUES[k_codes[block, g, at % bs]] * ks
            v = VALUES[v_codes[block, g, :, at % bs]] * vs
            for i in range(max(n, 0)):
                seen = at <= length - n + i
                if not seen.any():
                    continue
                for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                    x = q[lo + i, h]
                    y = scale * (k[seen] @ x)
                    m = y.max()
                    w = np.exp(y - m)
                    out[lo + i, h] = w @ v[seen] / w.sum()
                    lse[lo + i, h] = m + np.log(w.sum())
                    if bounds:
                        size[lo + i, h] = w @ np.abs(v[seen]) / w.sum()
                        dots[lo + i, h] = scale * (np.abs(k[seen]) @ np.abs(x)).max()
                        top[lo + i, h] = 448 * (w[:, None] * vs[seen]).max() / w.sum()
                        count[lo + i, h] = seen.sum()
    if bounds:
        return out, lse, (size, dots, top, count)
    return out, lse
