"""Pins of the oracle of a step of generation (oracle/cache.py and
rows.verify_rows): codes against torch's own 8-bit type, scales, block tables
against a pool kept by hand, attention against one softmax over dense arrays, and
verified tokens against the distribution they have to have."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache


def test_codes_are_those_of_the_type():
    bits = torch.arange(256, dtype=torch.uint8)
    theirs = bits.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache.VALUES, theirs, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    rng = np.random.default_rng(1)
    x = rng.standard_normal(20000) * np.exp2(rng.uniform(-12, 9, 20000))
    mid = (cache.VALUES[:126] + cache.VALUES[1:127]) / 2
    x = np.concatenate([x.clip(-448, 448), mid, -mid, cache.VALUES[:127], [0.0, -0.0, 448.0, 2.0 ** -10, 2.0 ** -11]])
    theirs = torch.tensor(x).to(torch.float32)
    keep = theirs.double().numpy() == x               # so that both round the same number
    got = cache.encode(x[keep])
    assert np.array_equal(got, theirs[torch.tensor(keep)].to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert keep[-260:].all()
    assert cache.VALUES[cache.encode(1e9)] == 448 and cache.VALUES[cache.encode(-500.0)] == -448


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.0001, 2.0), (0.0, 2.0 ** -40), (1e30, 2.0 ** 40),
                                       (224.0, 0.5), (225.0, 1.0), (1.0, 2.0 ** -8), (3.5, 2.0 ** -7)])
def test_scales(amax, want):
    assert cache.scale_for(amax) == want


def test_append_keeps_what_stands_when_a_scale_grows():
    rng = np.random.default_rng(2)
    codes, scales = np.zeros((2, 1, 16, 4), dtype=np.uint8), np.ones((2, 1))
    a = rng.standard_normal((3, 1, 4)).clip(-1.7, 1.7)
    cache.append_part(a, [16, 17, 18], codes, scales)
    held = cache.VALUES[codes[1, 0, :3]] * scales[1, 0]
    assert scales[1, 0] == 2.0 ** -8 and np.abs(held - a[:, 0]).max() <= 2.0 ** -4 * 1.8
    b = np.full((1, 1, 4), 100.0)
    cache.append_part(b, [19], codes, scales)
    assert scales[1, 0] == 2.0 ** -2
    again = cache.VALUES[codes[1, 0, :3]] * scales[1, 0]
    normal = np.abs(held) >= 2.0 ** -2 * 2.0 ** -6
    assert np.array_equal(again[normal], held[normal])
    assert np.abs(again - held).max() <= 2.0 ** -2 * 2.0 ** -10
    # a block's first slot starts it anew
    cache.append_part(a[:1], [16], codes, scales)
    assert scales[1, 0] == cache.scale_for(np.abs(a[0]).max())


def test_tables_against_a_pool_kept_by_hand():
    rng = np.random.default_rng(3)
    N, width, bs, S = 40, 6, 16, 7
    table, ring, state = np.full((S, width), -1), rng.permutation(N), np.array([0, N, 0, 0])
    lens = np.zeros(S, dtype=int)
    for step in range(60):
        want = lens + rng.integers(-60, 70, S)
        T = int(np.maximum(want - lens, 0).sum()) + 3
        free = int(state[1])
        got, off, slots = cache.tables(lens, want, table, ring, state, bs, T)
        asked = 0
        for s in range(S):
            need, have = -(-max(want[s], 0) // bs), -(-lens[s] // bs)
            asked += max(0, need - have) if need <= width else 0
            fine = need <= width and (need <= have or asked <= free)
            assert got[s] == (max(want[s], 0) if fine else lens[s])
            mine = slots[off[s]:off[s + 1]]
            if fine:
                pos = np.arange(lens[s], lens[s] + len(mine))
                assert np.array_equal(mine, table[s][pos // bs] * bs + pos % bs)
            else:
                assert (mine == -1).all()
        assert (slots[off[-1]:] == -1).all()
        lens = got
        held = [table[s, i] for s in range(S) for i in range(-(-lens[s] // bs))]
        pool = [ring[(state[0] + i) % N] for i in range(state[1])]
        assert sorted(held + pool) == list(range(N))
        assert all(table[s, i] == -1 for s in range(S) for i in range(-(-lens[s] // bs), width))


def test_attention_is_a_softmax():
    rng = np.random.default_rng(4)
    N, hkv, bs, dim, L, n = 5, 2, 16, 8, 37, 3
    kc, vc = rng.integers(0, 127, (2, N, hkv, bs, dim)).astype(np.uint8)
    vc = np.ascontiguousarray(vc.transpose(0, 1, 3, 2))
    ks, vs = np.exp2(rng.integers(-9, -6, (2, N, hkv)).astype(float))
    table = np.array([[3, 0, 4]])
    q = rng.standard_normal((n, 4, dim))
    out, lse = cache.attention(q, [0, n], [L], table, kc, vc, ks, vs, 0.3)
    for h in range(4):
        k = np.concatenate([cache.VALUES[kc[b, h // 2]] * ks[b, h // 2] for b in table[0]])[:L]
        v = np.concatenate([cache.VALUES[vc[b, h // 2]].T * vs[b, h // 2] for b in table[0]])[:L]
        y = torch.tensor(0.3 * q[:, h] @ k.T)
        y = y.masked_fill(torch.ones(n, L).triu(L - n + 1).bool(), -math.inf)
        assert np.allclose(lse[:, h], torch.logsumexp(y, 1), rtol=1e-12)
        assert np.allclose(out[:, h], torch.softmax(y, 1) @ torch.tensor(v), rtol=1e-12)


def test_attention_of_nothing():
    z = np.zeros((3, 1, 16, 4), dtype=np.uint8)
    one = np.ones((3, 1))
    out, lse = cache.attention(np.ones((4, 1, 4)), [0, 1, 3], [0, 2], np.array([[0], [-1]]), z,
                               z.transpose(0, 1, 3, 2), one, one, 1.0)
    assert not out.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("drafter", [True, False])
def test_verified_tokens_have_the_targets_distribution(drafter):
    """The first emitted token over a fine grid of random numbers: its shares are
    p, whatever the drafter."""
    rng = np.random.default_rng(5)
    C, G = 5, 200
    z, d = rng.standard_normal((2, 2, C)) * 1.5
    p = np.exp(z[0]) / np.exp(z[0]).sum()
    q = np.exp(d[0]) / np.exp(d[0]).sum() if drafter else np.eye(C)[2]
    share = np.zeros(C)
    grid = (np.arange(G) + 0.5) / G
    for x in range(C):
        if q[x] == 0:
            continue
        taken = np.mean(grid * q[x] < p[x])
        share[x] += q[x] * taken
        if taken < 1:
            rest = np.zeros(C)
            for u in grid:
                t, a, _ = oracle.verify_rows(z, [x, -1], [0, 2], [1.0, 0.0], [u], d if drafter else None)
                assert a[0] == 0 and t[1] == -1
                rest[t[0]] += 1 / G
            share += q[x] * (1 - taken) * rest
    assert np.abs(share - p).max() < 2.0 / G * C


def test_verified_rows_by_hand():
    z = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.8, 0.1], [0.25, 0.25, 0.5]]))
    t, a, lp = oracle.verify_rows(z, [0, 1, 7], [0, 3], [0.4, 0.7, 0.9], [0.6])
    assert t.tolist() == [0, 1, 2] and a[0] == 2
    assert np.allclose(lp, np.log([0.5, 0.8, 0.5]))
    t, a, lp = oracle.verify_rows(z, [0, 1, 7], [0, 3], [0.4, 0.85, 0.9], [0.6])
    assert t.tolist() == [0, 2, -1] and a[0] == 1 and lp[2] == 0      # 0.1, 0, 0.1 of what is left
    t, a, _ = oracle.verify_rows(z, [0, -1, 0], [0, 3], [0.4, 0.0, 0.0], [0.05])
    assert t.tolist() == [0, 0, -1] and a[0] == 1                     # drafts end early: all of p
    t, a, lp = oracle.verify_rows(z, [0, 0, 0], [1, 1, 1], [0.4, 0.0, 0.0], [0.05, 0.1])
    assert t.tolist() == [-1] * 3 and a.tolist() == [0, 0] and not lp.any()
