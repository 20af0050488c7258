"""Weights far below a row's largest: attention over the 8-bit cache where one token
takes nearly all of the sum and its values are 0 in half of the dims, so that what the
others add is all that stands there; and value scales of blocks far apart.

Keys have one number that counts, against a power of two in the query: a score is one
exact product, and with s = log2(e) scale q k, L = log2(v_scale), both at most D,
u = 2^-24, a weight's relative error is

  exponent   log2(e) scale is rounded twice, 2 u |s|; L - m, u (D + 16 + |L|); the sum of
             both, u (D + 16); at most 2 (D + 16) above the largest of a tile each time
             that the reference moves: together 8 u (D + 16) with ln 2 < 1, twice that for
             scales that are no powers of two (their log2, u |L| more)
  exponential and factors of moves   2 u each, few

so e = 16 u (D + 16).  The weight is then rounded to 2^-11 of itself (float32: 2^-22), or,
where its product with v_scale is below 2^-25 (2^-29) of the row's largest, by at most
2^-36 (2^-51) of that.  The product is 2 e off by the sum above and the one below, sums
are float32 over up to L terms, (L / 16 + 64) u of the size of what is summed, and
the result is rounded once."""

import numpy as np
import pytest
import torch

from maxsim_scoring_02_amd import _lib
from oracle import cache as oc
from parity import say
from test_gpu_cache import BF16, F16, F32, U, Cache, host, i32

pytestmark = pytest.mark.gpu


def build(lens, bs, dim, hkv, seed, sinks, v_scale, gap_bits):
    """Requests whose tokens have scores 16 to `gap_bits` powers of two below those of
    `sinks` (positions), by the key's first number; values of sinks are 0 in every other dim."""
    rng = np.random.default_rng(seed)
    blocks = [-(-x // bs) for x in lens]
    N, S = sum(blocks), len(lens)
    c = Cache(N, hkv, bs, dim, seed)
    ids, table, at = rng.permutation(N), np.full((S, max(blocks)), -1), 0
    c.k[:] = 0
    # 448 for a sink, at most half of it for others
    c.k[..., 0] = rng.integers(0x50, 0x77, c.k[..., 0].shape)
    c.ks[:] = 1.0
    c.vs[:] = v_scale(rng, N)[:, None]
    for s, b in enumerate(blocks):
        table[s, :b] = ids[at:at + b]
        at += b
        for p in sinks:
            if p < lens[s]:
                block, o = table[s, p // bs], p % bs
                c.k[block, :, o, 0] = 0x7e
                c.v[block, :, ::2, o] = 0
    for g, x in ((c.gk, c.k), (c.gv, c.v)):
        g.view(torch.uint8).copy_(torch.from_numpy(x))
    c.gks.copy_(torch.tensor(c.ks)), c.gvs.copy_(torch.tensor(c.vs))
    scale = float(np.float32(gap_bits / 448 * np.log(2)))
    return c, table, scale


def check(c, table, scale, lens, n, hq, dtype, seed):
    N, hkv, bs, dim = c.sizes
    off = np.arange(len(lens) + 1) * n
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(off[-1], hq, dim, generator=gen)
    q[..., 0] = 1.0
    q = q.to(dtype).cuda()
    got, lse = _lib.lik_cache_attention(q, i32(off), i32(lens), i32(table), *c.parts, scale=scale, want_lse=True)
    want, rl, (size, _, top, count) = oc.attention(host(q), off, lens, table, c.k, c.v, c.ks, c.vs, scale, bounds=True)
    D = 448 * scale * np.log2(np.e) + np.abs(np.log2(c.vs)).max()
    e = 16 * U * (D + 16)
    part, least = (2.0 ** -22, 2.0 ** -51) if dtype == F32 else (2.0 ** -11, 2.0 ** -36)
    tol = size * (2 * e + part + (count / 16 + 64) * U)[..., None] + (count * least * top)[..., None]
    tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(want) + tol) + {F16: 2.0 ** -25, BF16: 2.0 ** -133, F32: 2.0 ** -149}[dtype]
    x = host(got)
    # what lies beyond the type (float16: from 65520 on) is infinite, and next to its end either
    most = float(torch.finfo(dtype).max)
    beyond = np.abs(want) - tol > most * (1 + 2.0 ** -11)
    assert (x[beyond] == np.copysign(np.inf, want[beyond])).all()
    fits = np.abs(want) + tol < most
    over = np.where(fits, np.abs(np.where(fits, x, 0.0) - want) / tol, 0.0)
    assert np.isfinite(x[fits]).all() and over.max() <= 1, f"{over.max():.3g} of the bound at {np.unravel_index(over.argmax(), over.shape)}"
    assert (np.abs(host(lse) - rl) <= e + (count / 16 + 64) * U + 4 * U * (np.abs(rl) + 1)).all()
    return want, tol


DTYPES = [F16, BF16, F32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,n,hq,hkv,dim,bs,sinks", [
    ([9000], 1, 4, 1, 64, 16, [0]), ([4097, 3000], 1, 8, 2, 128, 32, [2500]), ([2600], 3, 2, 1, 256, 64, [2590]),
    ([3000, 2900], 40, 2, 2, 64, 16, [5, 1700]), ([1500], 50, 2, 1, 128, 128, [0])])
def test_tokens_beside_a_sink(lens, n, hq, hkv, dim, bs, sinks, dtype):
    say(f"[cache] {lens} tokens beside a sink, {hq} / {hkv} heads of {dim}, {dtype}")
    # float16's smallest numbers must not decide (the sink's own values pass its largest)
    up = 2.0 ** 10
    c, table, scale = build(lens, bs, dim, hkv, len(lens) + dim, sinks, lambda rng, N: np.full(N, up), 30)
    want, tol = check(c, table, scale, lens, n, hq, dtype, 1)
    zero = want[..., ::2]                  # what the others add: known to a few bits at least, or to most
    known = np.abs(zero) / tol[..., ::2]
    assert np.median(known) > (2.0 ** 9 if dtype == F32 else 2.0 ** 4)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("apart", [20, 30, 40])
def test_values_scales_apart(apart, dtype):
    """Blocks whose value scales are 2^20 to 2^40 above the others', their values 0 in half the dims."""
    lens, n, hq, hkv, dim, bs = [2000, 700], 2, 4, 2, 64, 32

    def v_scale(rng, N):
        return np.where(rng.random(N) < 0.1, 2.0 ** (apart - 10), 2.0 ** -10)

    c, table, scale = build(lens, bs, dim, hkv, apart, [], v_scale, 3)
    high = c.vs[:, 0] > 2.0 ** -10
    c.v[high, :, ::2] = 0
    c.gv.view(torch.uint8).copy_(torch.from_numpy(c.v))
    want, tol = check(c, table, scale, lens, n, hq, dtype, 2)
    if apart == 20:
        assert np.median(np.abs(want[..., ::2]) / tol[..., ::2]) > (2.0 ** 9 if dtype == F32 else 2.0 ** 4)


@pytest.mark.parametrize("dtype", DTYPES)
def test_sinks_that_come_late(dtype):
    """The largest score grows from tile to tile by less and by more than the weights' room."""
    lens, n, hq, hkv, dim, bs = [1200], 1, 2, 1, 64, 16
    for step in (0.5, 3.9, 4.4, 11.0):
        c, table, scale = build(lens, bs, dim, hkv, 3, [], lambda rng, N: np.full(N, 2.0 ** 10), 1)
        # token p's key: 2^(p / 64) tiles up, as far as codes go
        value = np.minimum(1 + np.arange(lens[0] // 64 + 1), 448.0)
        for p in range(lens[0]):
            c.k[table[0, p // bs], :, p % bs, 0] = oc.encode(value[p // 64])
        c.gk.view(torch.uint8).copy_(torch.from_numpy(c.k))
        check(c, table, float(np.float32(step * np.log(2))), lens, n, hq, dtype, 5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_far_from_zero(dtype):
    """Rows whose scores are all near +-2^20 .. 2^30: equal ones share the sum, none overflows."""
    lens, n, hq, hkv, dim, bs = [500], 1, 2, 1, 64, 16
    for bits in (20, 21, 22, 23, 24, 25, 26, 27, 30):
        for sign in (1.0, -1.0):
            c, table, _ = build(lens, bs, dim, hkv, 9, [], lambda rng, N: np.ones(N), 1)
            c.k[..., 0] = oc.encode(256.0)
            c.gk.view(torch.uint8).copy_(torch.from_numpy(c.k))
            q = torch.zeros((1, hq, dim), dtype=dtype, device="cuda")
            q[..., 0] = sign
            off = [0, 1]
            got, _ = _lib.lik_cache_attention(q, i32(off), i32(lens), i32(table), *c.parts, scale=2.0 ** (bits - 8))
            # all weights are equal, whatever they are: their mean, of weights rounded alike
            want = oc.attention(host(q), off, lens, table, c.k, c.v, c.ks, c.vs, 2.0 ** (bits - 8))[0]
            size = oc.attention(host(q), off, lens, table, c.k, c.v & 0x7f, c.ks, c.vs, 2.0 ** (bits - 8))[0]
            tol = size * (2.0 ** -10 + (500 / 16 + 64) * U) + torch.finfo(dtype).eps * np.abs(want)
            assert (np.abs(host(got) - want) <= tol).all(), (bits, sign)
