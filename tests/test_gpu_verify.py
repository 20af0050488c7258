"""GPU parity of lik_verify_rows against the definition in float64.

Accepting and drawing are decisions, so a call's own decisions are followed and
each is held to the border it goes by: with the error of a probability from
rows_bounds.row_bounds (relative q_rel), a draft must not be accepted where
u q exceeds p by more than their errors, nor turned down where p exceeds u q, and a
drawn token's interval of the running sum, widened by the errors of all that is
summed, has to hold the random number's point."""

import math

import numpy as np
import pytest
import torch

import oracle
from maxsim_scoring_02_amd import _lib
from parity import say
from rows_bounds import U, logp_bound, row_bounds
from test_gpu_rows import on_gpu

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def f32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).cuda()


def row(z, scale):
    """(p, error of p, log p, error of ln Z) of one row of values; None without a softmax."""
    with np.errstate(invalid="ignore"):
        if not np.isfinite(z.max()) or np.isnan(z).any():
            return None
        p, logp, rel, ln_z = row_bounds(z[None], scale)
    return p[0], p[0] * (rel[0] + 4 * U), logp[0], ln_z[0]


def check(z, d, drafts, off, u, su, scale, dscale, got):
    tokens, accepted, logp = (x.cpu().numpy() for x in got)
    R, C = z.shape
    want_tokens, want_logp = np.full(R, -1), np.zeros(R)
    for s in range(len(off) - 1):
        lo, hi = max(int(off[s]), 0), min(int(off[s + 1]), R)
        if hi <= lo:
            assert accepted[s] == 0
            continue
        end = lo + accepted[s]
        assert lo <= end < hi
        for r in range(lo, end + 1):
            x = int(drafts[r])
            more = r + 1 < hi and x >= 0
            p, q = row(z[r], scale), row(d[r], dscale) if d is not None and more else None
            broken = p is None or (more and d is not None and q is None)
            assert r == end or (more and not broken)
            if broken:
                assert tokens[r] == -1 and math.isnan(logp[r])
                want_tokens[r], want_logp[r] = -1, np.nan
                break
            p, dp, lp, ln_z = p
            if more:
                px, ex = (p[x], dp[x]) if x < C else (0.0, 0.0)
                if d is None:
                    qx, eq = 1.0, 0.0
                else:
                    qx, eq = (q[0][x], q[1][x]) if x < C else (0.0, 0.0)
                un = float(np.float32(u[r]))
                if r < end:
                    assert un * (qx - eq) < px + ex, f"row {r}: accepted"
                    assert tokens[r] == x
                    want_tokens[r] = x
                else:
                    assert not (un * (qx + eq) < px - ex), f"row {r}: turned down"
            if r == end:
                w, e = p, dp
                if more:
                    qd, qe = (q[0], q[1]) if d is not None else (np.arange(C) == x, 0.0)
                    w, e = np.maximum(p - qd, 0), np.where(p - qd > -(dp + qe), dp + qe, 0.0)
                un = float(np.float32(su[s]))
                t = int(tokens[r])
                want_tokens[r] = t
                if math.isnan(un):
                    assert t == -1 and logp[r] == 0
                    continue
                assert 0 <= t < C
                c, slack = np.cumsum(w), e.sum() * (1 + abs(un)) + 1e-12 * w.sum()
                goal = un * c[-1]
                if c[-1] > 2 * slack:
                    assert w[t] + e[t] > 0
                    assert c[t] + slack >= min(goal, c[-1]) and c[t] - w[t] - slack <= max(goal, 0), f"row {r}: drew {t}"
            if want_tokens[r] >= 0:
                t = want_tokens[r]
                want_logp[r] = lp[t]
                x_t = (z[r].max() - z[r, t]) * scale
                if np.isfinite(lp[t]):
                    assert abs(logp[r] - lp[t]) <= logp_bound(lp[t], ln_z, min(x_t, 1e30)), f"row {r}: logp"
                else:
                    assert logp[r] == lp[t]
    assert np.array_equal(tokens, want_tokens)
    assert (logp[(want_tokens < 0) & (want_logp == 0)] == 0).all()       # no token, no log-probability


def make(counts, C, seed, drafter=True, spread=2.5, noise=0.6, lead=0, pad=0):
    """Rows, drafts drawn from the drafter, and uniform numbers."""
    rng = np.random.default_rng(seed)
    off = lead + np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1]) + pad
    z = (rng.standard_normal((R, C)) * spread).astype(np.float32)
    d = (z + noise * rng.standard_normal((R, C))).astype(np.float32)
    q = np.exp(d - d.max(1, keepdims=True))
    drafts = np.array([rng.choice(C, p=x / x.sum()) for x in q.astype(np.float64)]) if R else np.zeros(0, int)
    if not drafter:
        d = None
    for s in range(len(counts)):
        if counts[s]:
            drafts[off[s + 1] - 1] = [-1, 0, C + 5][s % 3]           # not looked at
    return z, d, drafts, off, rng.uniform(0, 1, R).astype(np.float32), rng.uniform(0, 1, len(counts)).astype(np.float32)


def run(z, d, drafts, off, u, su, dtype, scale=1.0, dscale=1.0, pad=0, shift=0):
    gz, hz = on_gpu(z, dtype, pad, shift)
    gd, hd = on_gpu(d, dtype, 2 * pad, shift) if d is not None else (None, None)
    got = _lib.lik_verify_rows(gz, i32(drafts), i32(off), f32(u), f32(su), draft_logits=gd, scale=scale,
                               draft_scale=dscale)
    check(hz, hd, drafts, off, u, su, scale, dscale, got)
    return got


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("C", [1, 2, 7, 64, 300, 2049, 5003, 33001])
def test_verify(C, drafter, dtype):
    say(f"[verify] C {C}, drafter {drafter}, {dtype}")
    counts = [5, 1, 3, 0, 2, 6]
    case = make(counts, C, C, drafter, lead=C % 2, pad=C % 3)
    pad, shift = [(0, 0), (3, 1), (8, 8)][C % 3]
    run(*case, dtype, scale=[1.0, 0.7][C % 2], dscale=[1.0, 1.3][C % 2], pad=pad, shift=shift)


@pytest.mark.parametrize("S,K,C,dtype", [(1, 1, 70000, BF16), (1, 9, 140001, F32), (300, 2, 4099, BF16), (3, 4, 131072, F16),
                                         (40, 5, 20000, F32), (700, 3, 65, F16), (33, 4, 66000, BF16)])
def test_many_and_long(S, K, C, dtype):
    say(f"[verify] {S} x {K + 1} x {C} {dtype}")
    run(*make([K + 1] * S, C, S + C), dtype)


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("S,top,C,dtype", [(170, 4, 33001, F16), (160, 3, 32768, BF16), (165, 3, 16411, F32),
                                           (161, 2, 140001, BF16), (159, 3, 33000, F16)])
def test_many_sequences_of_long_rows(S, top, C, dtype, drafter):
    """Rows of more than one part, beyond what the caches keep: every kind of end and of
    row among them."""
    say(f"[verify] {S} sequences of up to {top} rows of {C} {dtype}, drafter {drafter}")
    rng = np.random.default_rng(C)
    counts = rng.integers(0, top + 1, S)
    counts[:24] = top
    z, d, drafts, off, u, su = make(counts, C, C, drafter, lead=3, pad=2)
    z[:3], z[-2:] = np.nan, np.inf
    for r in (off[0], off[1] + 1):
        z[r] = -np.inf
    z[off[2] + 1, 77], z[off[3], C - 1] = np.nan, np.inf
    z[off[4] + 1, rng.random(C) < 0.99] = -np.inf
    z[off[5]], z[off[5], 5] = -np.inf, 1.0           # one column left
    z[off[6]:off[7]] = np.float32(-6e4 if dtype == F16 else -1e9)
    drafts[off[7]], drafts[off[8] + 1], drafts[off[9]] = -1, -7, C
    su[10:16] = [0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, 5.0, -0.25, math.nan]
    u[off[0]:off[10]] = 0.0
    u[off[16]], u[off[17] + 1] = math.nan, 2.0
    if drafter:
        d[:3] = np.nan
        d[off[18]], d[off[19] + 1, 9] = -np.inf, np.nan
        d[off[20] + top - 1] = np.nan                # a last row's draft is not read
        d[off[21]:off[22]] = z[off[21]:off[22]]
    run(z, d, drafts, off, u, su, dtype, scale=0.9, dscale=1.2, pad=C % 2, shift=C % 3)


def test_random_numbers_at_their_ends():
    z, d, drafts, off, u, su = make([4] * 7, 501, 3)
    u[:] = [0.0, np.nextafter(np.float32(1), np.float32(0))] * 14
    su[:] = [0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, 7.0, -0.5, math.nan, 0.5]
    t, a, _ = run(z, d, drafts, off, u, su, F32)
    u[0::4] = math.nan                       # does not accept
    t, a, _ = run(z, d, drafts, off, u, su, F32)
    assert a.tolist() == [0] * 7
    assert t[4 * 5] == -1 and t[4 * 4] == 0
    # behind the last draft nothing is taken away: the first and the last column
    one = make([1] * 7, 501, 4)
    t, _, _ = run(*one[:5], su, F32)
    assert t[0] == 0 and t[2] == t[3] == 500


def test_every_draft_of_the_target_itself_is_accepted():
    z, _, drafts, off, u, su = make([6] * 9, 1000, 5)
    t, a, _ = run(z, z.copy(), drafts, off, u, su, BF16)
    assert a.tolist() == [5] * 9


def test_drafts_that_end_early_and_that_do_not_exist():
    for drafter in (True, False):
        z, d, drafts, off, u, su = make([5] * 6, 77, 6, drafter)
        u[:] = 0.0
        drafts[off[0]] = -1
        drafts[off[1] + 2] = -9
        drafts[off[2]] = 77                 # no such column
        drafts[off[3] + 1] = 2 ** 31 - 1
        t, a, _ = run(z, d, drafts, off, u, su, F32)
        assert a.tolist() == [0, 2, 0, 1, 4, 4]


def test_masked_columns():
    """Columns that are ruled out: by the target, by the drafter, by both, all but one."""
    for dtype in (F16, F32):
        z, d, drafts, off, u, su = make([4] * 8, 600, 8)
        rng = np.random.default_rng(2)
        z[rng.random(z.shape) < 0.9] = -np.inf
        z[np.arange(len(z)), rng.integers(0, 600, len(z))] = 1.0
        d[rng.random(d.shape) < 0.5] = -np.inf
        d[np.arange(len(d)), drafts.clip(0, 599)] = 2.0
        z[3], z[3, 17] = -np.inf, 0.0
        z[4:8] = np.finfo(np.float16).min
        z[5, 3] = 2.0
        run(z, d, drafts, off, u, su, dtype)
        run(z, None, drafts, off, u, su, dtype)


def test_rows_without_a_softmax_end_their_sequence():
    z, d, drafts, off, u, su = make([4] * 6, 90, 9)
    u[:] = 0.0
    z[off[0]], z[off[1] + 1, 5], z[off[2] + 3, 0] = -np.inf, np.nan, np.inf
    d[off[3]], d[off[4] + 2, 7] = -np.inf, np.nan
    d[off[5] + 3] = np.nan                   # a last row's draft is not read
    t, a, lp = run(z, d, drafts, off, u, su, F32)
    assert a.tolist() == [0, 1, 3, 0, 2, 3]
    assert torch.isnan(lp).sum() == 5 and (t[torch.isnan(lp)] == -1).all()


def test_one_hot_targets():
    """The whole mass in one column: what is left after a draft that takes it is nothing."""
    z, d, drafts, off, u, su = make([3] * 4, 50, 10)
    z[:] = -80.0
    z[:, 7] = 80.0
    d[:] = z
    drafts[:] = 7
    u[off[1]] = 2.0                          # more than any probability
    t, a, _ = run(z, d, drafts, off, u, su, F32)
    assert a.tolist() == [2, 0, 2, 2] and t[off[1]] == 7
    t, a, _ = run(z, None, drafts, off, u, su, F32)
    assert a.tolist() == [2, 0, 2, 2]


def test_rows_outside_and_sequences_without_rows():
    z, d, drafts, off, u, su = make([0, 3, 0, 0, 2, 0], 40, 11, lead=4, pad=5)
    z[:4], z[-5:], d[:4], d[-5:] = np.nan, np.nan, np.nan, np.nan
    t, a, lp = run(z, d, drafts, off, u, su, BF16)
    assert (t[:4] == -1).all() and not lp[:4].any() and not lp[-5:].any()
    e = torch.empty(0, device="cuda")
    t, a, lp = _lib.lik_verify_rows(torch.randn(3, 9, device="cuda"), i32([1, 2, 3]), i32([0]), f32([0, 0, 0]), e)
    assert t.tolist() == [-1] * 3 and not lp.any() and a.shape == (0,)
    t, a, lp = _lib.lik_verify_rows(torch.randn(0, 9, device="cuda"), i32([]), i32([0, 0]), e, f32([0.5]))
    assert t.shape == (0,) and a.tolist() == [0]
    # offsets out of range stay inside
    z, d, drafts, off, u, su = make([3, 3], 40, 12)
    run(z, d, drafts, [-5, 3, 99], u, su, F32)


def test_far_rows_and_temperatures():
    for shift, scale in ((20000.0, 1.0), (-3e4, 0.5), (1e6, 3.0)):
        z, d, drafts, off, u, su = make([4] * 5, 999, 13)
        run(z + np.float32(shift), d - np.float32(shift), drafts, off, u, su, F32, scale=scale, dscale=1 / scale)
    z, d, drafts, off, u, su = make([4] * 5, 999, 14)
    run(z, d, drafts, off, u, su, F32, scale=2.0 ** -20, dscale=2.0 ** 10)
    z[:] = -1e9
    run(z, d, drafts, off, u, su, F32, scale=50.0)


def test_tokens_have_the_targets_distribution():
    """20000 sequences with random numbers of their own: the first token's shares
    are p within six standard deviations."""
    rng = np.random.default_rng(15)
    S, C = 20000, 12
    z, d = rng.standard_normal((2, C)).astype(np.float32) * 1.5
    q = np.exp(d - d.max()).astype(np.float64)
    drafts = np.full((S, 2), -1)
    drafts[:, 0] = rng.choice(C, S, p=q / q.sum())
    zz, dd = (torch.tensor(x).cuda().expand(2 * S, C).contiguous() for x in (z, d))
    t, a, _ = _lib.lik_verify_rows(zz, i32(drafts.ravel()), i32(np.arange(S + 1) * 2), torch.rand(2 * S).cuda(),
                                   torch.rand(S).cuda(), draft_logits=dd)
    p = np.exp(z - z.max()).astype(np.float64)
    p /= p.sum()
    share = np.bincount(t.view(S, 2)[:, 0].cpu().numpy(), minlength=C) / S
    assert (np.abs(share - p) < 6 * np.sqrt(p / S) + 1e-9).all()
    assert 0 < a.sum() < S


@pytest.mark.parametrize("S", [1, 63, 64, 65, 4095, 4097, 70001])
def test_last_rows_of_many_sequences(S):
    """Drafters' rows behind the last draft are anything, whatever their number and the
    sequences': the offsets are searched in steps of 64."""
    rng = np.random.default_rng(S)
    counts = rng.integers(0, 4, S)
    off = np.concatenate([[0], np.cumsum(counts)])
    R, C = int(off[-1]) + 1, 4
    z = torch.randn(R, C, device="cuda")
    d = z.clone()
    ends = torch.as_tensor(off[1:][counts > 0] - 1).cuda()
    d[ends] = float("nan")
    drafts = torch.zeros(R, dtype=torch.int32, device="cuda")
    t, a, lp = _lib.lik_verify_rows(z, drafts, i32(off), torch.full((R,), 0.99, device="cuda"),
                                    torch.full((S,), 0.5, device="cuda"), draft_logits=d)
    assert a.tolist() == np.maximum(counts - 1, 0).tolist()
    assert not torch.isnan(lp).any() and (t[ends] >= 0).all() and (t[:-1] >= 0).sum() == int(off[-1])


def test_offsets_past_32_bits():
    C = 2 ** 20
    R = 2 ** 32 // (2 * C) + 3
    z = torch.zeros(R, C, dtype=BF16, device="cuda")
    z[-2:] = torch.randn(2, C, device="cuda")
    off = [R - 2, R]
    t, a, lp = _lib.lik_verify_rows(z, torch.full((R,), 5, dtype=torch.int32, device="cuda"), i32(off),
                                    torch.full((R,), 0.99, device="cuda"), f32([0.3]))
    check(z[-2:].double().cpu().numpy(), None, [5, 5], [0, 2], [0.99, 0.99], [0.3], 1.0, 1.0, (t[-2:], a, lp[-2:]))
    assert (t[:-2] == -1).all()


def test_binding_on_the_gpu():
    z, t = torch.zeros(4, 6, device="cuda"), i32([0] * 4)
    u, off, su = torch.zeros(4, device="cuda"), i32([0, 4]), torch.zeros(1, device="cuda")
    good = dict(logits=z, draft_tokens=t, seq_offsets=off, accept_u=u, sample_u=su, draft_logits=z.clone())
    bad = [(dict(draft_tokens=t[:3]), "shape"), (dict(accept_u=u.half()), "float32"), (dict(sample_u=u), "shape"),
           (dict(draft_logits=z.half()), "type"), (dict(draft_logits=z.mT.contiguous().mT), "dense"),
           (dict(seq_offsets=off.cpu()), "device"), (dict(logits=z.double()), "float16"), (dict(draft_scale=-1.0), "draft_scale")]
    for kw, msg in bad:
        with pytest.raises((ValueError, _lib.LikError), match=msg):
            _lib.lik_verify_rows(**{**good, **kw})
    a = _lib.lik_verify_rows(**good)
    b = _lib.lik_verify_rows(**{**good, "draft_tokens": t.long(), "seq_offsets": off.long()})
    assert all(torch.equal(x, y) for x, y in zip(a, b))
