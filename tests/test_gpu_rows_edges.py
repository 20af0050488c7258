"""GPU checks of the row losses at their edges: rows without a log-probability,
pairs of a sequence with itself, calls from several host threads, sizes beyond
the library's, sums within the terms of a thread, and gradients of 16-bit logits
against differences.  Helpers and bounds as in test_gpu_rows.py and
rows_bounds.py."""

import threading

import numpy as np
import pytest
import torch

import oracle
from maxsim_scoring_02_amd import _lib
from parity import say
from rows_bounds import U, logp_bound, rounded, row_bounds
from test_gpu_rows import BF16, F16, F32, distill_case, f32, host, i32, on_gpu, policy_case, within

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def normal(R, C, dtype, seed):
    """Logits [R, C] and targets [R] made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.empty((R, C), device="cuda", dtype=dtype).normal_(0, 2, generator=g)
    return z, torch.randint(0, C, (R,), generator=g, device="cuda", dtype=torch.int32)


def same(x, where):
    return np.array_equal(host(x), where)


# one wave, 256 threads, 1024 threads, partly in LDS, in parts, many rows in parts
FORMS = [(9, 33, F32), (9, 9001, F16), (128, 70001, BF16), (130, 140001, BF16), (9, 70001, F32),
         (1030, 262200, BF16)]


@pytest.mark.parametrize("R,C,dtype", FORMS)
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_policy_without_advantage_keeps_nan(R, C, dtype, kl):
    """An advantage of 0 (a group of rollouts with equal rewards) has loss 0 and no
    gradient, but a row without a log-probability stays NaN."""
    say(f"[rows] policy advantage 0 {R} x {C} {dtype} kl {kl}")
    z, t = normal(R, C, dtype, 90)
    t[1], t[5], t[6] = C, 2 ** 31 - 1, -1       # two out of range, one left out
    z[2, C - 1] = NAN
    z[3] = -INF
    z[4, C // 2] = INF
    t[7], z[7] = 2, -INF                        # left out by its weight
    bad = np.zeros(R, dtype=bool)
    bad[1:6] = True
    w = torch.ones(R, device="cuda")
    w[7] = 0.0
    old, ref = torch.full((R,), -5.0, device="cuda"), torch.full((R,), -6.0, device="cuda")
    old[8] = -500.0                             # a ratio that overflows: inf * 0
    args = (z, t, old, torch.zeros(R, device="cuda"), ref)
    loss, rows, lp, grad = _lib.lik_policy_rows(*args, kl_coef=kl, row_weight=w)
    none = _lib.lik_policy_rows(*args, kl_coef=kl, row_weight=w, want_grad=False)
    for l, r, p in ((loss, rows, lp), none[:3]):
        assert torch.isnan(l).all()
        assert same(torch.isnan(r), bad) and same(torch.isnan(p), bad)
    assert same(torch.isnan(grad).all(1), bad) and same(torch.isnan(grad).any(1), bad)
    if kl == 0:
        good = torch.from_numpy(~bad).cuda()
        assert torch.all(rows[good] == 0) and torch.all(none[1][good] == 0)
        assert torch.all(grad[good] == 0)


@pytest.mark.parametrize("kind", [_lib.LIK_PREF_SIGMOID, _lib.LIK_PREF_HINGE, _lib.LIK_PREF_SQUARE])
@pytest.mark.parametrize("R,S", [(30, 6), (900, 300)])
@pytest.mark.parametrize("mean", [False, True])
def test_pair_of_a_sequence_with_itself(R, S, kind, mean):
    """Its difference is 0, and so is its part of the gradient; with a NaN in the
    sequence the pair's loss and the sequence's gradient are NaN."""
    say(f"[rows] preference with itself {R} rows kind {kind} mean {mean}")
    n = R // S
    z, t = normal(R, 50, F32, 92)
    off = i32(np.arange(0, R + 1, n))
    args = dict(kind=kind, beta=0.5, mean_logp=mean)
    one = _lib.lik_preference_rows(z, t, off, i32([1, 3]), i32([2, 3]), pair_weight=f32([1, 4]), **args)
    ref = _lib.lik_preference_rows(z, t, off, i32([1]), i32([2]), pair_weight=f32([1]), **args)
    assert torch.equal(one[3], ref[3]) and torch.all(one[3][3 * n:4 * n] == 0)
    z[3 * n + 1, 7] = NAN
    t[3 * n + 2] = -1
    loss, pairs, seq, grad = _lib.lik_preference_rows(z, t, off, i32([1, 3]), i32([2, 3]),
                                                      pair_weight=f32([1, 4]), **args)
    assert torch.isnan(loss).all() and same(torch.isnan(pairs), [False, True])
    rows = np.zeros(R, dtype=bool)
    rows[3 * n:4 * n] = True
    rows[3 * n + 2] = False                     # left out
    assert same(torch.isnan(grad).all(1), rows) and same(torch.isnan(grad).any(1), rows)
    assert torch.equal(grad[n:3 * n], ref[3][n:3 * n])
    # without weight the pair is left out of the sum and the gradient
    out = _lib.lik_preference_rows(z, t, off, i32([1, 3]), i32([2, 3]), pair_weight=f32([1, 0]), **args)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[3]).all()


@pytest.mark.parametrize("R,C,dtype", FORMS[:5])
def test_distill_rows_all_masked_without_listed_mass(R, C, dtype):
    """A row all of -inf has no softmax: NaN, with only the rest's term to it too
    (no entry listed, or entries without mass)."""
    say(f"[rows] distill all masked {R} x {C} {dtype}")
    z, t = normal(R, C, dtype, 94)
    z[1:4] = -INF
    idx = torch.stack([t, (t + 1) % C], 1).int()
    val = torch.zeros((R, 2), device="cuda")
    idx[1] = -1
    val[2] = -INF
    idx[4] = -1
    val[5] = -INF
    lse = torch.full((R,), 3.0, device="cuda")
    loss, rows, grad = _lib.lik_distill_rows(z, idx, val, lse)
    none = _lib.lik_distill_rows(z, idx, val, lse, want_grad=False)
    bad = np.isin(np.arange(R), [1, 2, 3])
    for l, r in ((loss, rows), none[:2]):
        assert torch.isnan(l).all() and same(torch.isnan(r), bad)
        assert torch.isfinite(r[torch.from_numpy(~bad).cuda()]).all()
    assert same(torch.isnan(grad).all(1), bad) and same(torch.isnan(grad).any(1), bad)
    # a student that rules out all that is not listed still has an infinite loss
    z, t = normal(R, C, dtype, 95)
    z[0] = -INF
    z[0, :2] = 1.0
    idx = i32(np.tile([0, 1], (R, 1)))
    rows = _lib.lik_distill_rows(z, idx, val.zero_(), lse)[1]
    assert rows[0] == INF and torch.isfinite(rows[1:]).all()


@pytest.mark.parametrize("R,C,dtype", FORMS[:5])
def test_policy_kl_of_an_impossible_token(R, C, dtype):
    """exp(d) - d - 1 for a target that the student (d = inf) or the reference
    (d = -inf) rules out is infinite, not undefined."""
    say(f"[rows] policy KL of impossible tokens {R} x {C} {dtype}")
    z, t = normal(R, C, dtype, 93)
    z[2, int(t[2])] = -INF
    ref = torch.full((R,), -6.0, device="cuda")
    ref[3] = -INF
    old, adv = torch.full((R,), -5.0, device="cuda"), torch.ones(R, device="cuda")
    for kl in (0.1, -0.1):
        loss, rows, lp, grad = _lib.lik_policy_rows(z, t, old, adv, ref, kl_coef=kl)
        none = _lib.lik_policy_rows(z, t, old, adv, ref, kl_coef=kl, want_grad=False)
        assert lp[2] == -INF
        for l, r in ((loss, rows), none[:2]):
            assert l[0] == INF * kl
            assert same(torch.isinf(r), np.isin(np.arange(R), [2, 3]))
            assert r[2] == INF * kl and r[3] == INF * kl
        keep = [r for r in range(R) if r != 2]
        assert torch.isfinite(grad[keep]).all() and not torch.isfinite(grad[2, int(t[2])])


def test_host_threads_with_lists_of_several_lengths():
    """Calls from several host threads at once, each on a stream of its own, whose
    kernels are the same and whose lists need different amounts of LDS beyond the
    default: every call succeeds, with the results of the calls one by one."""
    say("[rows] host threads")
    made = []
    for R, C, dtype, K in ((256, 900, F32, 1024), (256, 900, F32, 1000), (256, 900, F32, 5),
                           (256, 70001, F32, 700), (256, 70001, F32, 650), (256, 70001, F32, 3)):
        z, t = normal(R, C, dtype, 91 + K)
        idx = torch.randint(0, C, (R, K), device="cuda", dtype=torch.int32)
        made.append((z, idx, torch.randn((R, K), device="cuda"),
                     torch.full((R,), 9.0, device="cuda")))
    want = [_lib.lik_distill_rows(*m) for m in made]
    torch.cuda.synchronize()
    got, errors = [[] for _ in made], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(40):
                    got[i] = _lib.lik_distill_rows(*made[i])
            s.synchronize()
        except Exception as e:                # reported below, by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(made))]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors, errors
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_sizes_beyond_the_library_are_refused_by_it():
    """2^31 columns or rows: the library's status and message, not an allocation
    of a workspace that has no size."""
    say("[rows] sizes beyond the library")
    for shape in ((1, 2 ** 31), (2 ** 31, 1)):
        z = torch.empty(shape, dtype=F16, device="cuda")
        R = shape[0]
        t = torch.empty(1, dtype=torch.int32, device="cuda").expand(R) if R == 1 else \
            torch.empty(R, dtype=torch.int32, device="cuda")
        f = torch.empty(R, dtype=F32, device="cuda")
        off, one = i32([0, 1]), i32([0])
        for call in (lambda: _lib.lik_logprob_rows_fwd(z, t),
                     lambda: _lib.lik_policy_rows(z, t, f, f, want_grad=False),
                     lambda: _lib.lik_distill_rows(z, t[:, None], f[:, None], want_grad=False),
                     lambda: _lib.lik_preference_rows(z, t, off, one, one, want_grad=False)):
            with pytest.raises(_lib.LikError, match="below 2\\^31") as e:
                call()
            assert e.value.status == _lib.LIK_ERR_UNSUPPORTED
        del z, t, f


def sum_bound(held, scale):
    """Error of ln Z as in rows_bounds, with what a kernel's thread sums at most:
    32 pieces of 8 columns, then trees over lanes, waves and parts whose factors
    are good to 4 U each, three of them."""
    q, _, _, _ = row_bounds(held, scale)
    y = np.asarray(held, dtype=np.float64) * scale
    x = np.minimum(y.max(1, keepdims=True) - y, 200.0)
    return U * (2 * (q * x).sum(1) + 4 + min(held.shape[1] / 64, 256) + 18 + 12)


# rows of an odd stride, so that they start at every alignment
LONG = [(130, 520, F32), (6, 9001, BF16), (128, 33001, F16), (128, 131007, BF16), (3, 140001, F16),
        (128, 100003, F32), (128, 200003, BF16), (2, 300007, F32)]


@pytest.mark.parametrize("R,C,dtype", LONG)
def test_row_sums_within_the_terms_of_a_thread(R, C, dtype):
    say(f"[rows] sums {R} x {C} {dtype}")
    rng = np.random.default_rng(R + C)
    dev, held = on_gpu((rng.standard_normal((R, C)) * 2).astype(np.float32), dtype, 3 + C % 2, 1)
    t = rng.integers(0, C, R)
    rl, rs = oracle.logprob_rows(held, t)
    tol = sum_bound(held, 1.0)
    logp, lse = _lib.lik_logprob_rows_fwd(dev, i32(t))
    within(host(logp), rl, logp_bound(rl, tol, np.abs(rl)), "logp")
    within(host(lse), rs, tol + 2 * U * np.abs(rs), "lse")
    zero = f32(np.zeros(R))
    for want in (True, False):
        lp = _lib.lik_policy_rows(dev, i32(t), zero, zero, want_grad=want)[2]
        within(host(lp), rl, logp_bound(rl, tol, np.abs(rl)), "policy logp")
    seq = _lib.lik_preference_rows(dev, i32(t), i32(np.arange(R + 1)), i32([0]), i32([1]))[2]
    within(host(seq), rl, logp_bound(rl, tol, np.abs(rl)), "preference logp")


@pytest.mark.parametrize("R,C,dtype", LONG)
def test_mass_in_the_first_and_last_columns(R, C, dtype):
    """Nearly all of a row's probability in the few columns before its first and
    behind its last aligned piece: one of them left out would change every sum."""
    say(f"[rows] edges {R} x {C} {dtype}")
    rng = np.random.default_rng(C)
    at = dict(pad=3 + C % 2, shift=1)
    z = np.full((R, C), -25.0, dtype=np.float32)
    edge = np.r_[0:8, C - 8:C]
    z[:, edge] = rng.uniform(-0.5, 0.5, (R, 16))
    t = edge[np.arange(R) % 16]
    t[R // 2] = C // 2
    dev, held = on_gpu(z, dtype, **at)
    rl, rs = oracle.logprob_rows(held, t)
    tol = sum_bound(held, 1.0)
    logp, lse = _lib.lik_logprob_rows_fwd(dev, i32(t))
    within(host(logp), rl, logp_bound(rl, tol, np.abs(rl)), "logp")
    within(host(lse), rs, tol + 2 * U * np.abs(rs), "lse")
    policy_case(z, t, dtype, 1.0, 96, **at)
    idx = np.stack([np.r_[edge[rng.permutation(16)[:5]], C // 3] for _ in range(R)])
    val = rng.standard_normal((R, 6)).astype(np.float32)
    for lse in (None, np.full(R, 4.0, dtype=np.float32)):
        distill_case(R, C, 6, lse is not None, dtype, 1.0, 97, idx=idx, val=val, lse=lse, z=z,
                     **at)


@pytest.mark.parametrize("op", ["logprob", "distill", "policy", "preference"])
@pytest.mark.parametrize("R,C,dtype", [(7, 100, F16), (7, 100, BF16), (40, 9001, BF16), (12, 20001, F16),
                                       (3, 131072, BF16), (130, 33001, F16)])
def test_gradient_of_16_bit_logits_against_differences(op, R, C, dtype):
    """The gradient of 16-bit logits along a direction against central differences
    of the loss of the same kernel.  Logits of at most 8 on a grid of 2 h, so that
    they and both steps are held exactly (h = 2^-4 takes 8 bits, 2^-6 takes 10).
    Off by the two losses' rounding over the step, by h^2 / 6 of a third derivative
    (along +-1 at most 2 of a log-softmax, 16 of a ratio, 17 of a pair of four rows:
    below 32 a row), and by half a step of every gradient entry."""
    say(f"[rows] differences {op} {R} x {C} {dtype}")
    h = 2.0 ** -4 if dtype == BF16 else 2.0 ** -6
    rng = np.random.default_rng(98)
    z = rng.standard_normal((R, C)).astype(np.float32) * 2
    t = rng.integers(0, C, R)
    z[np.arange(R), t] += 2
    z = np.clip(np.round(z / (2 * h)) * 2 * h, -8 + 2 * h, 8 - 2 * h)
    v = rng.choice([-1.0, 1.0], size=(R, C))
    old = oracle.logprob_rows(z, t)[0] - 0.1
    idx = rng.integers(0, C, size=(R, 4))
    val = rng.standard_normal((R, 4))
    one = f32(np.ones(R))

    def run(x, grad):
        dev, held = on_gpu(x.astype(np.float32), dtype)
        assert np.array_equal(held, x)
        if op == "logprob":
            lp, lse = _lib.lik_logprob_rows_fwd(dev, i32(t))
            return host(lp).sum(), _lib.lik_logprob_rows_bwd(dev, i32(t), lse, one) if grad else None
        if op == "distill":
            _, rows, g = _lib.lik_distill_rows(dev, i32(idx), f32(val), f32(np.full(R, 3.0)),
                                               row_weight=one, want_grad=grad)
            return host(rows).sum(), g
        if op == "policy":
            _, rows, _, g = _lib.lik_policy_rows(dev, i32(t), f32(old), one, clip_high=9.0, clip_low=1.0,
                                                 row_weight=one, want_grad=grad)
            return host(rows).sum(), g
        _, pairs, _, g = _lib.lik_preference_rows(dev, i32(t), i32([0, 1, min(R, 4)]), i32([0]),
                                                  i32([1]), beta=0.5, want_grad=grad)
        return host(pairs).sum(), g

    g = host(run(z, True)[1])
    up, down = run(z + h * v, False)[0], run(z - h * v, False)[0]
    size = R * (8 + np.log(C) + 1)
    tol = 2 * (20 + C / 64) * U * size / (2 * h) + h * h / 6 * R * 32
    tol += 1.02 * rounded(g, 0.0, dtype).sum()
    along = float(np.sum(g * v))
    assert abs((up - down) / (2 * h) - along) <= tol, (along, (up - down) / (2 * h), tol)
