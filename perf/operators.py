"""The row losses over logits, as they are measured: cases, inputs, plain forms and 64-bit values.

Operators (R rows of C logits each, y = scale * logits, q = softmax of a row of y):

* logprob     log-probabilities of one column a row, forward and backward
* distill     KL divergence from a teacher known by its top logits, with its gradient
* policy      clipped policy loss with a KL term, with its gradient
* preference  loss on paired log ratios of whole sequences, with its gradient
"""

import math

import torch

own = False

SIGMOID, HINGE, SQUARE = 0, 1, 2
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
#: float16 gradients are kept off the smallest numbers, as in training
LOSS_SCALE = 4096.0
#: of the rows that carry a target, the share that is ignored (prompts, padding)
IGNORED = 0.125


def listed():
    return [
        # a few answers scored against a language model's whole vocabulary, token by token
        {"name": "logprob-fwd-few", "op": "logprob_fwd", "rows": 8, "cols": 131072, "dtype": "bf16", "scale": 1.0},
        # the reference model's log-probabilities of a batch of rollouts
        {"name": "logprob-fwd-batch", "op": "logprob_fwd", "rows": 4096, "cols": 100003, "dtype": "bf16", "scale": 1.0},
        # a user's own loss on log-probabilities: its gradient comes in, the logits' goes out
        {"name": "logprob-bwd-batch", "op": "logprob_bwd", "rows": 2048, "cols": 50001, "dtype": "f16", "scale": 0.7},
        # 256 queries with 16 candidates each, every candidate ranked by the teacher
        {"name": "distill-candidates", "op": "distill", "rows": 256, "cols": 16, "top": 16, "tail": False,
         "dtype": "f32", "scale": 1.0},
        # scores of 256 queries against 1000 documents, a teacher's 32 best with what it leaves to the others
        {"name": "distill-documents", "op": "distill", "rows": 256, "cols": 1000, "top": 32, "tail": True,
         "dtype": "f32", "scale": 0.5},
        # a language model taught from stored top logits
        {"name": "distill-vocabulary", "op": "distill", "rows": 4096, "cols": 65536, "top": 64, "tail": True,
         "dtype": "bf16", "scale": 0.5},
        # a short rollout over an odd vocabulary
        {"name": "policy-few", "op": "policy", "rows": 61, "cols": 100003, "dtype": "bf16", "scale": 1.0, "kl": 0.05},
        # a batch of rollouts with float32 logits
        {"name": "policy-f32", "op": "policy", "rows": 1024, "cols": 32001, "dtype": "f32", "scale": 1.0, "kl": 0.0},
        # a large batch of rollouts over a large vocabulary
        {"name": "policy-batch", "op": "policy", "rows": 4096, "cols": 131072, "dtype": "bf16", "scale": 1.0,
         "kl": 0.05},
        # search sessions: every step ranks 300 documents, one positive session against negatives
        {"name": "preference-sessions", "op": "preference", "rows": 120, "cols": 300, "seqs": 16, "pairs": 15,
         "kind": SIGMOID, "mean": False, "dtype": "f32", "scale": 1.0},
        # pairs of short answers
        {"name": "preference-answers", "op": "preference", "rows": 1999, "cols": 32768, "seqs": 16, "pairs": 8,
         "kind": SIGMOID, "mean": False, "dtype": "f16", "scale": 1.0},
        # pairs of long answers over a large vocabulary
        {"name": "preference-long", "op": "preference", "rows": 4096, "cols": 100000, "seqs": 16, "pairs": 8,
         "kind": SQUARE, "mean": True, "dtype": "bf16", "scale": 1.0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logprob_fwd", "logprob_bwd", "distill", "policy", "preference"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    cols = spread(12, 150000)
    size = 2 if dtype != "f32" else 4
    rows = spread(1, max(1, min(8192, 2 ** 30 // (cols * size))))
    case = {"op": op, "dtype": dtype, "scale": rng.choice([1.0, 1.0, 0.5, 2.0]), "cols": cols, "rows": rows}
    if op == "distill":
        case["top"] = spread(1, min(cols, 256))
        case["tail"] = case["top"] < cols and rng.random() < 0.5
    elif op == "policy":
        case["kl"] = rng.choice([0.0, 0.02, 0.1])
    elif op == "preference":
        case["rows"] = rows = max(rows, 4)
        case["seqs"] = spread(2, min(64, rows // 2))
        case["pairs"] = spread(1, 64)
        case["kind"] = rng.choice([SIGMOID, HINGE, SQUARE])
        case["mean"] = rng.random() < 0.3
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, C, scale = case["rows"], case["cols"], case["scale"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    logits = torch.empty((R, C), device="cuda", dtype=DTYPES[case["dtype"]]).normal_(0, 2.5, generator=gen)
    rows = torch.arange(R, device="cuda")
    state = {"case": case, "logits": logits}
    loss_scale = LOSS_SCALE if case["dtype"] == "f16" else 1.0
    if case["op"] == "distill":
        K = case["top"]
        # K columns of every row, none twice, that the student ranks high too
        width = C // K
        idx = torch.arange(K, device="cuda") * width + (uniform(R, K) * width).long().clamp_(max=width - 1)
        lift = 4 + 3 * normal(R, K)
        logits.scatter_add_(1, idx, lift.to(logits.dtype))
        val = logits.gather(1, idx).float() + 0.7 * normal(R, K)
        idx = idx.int()
        if K > 4:  # some lists are shorter
            short = uniform(R, K) < 0.03
            short[:, 0] = False
            idx[short] = -1
        state |= {"idx": idx, "val": val, "t_lse": None,
                  "weight": None if loss_scale == 1 else torch.full((R,), loss_scale / R, device="cuda")}
        if case["tail"]:
            listed_lse = torch.logsumexp(torch.where(idx >= 0, val.double() * scale, -math.inf), 1)
            state["t_lse"] = (listed_lse + 0.02 + 0.4 * uniform(R)).float()
        return state

    targets = torch.randint(0, C, (R,), generator=gen, device="cuda")
    # what was sampled is mostly what the model finds likely
    logits[rows, targets] += (7 + 2 * normal(R)).to(logits.dtype)
    ignored = torch.zeros(R, dtype=torch.bool, device="cuda")
    if R >= 8:
        ignored[torch.randperm(R, generator=gen, device="cuda")[:int(R * IGNORED)]] = True
    state["targets"] = torch.where(ignored, -1, targets).int()
    if case["op"] == "logprob_fwd":
        return state
    lse = torch.empty(R, device="cuda", dtype=torch.float64)
    step = max(1, 2 ** 25 // C)
    for r in range(0, R, step):
        lse[r:r + step] = torch.logsumexp(logits[r:r + step].double() * scale, 1)
    logp = torch.where(ignored, 0.0, logits[rows, targets].double() * scale - lse)
    if case["op"] == "logprob_bwd":
        state |= {"lse": torch.where(ignored, 0.0, lse).float(), "g": normal(R) * (loss_scale / R)}
    elif case["op"] == "policy":
        drift = 0.25 * normal(R).double()
        # none next to the borders of the clip, where a gradient jumps
        for border in (math.log(0.8), math.log(1.28)):
            drift = torch.where((drift - border).abs() < 1e-3, border + 2e-3, drift)
        state |= {"old": (logp - drift).float(), "adv": normal(R), "ref": None,
                  "weight": torch.where(ignored, 0.0, loss_scale) / max(1, R - int(ignored.sum()))}
        if case["kl"]:
            state["ref"] = (logp + 0.2 * normal(R)).float()
    else:
        S, P = case["seqs"], case["pairs"]
        # S sequences of ragged lengths, one token at least, and padding behind the last
        end = R - R // 64
        cuts = torch.randperm(end - 1, generator=gen, device="cuda")[:S - 1].sort().values + 1
        offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), end)])
        total = torch.cat([logp.new_zeros(1), logp.cumsum(0)])[offsets].diff()
        if case["mean"]:
            total = total / _tokens(state["targets"], offsets)
        chosen = torch.randint(0, S, (P,), generator=gen, device="cuda")
        rejected = (chosen + torch.randint(1, S, (P,), generator=gen, device="cuda")) % S
        beta = 0.5 if case["mean"] else 0.1
        ref = (total + normal(S) / beta).float()
        if case["kind"] == HINGE:  # none next to the hinge, where the gradient jumps
            drop = (total - ref.double())
            h = beta * (drop[chosen] - drop[rejected])
            rejected = torch.where((h - 1).abs() < 1e-3, chosen, rejected)
        state |= {"offsets": offsets.int(), "chosen": chosen.int(), "rejected": rejected.int(), "ref": ref,
                  "beta": beta, "weight": loss_scale * (0.5 + uniform(P))}
    return state


def _tokens(targets, offsets):
    """How many tokens with a target each sequence has, one at least."""
    seen = torch.cat([targets.new_zeros(1, dtype=torch.int64), (targets >= 0).cumsum(0)])
    return seen[offsets.long()].diff().clamp_(min=1)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _calls(state) if own else _plain(state)


def _calls(state):
    import maxsim_scoring_02_amd as lik

    case, z = state["case"], state["logits"]
    op, scale = case["op"], case["scale"]
    if op == "logprob_fwd":
        logp, lse = lik.lik_logprob_rows_fwd(z, state["targets"], scale=scale)
        return {"logp": logp, "lse": lse}
    if op == "logprob_bwd":
        return {"grad": lik.lik_logprob_rows_bwd(z, state["targets"], state["lse"], state["g"], scale=scale)}
    if op == "distill":
        loss, row_loss, grad = lik.lik_distill_rows(z, state["idx"], state["val"], teacher_lse=state["t_lse"],
                                                    scale=scale, row_weight=state["weight"])
        return {"loss": loss, "row_loss": row_loss, "grad": grad}
    if op == "policy":
        loss, row_loss, logp, grad = lik.lik_policy_rows(
            z, state["targets"], state["old"], state["adv"], ref_logp=state["ref"], scale=scale, clip_low=0.2,
            clip_high=0.28, kl_coef=case["kl"], row_weight=state["weight"])
        return {"loss": loss, "row_loss": row_loss, "logp": logp, "grad": grad}
    loss, pair_loss, seq_logp, grad = lik.lik_preference_rows(
        z, state["targets"], state["offsets"], state["chosen"], state["rejected"], ref_logp=state["ref"],
        kind=case["kind"], beta=state["beta"], mean_logp=case["mean"], scale=scale, pair_weight=state["weight"])
    return {"loss": loss, "pair_loss": pair_loss, "seq_logp": seq_logp, "grad": grad}


def _plain(state):
    case, z = state["case"], state["logits"]
    op, scale = case["op"], case["scale"]
    R, C = z.shape
    y = z.float() * scale
    if op == "distill":
        return _plain_distill(state, y)
    valid = state["targets"] >= 0
    t = state["targets"].long().clamp(min=0)[:, None]
    if op == "logprob_bwd":
        q = torch.exp(y - state["lse"][:, None])
        return {"grad": _plain_grad(z, q, t, torch.where(valid, state["g"] * scale, 0.0))}
    top = y.amax(1, keepdim=True)
    e = torch.exp(y - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    logp = torch.where(valid, (y.gather(1, t) - lse)[:, 0], 0.0)
    if op == "logprob_fwd":
        return {"logp": logp, "lse": torch.where(valid, lse[:, 0], 0.0)}
    q = e / total
    if op == "policy":
        adv, w = state["adv"], state["weight"]
        ratio = torch.exp(logp - state["old"])
        low, high = 0.8, 1.28
        loss = -torch.minimum(ratio * adv, ratio.clamp(low, high) * adv)
        flows = torch.where(adv >= 0, ratio <= high, ratio >= low)
        slope = torch.where(flows, -ratio * adv, 0.0)
        if state["ref"] is not None:
            away = state["ref"] - logp
            loss = loss + case["kl"] * (torch.exp(away) - away - 1)
            slope = slope + case["kl"] * (1 - torch.exp(away))
        loss = torch.where(valid, loss, 0.0)
        coef = torch.where(valid, w * slope * scale, 0.0)
        return {"loss": (w.double() * loss).sum(0, keepdim=True).float(), "row_loss": loss, "logp": logp,
                "grad": _plain_grad(z, q, t, coef)}
    # preference: sums over whole sequences in 64 bits
    offsets, beta, w = state["offsets"].long(), state["beta"], state["weight"].double()
    count = _tokens(state["targets"], offsets) if case["mean"] else torch.ones_like(offsets[1:])
    seq = torch.cat([logp.new_zeros(1, dtype=torch.float64), logp.double().cumsum(0)])[offsets].diff() / count
    c, r = state["chosen"].long(), state["rejected"].long()
    off = seq - state["ref"].double()
    delta = off[c] - off[r]
    h = beta * delta
    if case["kind"] == SIGMOID:
        loss, slope = torch.log1p(torch.exp(-h.abs())) + (-h).clamp(min=0), -beta / (1 + torch.exp(h))
    elif case["kind"] == HINGE:
        loss, slope = (1 - h).clamp(min=0), torch.where(h < 1, -beta, 0.0).double()
    else:
        loss, slope = (delta - 0.5 / beta) ** 2, 2 * (delta - 0.5 / beta)
    per_seq = torch.zeros_like(seq).index_add_(0, c, w * slope).index_add_(0, r, -w * slope) / count
    rows = torch.arange(R, device=z.device)
    at = torch.searchsorted(offsets, rows, right=True) - 1
    inside = valid & (at >= 0) & (at < len(seq))
    coef = torch.where(inside, per_seq[at.clamp(0, len(seq) - 1)] * scale, 0.0).float()
    return {"loss": (w * loss).sum(0, keepdim=True).float(), "pair_loss": loss.float(), "seq_logp": seq.float(),
            "grad": _plain_grad(z, q, t, coef)}


def _plain_grad(z, q, t, coef):
    """coef * ([c = t] - q), rounded to the logits' type; rows of coefficient 0 are 0."""
    g = -q * coef[:, None]
    g = g.scatter_add(1, t, coef[:, None])
    return g.to(z.dtype)


def _plain_distill(state, y):
    case, z = state["case"], state["logits"]
    scale, R = case["scale"], y.shape[0]
    there = state["idx"] >= 0
    idx = state["idx"].long().clamp(min=0)
    tv = torch.where(there, state["val"] * scale, -math.inf)
    if state["t_lse"] is None:
        high = tv.amax(1, keepdim=True)
        t_lse = high + torch.log(torch.exp(tv - high).sum(1, keepdim=True))
    else:
        t_lse = state["t_lse"][:, None]
    p = torch.exp(tv - t_lse)
    top = y.amax(1, keepdim=True)
    e = torch.exp(y - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    row_loss = torch.where(there, p * (tv - t_lse - (y.gather(1, idx) - lse)), 0.0).sum(1)
    mass = p.new_zeros(R, 1).add(1.0)
    p_cols = torch.zeros_like(y).scatter_add_(1, idx, p)
    if state["t_lse"] is None:
        g = e / total - p_cols
    else:
        is_listed = torch.zeros_like(y).scatter_add_(1, idx, there.float()) > 0
        p_sum = p.double().sum(1, keepdim=True)
        p_tail = (1 - p_sum).clamp(min=0).float()
        mass = torch.maximum(p_sum.float(), mass)
        rest = torch.where(is_listed, 0.0, e).sum(1, keepdim=True)
        row_loss = row_loss + (p_tail * (torch.log(p_tail) - torch.log(rest) + torch.log(total)))[:, 0]
        g = torch.where(is_listed, mass * e / total - p_cols, e * (mass / total - p_tail / rest))
    w = p.new_full((R,), 1.0 / R) if state["weight"] is None else state["weight"]
    return {"loss": (row_loss.double() * w).sum(0, keepdim=True).float(), "row_loss": row_loss,
            "grad": (g * (w * scale)[:, None]).to(z.dtype)}


def work(case):
    R, C = case["rows"], case["cols"]
    size = 4 if case["dtype"] == "f32" else 2
    # ignored rows are not read; every gradient row is written
    read = R if case["op"] == "distill" or R < 8 else R - int(R * IGNORED)
    grad = case["op"] != "logprob_fwd"
    more = {"distill": 8 * R * case.get("top", 0) + 8 * R, "policy": 32 * R, "preference": 8 * R}.get(case["op"], 16 * R)
    return {"bytes": (read + (R if grad else 0)) * C * size + more, "flops": (4 + 3 * grad) * read * C}


# ---------------------------------------------------------------------------
# the definition in 64 bits, some rows at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    z, scale, R, C = s["logits"], case["scale"], case["rows"], case["cols"]
    step = max(1, 2 ** 24 // C)
    blocks = [slice(r, min(R, r + step)) for r in range(0, R, step)]
    grad = None if case["op"] == "logprob_fwd" else torch.empty((R, C), dtype=torch.float64, device="cuda")
    if case["op"] == "distill":
        row_loss = torch.empty(R, dtype=torch.float64, device="cuda")
        for b in blocks:
            row_loss[b], grad[b] = _exact_distill(s, b, scale)
        w = torch.full_like(row_loss, 1.0 / R) if s["weight"] is None else s["weight"].double()
        return {"loss": (w @ row_loss)[None], "row_loss": row_loss, "grad": grad.mul_(w[:, None])}

    t = s["targets"].long()
    valid = t >= 0
    if case["op"] == "logprob_bwd":
        for b in blocks:
            g = -torch.exp(z[b].double() * scale - s["lse"][b, None].double())
            at = torch.nonzero(valid[b])[:, 0]
            g[at, t[b][at]] += 1
            grad[b] = g * (s["g"][b].double() * scale * valid[b])[:, None]
        return {"grad": grad}

    logp = torch.zeros(R, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(logp)
    for b in blocks:
        ls = torch.log_softmax(z[b].double() * scale, 1)
        at = torch.nonzero(valid[b])[:, 0]
        logp[b][at] = ls[at, t[b][at]]
        lse[b] = (z[b, 0].double() * scale - ls[:, 0]) * valid[b]
    if case["op"] == "logprob_fwd":
        return {"logp": logp, "lse": lse}
    if case["op"] == "policy":
        x = logp.clone().requires_grad_()
        adv, w = s["adv"].double(), s["weight"].double()
        ratio = (x - s["old"].double()).exp()
        row_loss = -torch.where(adv > 0, torch.clamp(ratio, max=1 + 0.28), torch.clamp(ratio, min=1 - 0.2)) * adv
        if s["ref"] is not None:
            d = s["ref"].double() - x
            row_loss = row_loss + case["kl"] * (torch.expm1(d) - d)
        row_loss = torch.where(valid, row_loss, torch.zeros_like(row_loss))
        loss = (row_loss * w).sum()
        loss.backward()
        slope, out = x.grad, {"loss": loss.detach()[None], "row_loss": row_loss.detach(), "logp": logp}
    else:
        x = logp.clone().requires_grad_()
        bounds = s["offsets"].tolist()
        parts = [x[a:b].sum() / (max(1, int(valid[a:b].sum())) if case["mean"] else 1)
                 for a, b in zip(bounds, bounds[1:])]
        seq = torch.stack(parts)
        beta, off = s["beta"], seq - s["ref"].double()
        delta = off[s["chosen"].long()] - off[s["rejected"].long()]
        if case["kind"] == SIGMOID:
            pair_loss = torch.nn.functional.softplus(-beta * delta, threshold=700)
        elif case["kind"] == HINGE:
            pair_loss = torch.relu(1 - beta * delta)
        else:
            pair_loss = (delta - 1 / (2 * beta)).square()
        loss = (pair_loss * s["weight"].double()).sum()
        loss.backward()
        slope = x.grad * valid
        out = {"loss": loss.detach()[None], "pair_loss": pair_loss.detach(), "seq_logp": seq.detach()}
    for b in blocks:
        g = -torch.softmax(z[b].double() * scale, 1)
        at = torch.nonzero(valid[b])[:, 0]
        g[at, t[b][at]] += 1
        grad[b] = g * (slope[b] * scale)[:, None]
    return out | {"grad": grad}


def _exact_distill(s, b, scale):
    """Row losses and their gradients (of the plain sum) of the rows in `b`."""
    x = s["logits"][b].double().requires_grad_()
    ls = torch.log_softmax(x * scale, 1)
    there = s["idx"][b] >= 0
    col = torch.where(there, s["idx"][b].long(), 0)
    tv = torch.where(there, s["val"][b].double() * scale, -math.inf)
    lt = torch.log_softmax(tv, 1) if s["t_lse"] is None else tv - s["t_lse"][b, None].double()
    p = lt.exp()
    row = (p * torch.where(there, lt - ls.gather(1, col), 0.0)).nan_to_num(0.0).sum(1)
    if s["t_lse"] is not None:
        p_tail = (1 - p.sum(1)).clamp(min=0)
        open_ = torch.ones_like(x).scatter_reduce(1, col, torch.where(there, 0.0, 1.0).to(x), "prod") > 0
        q_tail = torch.logsumexp(torch.where(open_, ls, -math.inf), 1)
        row = row + p_tail * (p_tail.log() - q_tail)
    row.sum().backward()
    return row.detach(), x.grad
