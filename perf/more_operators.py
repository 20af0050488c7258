"""A step of generation, as it is measured: cases, inputs, plain forms and 64-bit values.

* verify   drafted tokens accepted or turned down by the target's probabilities, from given random numbers
* tables   block tables and slot maps of a paged cache, from the lengths of its requests
* append   tokens written to a cache held in 8 bits, with a scale for each block and head
* attend   causal attention of ragged queries over such a cache
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
#: scales are powers of two within these
SCALE_MIN, SCALE_MAX = 2.0 ** -40, 2.0 ** 40


def listed():
    return [
        # one answer, four drafted tokens: what the latency of a single user's step is made of
        {"name": "verify-one", "op": "verify", "seqs": 1, "drafts": 4, "ragged": False, "cols": 32768, "dtype": "bf16",
         "scale": 1.0, "drafter": True},
        # drafts copied from the prompt (no drafter's probabilities), of any length, over an odd vocabulary
        {"name": "verify-copied", "op": "verify", "seqs": 61, "drafts": 7, "ragged": True, "cols": 50001,
         "dtype": "f16", "scale": 1.3, "drafter": False},
        # a batch of rollouts over a large vocabulary
        {"name": "verify-batch", "op": "verify", "seqs": 256, "drafts": 4, "ragged": False, "cols": 131072,
         "dtype": "bf16", "scale": 1.0, "drafter": True},
        # every request of a batch takes five tokens more, and gives them back
        {"name": "tables-step", "op": "tables", "seqs": 64, "old": 8192, "new": 5, "block": 16},
        # a thousand prompts come in, and leave
        {"name": "tables-prompts", "op": "tables", "seqs": 1000, "old": 0, "new": 4096, "block": 32},
        # one token of every request of a batch
        {"name": "append-step", "op": "append", "seqs": 64, "new": 1, "hkv": 8, "dim": 128, "block": 16,
         "dtype": "bf16"},
        # prompts of all lengths
        {"name": "append-prompts", "op": "append", "seqs": 9, "new": 4096, "hkv": 8, "dim": 128, "block": 64,
         "dtype": "f16"},
        # one request with a page's 1030 tokens
        {"name": "attend-one", "op": "attend", "seqs": 1, "new": 1, "len": 1030, "hq": 32, "hkv": 8, "dim": 128,
         "block": 16, "dtype": "bf16"},
        # a batch of answers, one token each
        {"name": "attend-batch", "op": "attend", "seqs": 64, "new": 1, "len": 8192, "hq": 32, "hkv": 8, "dim": 128,
         "block": 16, "dtype": "bf16"},
        # drafts verified over long documents
        {"name": "attend-drafts", "op": "attend", "seqs": 16, "new": 5, "len": 32768, "hq": 20, "hkv": 4, "dim": 64,
         "block": 32, "dtype": "f16"},
        # one head of keys and values for all, in float32
        {"name": "attend-f32", "op": "attend", "seqs": 7, "new": 3, "len": 4000, "hq": 8, "hkv": 1, "dim": 256,
         "block": 64, "dtype": "f32"},
        # parts of prompts behind what the cache holds of them
        {"name": "attend-prompts", "op": "attend", "seqs": 3, "new": 2048, "len": 8192, "hq": 32, "hkv": 8,
         "dim": 128, "block": 16, "dtype": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["verify", "tables", "append", "attend", "attend"])
    if op == "verify":
        cols = spread(60, 150000)
        seqs = spread(1, 256)
        drafts = max(1, min(rng.randint(1, 9), 160_000_000 // (seqs * cols) - 1))
        return {"op": op, "seqs": seqs, "drafts": drafts, "ragged": rng.random() < 0.5, "cols": cols,
                "dtype": rng.choice(["f16", "bf16", "f32"]), "scale": rng.choice([1.0, 0.7, 1.4]),
                "drafter": rng.random() < 0.7}
    block = rng.choice([16, 32, 64, 128])
    if op == "tables":
        old = rng.choice([0, spread(1, 8192)])
        return {"op": op, "seqs": spread(1, 1000), "old": old, "new": spread(1, 4096 if old == 0 else 64),
                "block": block}
    dtype, dim = rng.choice(["f16", "bf16", "bf16", "f32"]), rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        seqs = spread(1, 128)
        return {"op": op, "seqs": seqs, "new": spread(1, max(1, 8000000 // (seqs * hkv * dim))), "hkv": hkv,
                "dim": dim, "block": block, "dtype": dtype}
    seqs, group = spread(1, 64), rng.choice([1, 2, 3, 4, 5, 8])
    most = max(64, 300_000_000 // (seqs * hkv * dim))
    length = spread(17, min(32768, most))
    new = rng.choice([1, 1, rng.randint(2, 9), spread(16, 1024)])
    new = max(1, min(new, length, 900_000_000 // (seqs * hkv * group * length)))
    return {"op": op, "seqs": seqs, "new": new, "len": length, "hq": hkv * group, "hkv": hkv, "dim": dim,
            "block": block, "dtype": dtype}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

class _Gen:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device="cuda")

    def perm(self, n):
        return torch.randperm(n, generator=self.gen, device="cuda")

    def ints(self, lo, hi, n):
        """n whole numbers within [lo, hi]."""
        return torch.randint(lo, hi + 1, (n,), generator=self.gen, device="cuda")

    def shares(self, n):
        """n numbers spread evenly over (0, 1), in any order: their sum is the same for every seed."""
        return ((self.perm(n) + 0.5) / n).double()


def prepare(case, seed):
    g = _Gen(seed)
    make = {"verify": _make_verify, "tables": _make_tables, "append": _make_append, "attend": _make_attend}
    return {"case": case} | make[case["op"]](case, g)


def _starts(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)])


def _softmax64(x, scale):
    y = x.double() * scale
    e = torch.exp(y - y.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _make_verify(case, g):
    S, K, C, scale = case["seqs"], case["drafts"], case["cols"], case["scale"]
    dtype = DTYPES[case["dtype"]]
    counts = ((K + 1) * g.shares(S)).long() if case["ragged"] else torch.full((S,), K, device="cuda")
    offsets = _starts(counts + 1)
    R = int(offsets[-1])
    last = torch.zeros(R, dtype=torch.bool, device="cuda")
    last[offsets[1:] - 1] = True
    logits = torch.empty((R, C), device="cuda", dtype=dtype).normal_(0, 2.5, generator=g.gen)
    drafts = torch.empty(R, dtype=torch.int64, device="cuda")
    p_x = torch.empty(R, dtype=torch.float64, device="cuda")
    q_x = torch.ones_like(p_x)
    draft_logits = torch.empty_like(logits) if case["drafter"] else None
    step = max(1, 2 ** 25 // C)
    for r in range(0, R, step):
        b = slice(r, min(R, r + step))
        rows = torch.arange(b.stop - b.start, device="cuda")
        z = logits[b]
        if case["drafter"]:  # a drafter that is off by some noise, and draws from what it finds
            draft_logits[b] = (z.float() + 0.5 * g.normal(*z.shape)).to(dtype)
            q = _softmax64(draft_logits[b], scale)
        else:                # copied tokens: mostly likely ones
            at = g.ints(0, C - 1, len(z))
            z[rows, at] += (8 + 3 * g.normal(len(z))).to(dtype)
            logits[b] = z
            q = None
        if q is not None:
            c = q.cumsum(1)
            at = torch.searchsorted(c, (g.uniform(len(z), 1).double() * c[:, -1:]).contiguous())[:, 0].clamp(max=C - 1)
            q_x[b] = q[rows, at]
        p_x[b] = _softmax64(z, scale)[rows, at]
        drafts[b] = at
    u = g.uniform(R).double()
    # none next to the border, where rounding decides
    u = torch.where((u * q_x / p_x - 1).abs() < 1e-3, u * 0.99, u)
    taken = (u * q_x < p_x) & ~last
    stop = torch.where(taken, R, torch.arange(R, device="cuda"))
    ends = torch.stack([stop[a:b].min() for a, b in zip(offsets[:-1].tolist(), offsets[1:].tolist())])
    sample = torch.empty(S, device="cuda")
    for s in range(0, S, step):  # the middle of the interval of a token that is not among the rarest
        at = ends[s:s + step]
        w = _softmax64(logits[at], scale)
        more = ~last[at]
        if case["drafter"]:
            w = torch.where(more[:, None], (w - _softmax64(draft_logits[at], scale)).clamp(min=0), w)
        else:
            rows = torch.arange(len(at), device="cuda")
            w[rows, drafts[at]] = torch.where(more, 0.0, w[rows, drafts[at]])
        c = w.cumsum(1)
        total = c[:, -1:]
        likely = torch.where(w >= torch.minimum(1e-4 * total, 0.5 * w.amax(1, keepdim=True)), w, 0.0)
        lc = likely.cumsum(1)
        t = torch.searchsorted(lc, (g.uniform(len(at), 1).double() * lc[:, -1:]).contiguous()).clamp(max=C - 1)
        sample[s:s + step] = ((c.gather(1, t) - 0.5 * w.gather(1, t)) / total)[:, 0].float()
    return {"logits": logits, "draft_logits": draft_logits, "drafts": torch.where(last, -1, drafts).int(),
            "offsets": offsets.int(), "u": u.float(), "sample": sample}


def _make_tables(case, g):
    S, bs = case["seqs"], case["block"]
    old = (case["old"] * (0.25 + 0.75 * g.shares(S))).long()
    # prompts are mostly short and now and then long; a step is the same for all
    new = old + ((case["new"] * g.shares(S) ** 3).long() + 1 if case["old"] == 0 else case["new"])
    most = new.sort().values
    leave = S // 5 if case["old"] else 0
    new[g.perm(S)[:leave]] = 0  # some requests are at their end
    have, need = (old + bs - 1) // bs, (new + bs - 1) // bs
    width = int(most[-1]) // bs + 2
    N = int((most // bs + 1).sum()) + 4
    ids = g.perm(N)
    used = int(have.sum())
    at = torch.arange(width, device="cuda")[None]
    table = torch.where(at < have[:, None], ids[(_starts(have)[:-1, None] + at).clamp(max=N - 1)], -1)
    ring = torch.full((N,), -1, device="cuda")
    ring[:N - used] = ids[used:]
    return {"old": old.int(), "new": new.int(), "table": table.int().contiguous(), "ring": ring.int(),
            "ring_state": torch.tensor([0, N - used, 0, 0], dtype=torch.int32, device="cuda"),
            "tokens": int((new - old).clamp(min=0).sum()),
            # room for the longest requests to come back, whichever left
            "back": int((most[S - leave:] if leave else (old - new).clamp(min=0)).sum())}


def _blocks(x, dims):
    """(codes, scales) of blocks of values [N, Hkv, ...]."""
    scale = _scale_of(x.abs().amax(dims))
    return (x / scale[..., None, None]).to(F8), scale


def _scale_of(amax):
    """The smallest power of two with amax <= 448 times it."""
    m, e = torch.frexp(amax / F8_MAX)
    one = torch.ones((), device=amax.device, dtype=amax.dtype)
    s = torch.ldexp(one, torch.where(m == 0.5, e - 1, e))
    return torch.where(amax == 0, SCALE_MIN, s.clamp(SCALE_MIN, SCALE_MAX))


def _cache(g, N, hkv, bs, dim):
    """A cache of N blocks whose heads and channels are of different sizes, as keys' are."""
    k_cache = torch.empty((N, hkv, bs, dim), dtype=F8, device="cuda")
    v_cache = torch.empty((N, hkv, dim, bs), dtype=F8, device="cuda")
    k_scale = torch.empty((N, hkv), device="cuda")
    v_scale = torch.empty((N, hkv), device="cuda")
    head = torch.exp(0.5 * g.normal(2, hkv, 1, 1))
    channel = torch.exp(0.3 * g.normal(dim))
    step = max(1, 2 ** 26 // (hkv * bs * dim))
    for n in range(0, N, step):
        m = min(N, n + step) - n
        k = g.normal(m, hkv, bs, dim) * head[0] * channel
        v = g.normal(m, hkv, dim, bs) * head[1]
        (k_cache[n:n + m], k_scale[n:n + m]), (v_cache[n:n + m], v_scale[n:n + m]) = _blocks(k, (2, 3)), _blocks(v, (2, 3))
    return {"k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale, "head": head,
            "channel": channel}


def _make_append(case, g):
    S, hkv, dim, bs = case["seqs"], case["hkv"], case["dim"], case["block"]
    dtype = DTYPES[case["dtype"]]
    if case["new"] == 1:
        counts, first = torch.ones(S, dtype=torch.int64, device="cuda"), g.ints(0, 4 * bs, S)
    else:
        counts = (case["new"] * g.shares(S)).long() + 1
        first = torch.where(g.uniform(S) < 0.5, 0, g.ints(0, 2 * bs, S))
    T = int(counts.sum())
    blocks = (first + counts + bs - 1) // bs
    N = T // bs + (4 if case["new"] == 1 else 3) * S + 5
    ids, base = g.perm(N), _starts(blocks)
    s = torch.repeat_interleave(torch.arange(S, device="cuda"), counts)
    p = first[s] + torch.arange(T, device="cuda") - _starts(counts)[s]
    state = _cache(g, N, hkv, bs, dim)
    # a part of a row that holds queries, keys and values
    qkv = torch.empty((T, 3, hkv, dim), device="cuda", dtype=dtype)
    qkv[:, 1] = (g.normal(T, hkv, dim) * state["head"][0, :, 0] * state["channel"]).to(dtype)
    qkv[:, 2] = (g.normal(T, hkv, dim) * state["head"][1, :, 0]).to(dtype)
    qkv[:, 0] = 0
    return state | {"k": qkv[:, 1], "v": qkv[:, 2], "slots": (ids[base[s] + p // bs] * bs + p % bs).int()}


def _make_attend(case, g):
    S, hq, hkv, dim, bs = (case[k] for k in ("seqs", "hq", "hkv", "dim", "block"))
    n = torch.full((S,), case["new"], device="cuda")
    if case["new"] > 16:  # parts of prompts of any size
        n = (case["new"] * (0.3 + 0.7 * g.shares(S))).long().clamp(min=1)
    lens = (case["len"] * (0.25 + 0.75 * g.shares(S))).long()
    if S == 1:
        lens[0] = case["len"]
    lens = torch.maximum(lens, n)
    blocks = (lens + bs - 1) // bs
    N = int(blocks.sum()) + 2
    ids, base = g.perm(N), _starts(blocks)
    at = torch.arange(int(blocks.max()), device="cuda")[None]
    table = torch.where(at < blocks[:, None], ids[(base[:-1, None] + at).clamp(max=N - 1)], -1)
    state = _cache(g, N, hkv, bs, dim)
    T = int(n.sum())
    size = 1.6 / (state["head"][0, :, 0] * state["channel"].square().mean().sqrt())
    q = g.normal(T, hkv, hq // hkv, dim) * size[:, None]
    return state | {"q": q.view(T, hq, dim).to(DTYPES[case["dtype"]]), "q_offsets": _starts(n).int(),
                    "lens": lens.int(), "table": table.int().contiguous()}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _calls(state) if own else _plain(state)


def _calls(state):
    import maxsim_scoring_02_amd as lik

    case = state["case"]
    if case["op"] == "verify":
        tokens, accepted, logp = lik.lik_verify_rows(
            state["logits"], state["drafts"], state["offsets"], state["u"], state["sample"],
            draft_logits=state["draft_logits"], scale=case["scale"], draft_scale=case["scale"])
        return {"tokens": tokens, "accepted": accepted, "logp": logp}
    if case["op"] == "tables":
        return _two_tables(state, lik.lik_cache_tables)
    cache = [state[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")]
    if case["op"] == "append":
        lik.lik_cache_append(state["k"], state["v"], state["slots"], *cache)
        return _written(state)
    out, _ = lik.lik_cache_attention(state["q"], state["q_offsets"], state["lens"], state["table"], *cache)
    return {"out": out}


def _two_tables(state, call):
    """A step's lengths and back again, so that a pass can follow a pass."""
    pool = (state["table"], state["ring"], state["ring_state"], state["case"]["block"])
    granted, offsets, slots = call(state["old"], state["new"], *pool, state["tokens"])
    back, back_offsets, back_slots = call(granted, state["old"], *pool, state["back"])
    return {"granted": granted, "offsets": offsets, "slots": slots, "back": back, "back_offsets": back_offsets,
            "back_slots": back_slots, "table": state["table"], "ring": state["ring"], "state": state["ring_state"]}


def _written(state):
    return {k: state[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain(state):
    op = state["case"]["op"]
    if op == "verify":
        return _plain_verify(state)
    if op == "tables":
        return _two_tables(state, _plain_tables)
    if op == "append":
        _plain_append(state["k"], state["slots"], state["k_cache"], state["k_scale"])
        _plain_append(state["v"], state["slots"], state["v_cache"].mT, state["v_scale"])
        return _written(state)
    return _plain_attend(state)


def _plain_softmax(x, scale):
    y = x.float() * scale
    top = y.amax(1, keepdim=True)
    e = torch.exp(y - top)
    total = e.sum(1, keepdim=True)
    return y, e / total, top + torch.log(total)


def _plain_verify(state):
    case, z, d = state["case"], state["logits"], state["draft_logits"]
    R, C = z.shape
    x = state["drafts"].long().clamp(min=0)[:, None]
    offsets = state["offsets"].long()
    rows = torch.arange(R, device=z.device)
    y, p, lse = _plain_softmax(z, case["scale"])
    q = None if d is None else _plain_softmax(d, case["scale"])[1]
    q_x = torch.ones_like(lse) if q is None else q.gather(1, x)
    taken = ((state["u"].double()[:, None] * q_x < p.gather(1, x)) & (state["drafts"] >= 0)[:, None])[:, 0]
    seq = torch.searchsorted(offsets, rows, right=True) - 1
    # the first row of each sequence whose token is not taken
    end = torch.full_like(offsets[1:], R).scatter_reduce_(0, seq, torch.where(taken, R, rows), "amin")
    drafted = state["drafts"][end] >= 0
    w = p[end]
    if q is None:
        w = torch.where(drafted[:, None] & (torch.arange(C, device=z.device) == x[end]), 0.0, w)
    else:
        w = torch.where(drafted[:, None], (w - q[end]).clamp(min=0), w)
    # sums of a whole vocabulary in 64 bits: a token's interval is narrow
    c = w.double().cumsum(1)
    drawn = torch.searchsorted(c, (state["sample"].double()[:, None] * c[:, -1:]).contiguous(), right=True)
    tokens = torch.where(rows < end[seq], state["drafts"].long(), -1)
    tokens[end] = drawn[:, 0].clamp(max=C - 1)
    logp = torch.where(tokens >= 0, (y.gather(1, tokens.clamp(min=0)[:, None]) - lse)[:, 0], 0.0)
    return {"tokens": tokens.int(), "accepted": (end - offsets[:-1]).int(), "logp": logp}


def _plain_tables(old, new, table, ring, state, bs, tokens):
    S, W = table.shape
    N = len(ring)
    old, new = old.long().clamp(0, W * bs), new.long().clamp(min=0)
    have, need = (old + bs - 1) // bs, (new + bs - 1) // bs
    fits = need <= W
    ask = torch.where(fits, (need - have).clamp(min=0), 0)
    give = torch.where(fits, (have - need).clamp(min=0), 0)
    upto = ask.cumsum(0)
    head, count = state[0].long(), state[1].long()
    ok = fits & ((ask == 0) | (upto <= count))
    offsets = _starts((new - old).clamp(min=0))
    at = torch.arange(W, device=table.device)[None]
    fresh = ok[:, None] & (at >= have[:, None]) & (at < need[:, None])
    gone = ok[:, None] & (at >= need[:, None]) & (at < have[:, None])
    came = ring[(head + (upto - ask)[:, None] + at - have[:, None]) % N]
    to = (head + count + (give.cumsum(0) - give)[:, None] + at - need[:, None]) % N
    ring.copy_(torch.cat([ring, ring[:1]]).scatter_(0, torch.where(gone, to, N).flatten(), table.flatten())[:N])
    table.copy_(torch.where(fresh, came, torch.where(gone, -1, table)))
    taken = torch.where(ok, ask, 0).sum()
    state[0] = (head + taken) % N
    state[1] = count - taken + torch.where(ok, give, 0).sum()
    i = torch.arange(tokens, device=table.device)
    s = torch.searchsorted(offsets[1:], i, right=True).clamp(max=S - 1)
    p = old[s] + i - offsets[s]
    block = table[s, (p // bs).clamp(max=W - 1)].long()
    slots = torch.where(ok[s] & (i < offsets[-1]) & (block >= 0), block * bs + p % bs, -1)
    return torch.where(ok, new, old).int(), offsets.int(), slots.int()


def _plain_append(x, slots, cache, scale):
    """cache [N, Hkv, bs, dim], of any strides"""
    N, hkv, bs, dim = cache.shape
    block, at = slots.long() // bs, slots.long() % bs
    x = x.float()
    amax = torch.zeros_like(scale).scatter_reduce_(0, block[:, None].expand(-1, hkv), x.abs().amax(2), "amax")
    touched, fresh = torch.zeros((2, N), dtype=torch.bool, device=x.device)
    touched[block] = True
    fresh[block[at == 0]] = True
    needed = _scale_of(amax)
    now = torch.where(fresh[:, None], needed, torch.maximum(scale, needed))
    now = torch.where(touched[:, None], now, scale)
    which = (touched & ~fresh).nonzero()[:, 0]
    codes = cache.view(torch.uint8)
    was = codes[which].view(F8).float()
    codes[which] = (was * (scale / now)[which][..., None, None]).to(F8).view(torch.uint8)
    scaled = (x / now[block][..., None]).clamp(-F8_MAX, F8_MAX)
    codes[block, :, at] = scaled.to(F8).view(torch.uint8)
    scale.copy_(now)


def _plain_attend(state):
    q, lens = state["q"], state["lens"].long()
    T, hq, dim = q.shape
    S, hkv = len(lens), state["k_scale"].shape[1]
    offsets = state["q_offsets"].long()
    n = offsets.diff()
    table = state["table"].long().clamp(min=0)

    def values(cache, scale):
        blocks = cache.view(torch.uint8)[table].view(F8).float() * scale[table][..., None, None]
        return blocks.transpose(1, 2)

    k = values(state["k_cache"], state["k_scale"]).flatten(2, 3)
    v = values(state["v_cache"], state["v_scale"]).mT.flatten(2, 3).contiguous()
    most = int(state["case"]["new"])
    at = torch.arange(most, device=q.device)
    rows = (offsets[:-1, None] + at).clamp(max=T - 1)
    qp = q[rows].float().view(S, most, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = torch.matmul(qp, k.mT.contiguous()) / math.sqrt(dim)
    pos = (lens - n)[:, None] + at
    seen = torch.arange(k.shape[2], device=q.device) <= pos[..., None]
    s = s.view(S, hkv, hq // hkv, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(S, hkv, -1, s.shape[-1]), v).view(S, hkv, hq // hkv, most, dim) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(S, most, hq, dim)
    return {"out": o[at < n[:, None]].to(q.dtype)}


def work(case):
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        K = case["drafts"] / (2 if case["ragged"] else 1)
        rows = case["seqs"] * (K + 1) + (case["seqs"] * K if case["drafter"] else 0)
        return {"bytes": rows * case["cols"] * size + case["seqs"] * (20 * K + 28), "flops": 4 * rows * case["cols"]}
    S, bs = case["seqs"], case["block"]
    if case["op"] == "tables":
        new = case["new"] / 4 if case["old"] == 0 else case["new"]
        blocks = new / bs + 1
        return {"bytes": S * (4 * new + 24 + 24 * blocks), "flops": S * new}
    if case["op"] == "append":
        size = 4 if case["dtype"] == "f32" else 2
        tokens = S * (1 if case["new"] == 1 else 1 + case["new"] / 2)
        values = 2 * tokens * case["hkv"] * case["dim"]
        return {"bytes": values * (size + 1) + 4 * tokens, "flops": 2 * values}
    size = 4 if case["dtype"] == "f32" else 2
    n = case["new"] * (0.65 if case["new"] > 16 else 1)
    seen = max(0.625 * case["len"], n)
    pairs = S * n * max(seen - n / 2, n / 2)
    return {"bytes": 2 * S * seen * case["hkv"] * (case["dim"] + 4 / bs) + 2 * S * n * case["hq"] * case["dim"] * size,
            "flops": 4 * pairs * case["hq"] * case["dim"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers alone
    s = prepare(case, seed)
    return {"verify": _exact_verify, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_verify(s):
    z, d, scale = s["logits"], s["draft_logits"], s["case"]["scale"]
    logp = torch.zeros(len(z), dtype=torch.float64, device="cuda")
    bounds, drafts = s["offsets"].tolist(), s["drafts"].tolist()
    u, sample = s["u"].tolist(), s["sample"].tolist()
    for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
        ls = torch.log_softmax(z[a:b].double() * scale, 1)
        lq = None if d is None else torch.log_softmax(d[a:b].double() * scale, 1)
        x = torch.tensor(drafts[a:b - 1], dtype=torch.int64, device="cuda")
        at = torch.arange(b - a - 1, device="cuda")
        chance = (ls[at, x] - (0 if d is None else lq[at, x])).exp().tolist()
        n = next((j for j, c in enumerate(chance) if u[a + j] >= c), b - a - 1)
        rest = ls[n].exp()
        if n < b - a - 1:
            if d is None:
                rest[drafts[a + n]] = 0
            else:
                rest = torch.relu(rest - lq[n].exp())
        rest = rest.cumsum(0)
        token = int((rest <= sample[i] * rest[-1]).sum())
        logp[a:a + n] = ls[at[:n], x[:n]]
        logp[a + n] = ls[n, token]
    return {"tokens": None, "accepted": None, "logp": logp}


def _exact_append(s):
    """Codes as the numbers that they stand for, before their rounding."""
    out = {}
    slots = s["slots"].cpu()
    bs = s["case"]["block"]
    block, at = (slots // bs).tolist(), (slots % bs).tolist()
    runs = {}
    for t, b in enumerate(block):
        runs.setdefault(b, []).append(t)
    if len(runs) > 3000:
        return None
    for name, x in (("k", s["k"]), ("v", s["v"])):
        cache, scale = s[name + "_cache"].to(torch.float64), s[name + "_scale"].double()
        cache = cache.mT.contiguous() if name == "v" else cache
        for b, tokens in runs.items():
            new = x[tokens[0]:tokens[-1] + 1].double()
            top = new.abs().amax((0, 2)) / F8_MAX
            need = torch.exp2(torch.ceil(torch.log2(top))).clamp(SCALE_MIN, SCALE_MAX)
            if at[tokens[0]] > 0:
                need = torch.maximum(need, scale[b])
                cache[b] *= (scale[b] / need)[:, None, None]
            scale[b] = need
            cache[b][:, at[tokens[0]]:at[tokens[-1]] + 1] = (new / need[:, None]).transpose(0, 1)
        out[name + "_cache"] = cache.mT.contiguous() if name == "v" else cache
        out[name + "_scale"] = scale
    return {k: out[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _exact_attend(s):
    case, q = s["case"], s["q"]
    group, bs, dim = case["hq"] // case["hkv"], case["block"], case["dim"]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    bounds = s["q_offsets"].tolist()
    for i, length in enumerate(s["lens"].tolist()):
        a, b = bounds[i], bounds[i + 1]
        ids = s["table"][i, :(length + bs - 1) // bs].long()
        hidden = torch.ones(b - a, length, device="cuda", dtype=torch.bool).triu(length - (b - a) + 1)
        for h in range(case["hkv"]):
            k = (s["k_cache"][:, h].view(torch.uint8)[ids].view(F8).double() * s["k_scale"][ids, h, None, None].double())
            v = (s["v_cache"][:, h].view(torch.uint8)[ids].view(F8).double() * s["v_scale"][ids, h, None, None].double())
            k, v = k.reshape(-1, dim)[:length], v.transpose(1, 2).reshape(-1, dim)[:length]
            for j in range(h * group, (h + 1) * group):
                w = (q[a:b, j].double() @ k.T) * dim ** -0.5
                out[a:b, j] = torch.softmax(w.masked_fill_(hidden, -math.inf), 1) @ v
    return {"out": out}
