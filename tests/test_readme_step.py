"""The step of generation that the readme shows, run as it stands there: on the CPU over
the oracle, and on the GPU over the library, with a pool that cannot serve every request.
A request that got no blocks keeps its length, its blocks and its tokens."""

import os
import re
import types

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F8 = torch.float8_e4m3fn


def step_of_readme():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    block = re.search(r"^    # a step of generation.*?(?=^\S|\Z)", text, re.M | re.S).group(0)
    return "\n".join(line[4:] for line in block.splitlines())


def oracle_library():
    """The library's calls of a step on CPU tensors."""
    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32)

    def codes(x):
        return x.view(torch.uint8).numpy()

    def tables(old, new, table, ring, state, block_size, tokens):
        return tuple(map(ints, oc.tables(old.numpy(), new.numpy(), table.numpy(), ring.numpy(), state.numpy(), block_size, tokens)))

    def append(k, v, slots, kc, vc, ks, vs):
        oc.append_part(k.numpy(), slots.tolist(), codes(kc), ks.numpy())
        oc.append_part(v.numpy(), slots.tolist(), codes(vc).transpose(0, 1, 3, 2), vs.numpy())

    def attention(q, off, lens, table, kc, vc, ks, vs):
        out, lse = oc.attention(q.numpy(), off.numpy(), lens.numpy(), table.numpy(), codes(kc), codes(vc), ks.numpy(),
                                vs.numpy(), q.shape[2] ** -0.5)
        return torch.tensor(out).to(q.dtype), None

    def verify(logits, drafts, off, u, su, draft_logits=None):
        t, a, p = oracle.verify_rows(logits.numpy(), drafts.tolist(), off.tolist(), u.tolist(), su.tolist(),
                                     None if draft_logits is None else draft_logits.numpy())
        return ints(t), ints(a), torch.tensor(p, dtype=torch.float32)

    return types.SimpleNamespace(lik_cache_tables=tables, lik_cache_append=append, lik_cache_attention=attention,
                                 lik_verify_rows=verify)


def run_steps(lik, dev):
    code = compile(step_of_readme(), "README.md", "exec")
    gen = torch.Generator().manual_seed(5)
    S, K, hq, hkv, dim, bs, N, C = 4, 3, 4, 2, 64, 16, 9, 40
    kc = torch.zeros((N, hkv, bs, dim), dtype=torch.uint8, device=dev).view(F8)
    vc = torch.zeros((N, hkv, dim, bs), dtype=torch.uint8, device=dev).view(F8)
    ks, vs = torch.ones((2, N, hkv), device=dev)
    cache = kc, vc, ks, vs
    table = torch.full((S, 6), -1, dtype=torch.int32, device=dev)
    ring = torch.randperm(N, generator=gen).int().to(dev)
    state = torch.tensor([0, N, 0, 0], dtype=torch.int32, device=dev)

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(dev)

    # 14 tokens each, and 30 of the last: five of nine blocks
    start = torch.tensor([14, 15, 14, 30], dtype=torch.int32, device=dev)
    lens, _, slots = lik.lik_cache_tables(torch.zeros_like(start), start, table, ring, state, bs, 73)
    lik.lik_cache_append(normal(73, hkv, dim), normal(73, hkv, dim), slots, *cache)
    env = {"lik": lik, "torch": torch, "K": K, "S": S, "table": table, "ring": ring, "ring_state": state, "cache": cache,
           "len": lens}
    short = 0
    for _ in range(25):
        T = S * (K + 1)
        env |= {"k": normal(T, hkv, dim), "v": normal(T, hkv, dim), "q": normal(T, hq, dim), "logits": normal(T, C),
                "d": normal(T, C), "drafts": torch.randint(0, C, (T,), generator=gen).int().to(dev),
                "u": torch.rand(T, generator=gen).to(dev), "u_draw": torch.rand(S, generator=gen).to(dev)}
        before = env["len"].tolist()
        rows = table.tolist()
        free = int(state[1])
        kept = [[kc.view(torch.uint8)[b].clone() for b in row if b >= 0] for row in rows]
        exec(code, env)
        after, accepted = env["len"].tolist(), env["accepted"].tolist()
        slots = env["slots"].tolist()
        need = 0
        for s in range(S):
            ask = -(-(before[s] + K + 1) // bs) - -(-before[s] // bs)
            need += ask
            got = ask == 0 or need <= free
            mine = slots[s * (K + 1):(s + 1) * (K + 1)]
            assert (min(mine) >= 0) == got
            if got:
                assert after[s] == before[s] + 1 + accepted[s]
                continue
            short += 1
            assert after[s] == before[s], "a request that got no blocks lost or won tokens"
            assert table[s].tolist() == rows[s]
            for b, x in zip(rows[s], kept[s]):
                assert torch.equal(kc.view(torch.uint8)[b], x)
        # every block is in one table or free
        used = [b for row in table.tolist() for b in row if b >= 0]
        head, count = state.tolist()[:2]
        free_now = [ring.tolist()[(head + i) % N] for i in range(count)]
        assert sorted(used + free_now) == list(range(N))
        assert [sum(b >= 0 for b in row) for row in table.tolist()] == [-(-x // bs) for x in after]
    assert short > 10


def test_the_step_over_the_oracle():
    run_steps(oracle_library(), torch.device("cpu"))


@pytest.mark.gpu
def test_the_step_on_the_gpu():
    import maxsim_scoring_02_amd as lik
    run_steps(lik, torch.device("cuda:0"))
