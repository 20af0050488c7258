"""Steps of generation as a program runs them: lengths grow by the drafts, blocks
and slots come from the tables, keys and values are appended, attention runs over
the cache, drafts are verified, and lengths shrink to what was accepted; then the
policy loss takes what was generated.  Eager, captured and replayed, on another
stream, and on two at once."""

import numpy as np
import pytest
import torch

from maxsim_scoring_02_amd import _lib
from oracle import cache as oc
from parity import say
from test_gpu_cache import check_attention, host, i32
from test_gpu_verify import check as check_verify

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


class Program:
    """Requests, their cache on the GPU, and the buffers of a step."""

    def __init__(self, S, K, hq, hkv, dim, bs, N, width, C, dtype, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.K, self.bs, self.dims = gen, K, bs, (S, hq, hkv, dim, C, dtype)
        self.T = S * (K + 1)
        self.lens = torch.randint(1, 3 * bs, (S,), generator=gen, device="cuda", dtype=torch.int32)
        self.table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(N, generator=gen, device="cuda").int()
        self.ring_state = torch.tensor([0, N, 0, 0], dtype=torch.int32, device="cuda")
        self.k = torch.zeros((N, hkv, bs, dim), dtype=torch.uint8, device="cuda").view(_lib._F8)
        self.v = torch.zeros((N, hkv, dim, bs), dtype=torch.uint8, device="cuda").view(_lib._F8)
        self.ks, self.vs = torch.ones((2, N, hkv), device="cuda")
        self.head = torch.randn((hq * dim, C), generator=gen, device="cuda") * 0.3
        # the prompts
        new = self.lens.clone()
        most = int(new.sum())
        _, off, slots = self.tables(torch.zeros_like(new), new, most)
        _lib.lik_cache_append(self.normal(most, hkv, dim), self.normal(most, hkv, dim), slots, *self.cache)
        self.inputs()

    @property
    def cache(self):
        return self.k, self.v, self.ks, self.vs

    @property
    def state(self):
        return (self.lens, self.table, self.ring, self.ring_state, self.k.view(torch.uint8), self.v.view(torch.uint8),
                self.ks, self.vs)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(self.dims[-1])

    def tables(self, old, new, tokens):
        return _lib.lik_cache_tables(old, new, self.table, self.ring, self.ring_state, self.bs, tokens)

    def inputs(self):
        """New numbers in the step's buffers, which stay where they are."""
        S, hq, hkv, dim, C, dtype = self.dims
        new = {"q": self.normal(self.T, hq, dim) * 2, "k": self.normal(self.T, hkv, dim), "v": self.normal(self.T, hkv, dim),
               "d": self.normal(self.T, C).float(), "u": torch.rand(self.T, generator=self.gen, device="cuda"),
               "su": torch.rand(S, generator=self.gen, device="cuda"),
               "drafts": torch.randint(0, C, (self.T,), generator=self.gen, device="cuda").int()}
        if hasattr(self, "buf"):
            for name, x in new.items():
                self.buf[name].copy_(x)
        else:
            self.buf = new

    def step(self):
        b = self.buf
        granted, off, slots = self.tables(self.lens, self.lens + self.K + 1, self.T)
        _lib.lik_cache_append(b["k"], b["v"], slots, *self.cache)
        out, lse = _lib.lik_cache_attention(b["q"], off, granted, self.table, *self.cache, want_lse=True)
        logits = out.float().flatten(1) @ self.head
        tokens, accepted, logp = _lib.lik_verify_rows(logits, b["drafts"], off, b["u"], b["su"], draft_logits=b["d"])
        kept, _, _ = self.tables(granted, self.lens + accepted + 1, 0)
        self.lens.copy_(kept)
        return granted, off, slots, out, lse, logits, tokens, accepted, logp


def codes(x):
    return x.view(torch.uint8).cpu().numpy().copy()


@pytest.mark.parametrize("S,K,hq,hkv,dim,bs,dtype", [(5, 4, 8, 2, 64, 16, BF16), (1, 1, 4, 4, 128, 32, F16),
                                                     (19, 2, 6, 1, 64, 64, F32)])
def test_steps(S, K, hq, hkv, dim, bs, dtype):
    say(f"[generation] {S} requests, {K} drafts, {hq} / {hkv} heads, {dtype}")
    p = Program(S, K, hq, hkv, dim, bs, 30 + 8 * S, 20, 97, dtype, S)
    for step in range(4):
        lens = p.lens.cpu().numpy().astype(int)
        table, ring, state = (x.cpu().numpy().astype(int) for x in (p.table, p.ring, p.ring_state))
        k, v, ks, vs = codes(p.k), codes(p.v), host(p.ks), host(p.vs)
        granted, off, slots, out, lse, logits, tokens, accepted, logp = p.step()
        wg, wo, ws = oc.tables(lens, lens + K + 1, table, ring, state, bs, p.T)
        assert granted.tolist() == wg.tolist() and off.tolist() == wo.tolist() and slots.tolist() == ws.tolist()
        oc.append_part(host(p.buf["k"]), ws, k, ks)
        oc.append_part(host(p.buf["v"]), ws, v.transpose(0, 1, 3, 2), vs)
        assert np.array_equal(codes(p.k), k) and np.array_equal(codes(p.v), v)
        assert np.array_equal(host(p.ks), ks) and np.array_equal(host(p.vs), vs)
        want = oc.attention(host(p.buf["q"]), wo, wg, table, k, v, ks, vs, dim ** -0.5)[0]
        assert np.abs(host(out) - want).max() < 0.02 * np.abs(want).max()     # its bounds: test_gpu_cache.py
        check_verify(host(logits), host(p.buf["d"]), p.buf["drafts"].tolist(), wo, p.buf["u"].tolist(),
                     p.buf["su"].tolist(), 1.0, 1.0, (tokens, accepted, logp))
        oc.tables(wg, lens + accepted.cpu().numpy() + 1, table, ring, state, bs, 0)
        assert np.array_equal(p.table.cpu().numpy(), table) and np.array_equal(p.ring.cpu().numpy(), ring)
        assert p.ring_state.tolist() == state.tolist()
        assert p.lens.tolist() == (lens + accepted.cpu().numpy() + 1).tolist()
        # what was generated, as the policy loss takes it: a ratio of 1
        adv = torch.randn(p.T, device="cuda")
        _, row_loss, again, grad = _lib.lik_policy_rows(logits, tokens, logp, adv)
        emitted = tokens >= 0
        assert emitted.sum() == accepted.sum() + S
        assert torch.allclose(row_loss[emitted], -adv[emitted], rtol=1e-4, atol=1e-6)
        assert not row_loss[~emitted].any() and not grad[~emitted].any()
        p.inputs()


def test_a_pool_that_runs_out():
    """Requests that get no blocks write nothing, and the others' results stay right."""
    p = Program(6, 3, 4, 2, 64, 16, 22, 20, 50, BF16, 3)
    short = False
    for step in range(12):
        lens = p.lens.cpu().numpy()
        granted, off, slots, out, lse, logits, tokens, accepted, logp = p.step()
        short |= bool((granted.cpu().numpy() < lens + 4).any())
        at = off.tolist()
        for s, g in enumerate(granted.tolist()):
            mine = slots[at[s]:at[s + 1]].tolist()
            assert (min(mine) >= 0) == (g == lens[s] + 4) and (g == lens[s] + 4 or max(mine) == -1)
        check_attention(CacheView(p), p.buf["q"], np.array(at), granted.cpu().numpy(), TableOf(p, granted))
        p.lens.copy_(granted)                  # everything kept
        p.inputs()
    assert short


class CacheView:
    def __init__(self, p):
        self.parts = p.cache
        self.k, self.v, self.ks, self.vs = codes(p.k), codes(p.v), host(p.ks), host(p.vs)


def TableOf(p, lens):
    """The table as it stood for these lengths (shrinking took entries away)."""
    _lib.lik_cache_tables(p.lens, lens, p.table, p.ring, p.ring_state, p.bs, 0)
    return p.table.cpu().numpy()


def test_captured_and_replayed():
    eager = Program(7, 3, 8, 2, 64, 16, 90, 24, 300, BF16, 9)
    played = Program(7, 3, 8, 2, 64, 16, 90, 24, 300, BF16, 9)
    for a, b in zip(eager.state, played.state):
        assert torch.equal(a, b)
    keep = [x.clone() for x in played.state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        played.step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(played.state, keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = played.step()
    for replay in range(5):
        want = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
        for a, b in zip(eager.state, played.state):
            assert torch.equal(a, b)
        eager.inputs()
        for name, x in eager.buf.items():
            played.buf[name].copy_(x)
        torch.empty(1 << 20, device="cuda").normal_().sum().item()      # other work in between


def test_two_streams_at_once():
    """Programs of their own on two streams, and the same one after the other."""
    def make():
        return [Program(9, 4, 8, 2, 128, 16, 150, 24, 5000, BF16, s) for s in (1, 2)]

    apart, together = make(), make()
    want = [[p.step() for _ in range(4)] for p in apart]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in together]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, (p, s) in enumerate(zip(together, streams)):
            with torch.cuda.stream(s):
                got[i].append(p.step())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert all(torch.equal(i, j) for i, j in zip(x, y))
