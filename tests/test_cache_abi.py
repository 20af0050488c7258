"""Host-side checks of the 8-bit cache's C ABI (include/lik_cache.h), of
lik_verify_rows and of their binding: exports, refusals with their status, and
calls with nothing to do.  No GPU is needed."""

import ctypes

import pytest
import torch

from maxsim_scoring_02_amd import _lib
from maxsim_scoring_02_amd._lib import (LIK_BF16, LIK_ERR_INVALID_ARG, LIK_ERR_UNSUPPORTED,
                                        LIK_F16, LIK_F32, LIK_OK)

P = ctypes.c_void_p
MIS = P(0x100002)
BIG = ctypes.c_size_t(-1).value


def at(i):
    """Pointers far from each other, never dereferenced."""
    return P(0x10000000 * (i + 1))


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_exports_every_declared_function(L):
    names = _lib.header_functions(_lib.CACHE_HEADER_PATH)
    assert set(names) == set(_lib.CACHE_SIGNATURES)
    for n in names:
        assert hasattr(L, n)


CACHE = dict(k_cache=at(0), v_cache=at(1), k_scale=at(2), v_scale=at(3), num_blocks=6, kv_heads=2,
             block_size=16, dim=64, k_stride=2048, v_stride=2048)
ARGS = {
    "lik_cache_tables": dict(old_len=at(0), new_len=at(1), S=3, block_size=16, block_table=at(2),
                             max_blocks=4, table_ld=4, ring=at(3), num_blocks=9, ring_state=at(4),
                             granted=at(5), token_offsets=at(6), slots=at(7), T=20, stream=None),
    "lik_cache_append": dict(k=at(4), v=at(5), dtype=LIK_BF16, T=5, k_ld=128, v_ld=128, slots=at(6),
                             **CACHE, stream=None),
    "lik_cache_attention": dict(q=at(4), dtype=LIK_BF16, T=5, q_heads=4, q_ld=256, q_offsets=at(5),
                                kv_len=at(6), S=2, block_table=at(7), max_blocks=4, table_ld=4,
                                **CACHE, scale=0.1, out=at(8), out_ld=256, lse=None, ws=at(9),
                                wsb=1 << 27, stream=None),
    "lik_verify_rows": dict(logits=at(0), dtype=LIK_F32, R=4, C=8, ld=8, draft_logits=at(1),
                            draft_ld=8, draft_tokens=at(2), seq_offsets=at(3), S=2, scale=1.0,
                            draft_scale=1.0, accept_u=at(4), sample_u=at(5), tokens=at(6),
                            accepted=at(7), logp=at(8), ws=at(9), wsb=1 << 27, stream=None),
}


def call(L, name, **kw):
    a = dict(ARGS[name])
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(L, name)(*a.values())


INVALID = [
    ("lik_cache_tables", dict(S=-1), "negative"), ("lik_cache_tables", dict(T=-1), "negative"),
    ("lik_cache_tables", dict(num_blocks=-1), "negative"),
    ("lik_cache_tables", dict(max_blocks=-1), "negative"),
    ("lik_cache_tables", dict(table_ld=3), "table_ld 3"),
    ("lik_cache_tables", dict(S=1 << 40, table_ld=1 << 40), "overflows"),
    ("lik_cache_tables", dict(ring=at(0)), "overlaps"),
    ("lik_cache_tables", dict(granted=at(0)), "overlaps"),
    ("lik_cache_tables", dict(slots=P(at(2).value + 44)), "overlaps"),
    ("lik_cache_tables", dict(ring_state=P(at(3).value + 32)), "overlaps"),
    ("lik_cache_append", dict(T=-1), "negative"), ("lik_cache_append", dict(dtype=3), "dtype"),
    ("lik_cache_append", dict(kv_heads=0), "kv_heads"),
    ("lik_cache_append", dict(k_ld=127), "less than 128"),
    ("lik_cache_append", dict(v_ld=132), "multiple of 16 bytes"),
    ("lik_cache_append", dict(v_ld=1 << 60), "overflows"),
    ("lik_cache_append", dict(k=MIS), "aligned"), ("lik_cache_append", dict(v=MIS), "aligned"),
    ("lik_cache_append", dict(k=at(1)), "overlaps"), ("lik_cache_append", dict(k_scale=at(6)), "overlaps"),
    ("lik_cache_append", dict(v_cache=at(0)), "k_cache overlaps v_cache"),
    ("lik_cache_append", dict(v_cache=P(at(0).value + 1024), k_stride=4096, v_stride=4096),
     "k_cache overlaps v_cache"),
    ("lik_cache_append", dict(v_cache=P(at(0).value + 2048), k_stride=4096, v_stride=2048),
     "k_cache overlaps v_cache"),
    ("lik_cache_attention", dict(T=-1), "negative"), ("lik_cache_attention", dict(S=-1), "negative"),
    ("lik_cache_attention", dict(dtype=3), "dtype"),
    ("lik_cache_attention", dict(q_heads=3), "multiple of kv_heads"),
    ("lik_cache_attention", dict(q_heads=0), "multiple of kv_heads"),
    ("lik_cache_attention", dict(kv_heads=0), "kv_heads"),
    ("lik_cache_attention", dict(q_ld=255), "less than 256"),
    ("lik_cache_attention", dict(out_ld=260), "multiple of 16 bytes"),
    ("lik_cache_attention", dict(out=MIS), "aligned"), ("lik_cache_attention", dict(lse=MIS), "aligned"),
    ("lik_cache_attention", dict(out=at(4)), "overlaps"),
    ("lik_cache_attention", dict(out=P(at(4).value + 512)), "overlaps"),
    ("lik_cache_attention", dict(lse=at(8)), "overlaps"),
    ("lik_cache_attention", dict(out=at(0)), "overlaps"),
    ("lik_cache_attention", dict(table_ld=2), "table_ld 2"),
    ("lik_verify_rows", dict(S=-1), "negative"), ("lik_verify_rows", dict(draft_ld=7), "draft_ld 7"),
    ("lik_verify_rows", dict(draft_logits=MIS), "aligned"),
    ("lik_verify_rows", dict(draft_scale=0.0), "draft_scale"),
    ("lik_verify_rows", dict(draft_scale=float("nan")), "draft_scale"),
    ("lik_verify_rows", dict(tokens=at(2)), "overlaps"), ("lik_verify_rows", dict(logp=at(4)), "overlaps"),
    ("lik_verify_rows", dict(accepted=at(6)), "overlaps"),
    ("lik_verify_rows", dict(tokens=P(at(1).value + 124)), "overlaps"),
    ("lik_verify_rows", dict(logits=None), "NULL"), ("lik_verify_rows", dict(ld=7), "ld 7"),
    ("lik_verify_rows", dict(dtype=7), "dtype"), ("lik_verify_rows", dict(scale=float("inf")), "scale"),
]
for _n in ("lik_cache_append", "lik_cache_attention"):
    INVALID += [(_n, dict(block_size=b), "block_size") for b in (0, 8, 24, 512, -16)]
    INVALID += [(_n, dict(num_blocks=-1), "negative"), (_n, dict(k_stride=2047), "less than a block"),
                (_n, dict(v_stride=2032), "less than a block"), (_n, dict(k_stride=2056), "multiples of 16"),
                (_n, dict(num_blocks=1 << 20, k_stride=1 << 40), "overflows")]
for _s in ("nan", "inf", "0", "-1"):
    INVALID.append(("lik_cache_attention", dict(scale=float(_s)), "scale"))


@pytest.mark.parametrize("name,kw,msg", INVALID)
def test_refusals(L, name, kw, msg):
    assert call(L, name, **kw) == LIK_ERR_INVALID_ARG
    assert msg in L.lik_last_error().decode()


@pytest.mark.parametrize("name,kw,msg", [
    ("lik_cache_tables", dict(T=1 << 31), "T must"), ("lik_cache_tables", dict(num_blocks=1 << 27), "2^31"),
    ("lik_cache_tables", dict(S=(1 << 20) + 1), "2^20"),
    ("lik_cache_tables", dict(max_blocks=1 << 27, table_ld=1 << 27), "2^31"),
    ("lik_cache_append", dict(T=1 << 31), "T must"), ("lik_cache_append", dict(dim=96), "dim"),
    ("lik_cache_append", dict(kv_heads=1 << 16, k_stride=1 << 30, v_stride=1 << 30), "2^16"),
    ("lik_cache_append", dict(num_blocks=1 << 27), "2^31"),
    ("lik_cache_attention", dict(dim=80), "dim"), ("lik_cache_attention", dict(T=1 << 29), "T x q_heads"),
    ("lik_cache_attention", dict(S=(1 << 20) + 1), "2^20"),
    ("lik_cache_attention", dict(max_blocks=1 << 27, table_ld=1 << 27), "2^31"),
    ("lik_verify_rows", dict(R=1 << 31), "2^31"), ("lik_verify_rows", dict(S=1 << 31), "2^31"),
])
def test_what_is_not_supported(L, name, kw, msg):
    assert call(L, name, **kw) == LIK_ERR_UNSUPPORTED
    assert msg in L.lik_last_error().decode()


def test_appends_whose_tokens_pass_32_bits(L):
    """The kernel's numbers of tokens are 32 bits, with a look at what follows them."""
    for T in (2 ** 31 - 2 ** 8, 2 ** 31 - 127, 2 ** 31 - 1):
        assert call(L, "lik_cache_append", T=T, k_ld=128, v_ld=128, v=P(1 << 44), slots=P(1 << 45),
                    k=P(1 << 46)) == LIK_ERR_UNSUPPORTED
        assert "T must be below 2^31 - 2^8" in L.lik_last_error().decode()


@pytest.mark.parametrize("name,fields", [
    ("lik_cache_tables", ["old_len", "new_len", "block_table", "ring", "ring_state", "granted",
                          "token_offsets", "slots"]),
    ("lik_cache_append", ["k", "v", "slots", "k_cache", "v_cache", "k_scale", "v_scale"]),
    ("lik_cache_attention", ["q", "q_offsets", "kv_len", "block_table", "k_cache", "v_cache", "k_scale",
                             "v_scale", "out"]),
    ("lik_verify_rows", ["draft_tokens", "seq_offsets", "accept_u", "sample_u", "tokens", "accepted",
                         "logp"]),
])
def test_required_pointers(L, name, fields):
    for f in fields:
        assert call(L, name, **{f: None}) == LIK_ERR_INVALID_ARG
        assert f + " is NULL" in L.lik_last_error().decode()
        assert call(L, name, **{f: MIS}) == LIK_ERR_INVALID_ARG
        assert "aligned" in L.lik_last_error().decode()


def test_workspaces(L):
    w = L.lik_cache_workspace_bytes
    for sizes in ((-1, 2, 4, 2, 64, LIK_F16), (5, -1, 4, 2, 64, LIK_F16), (5, 2, 3, 2, 64, LIK_F16),
                  (5, 2, 4, 0, 64, LIK_F16), (5, 2, 4, 2, 65, LIK_F16), (5, 2, 4, 2, 64, 3),
                  (1 << 40, 2, 4, 2, 64, LIK_F16)):
        assert w(*sizes) == BIG
    assert w(0, 2, 4, 2, 64, LIK_F16) == 0
    need = w(5, 2, 4, 2, 64, LIK_BF16)
    assert need < 1 << 27
    if need:
        for kw in (dict(ws=None), dict(wsb=need - 1)):
            assert call(L, "lik_cache_attention", **kw) == LIK_ERR_INVALID_ARG
            assert "workspace too small" in L.lik_last_error().decode()
        assert call(L, "lik_cache_attention", ws=P(at(9).value + 4)) == LIK_ERR_INVALID_ARG
    r = L.lik_rows_workspace_bytes
    assert r(_lib.LIK_ROWS_VERIFY, 4, 8, -1, LIK_F32, 1) == BIG and r(_lib.LIK_ROWS_VERIFY, 0, 8, 1, LIK_F32, 1) == 0
    need = r(_lib.LIK_ROWS_VERIFY, 4, 8, 2, LIK_F32, 1)
    if need:
        for kw in (dict(ws=None), dict(wsb=need - 1)):
            assert call(L, "lik_verify_rows", **kw) == LIK_ERR_INVALID_ARG
            assert "workspace too small" in L.lik_last_error().decode()


def test_calls_with_nothing_to_do(L):
    no = {k: None for k, v in ARGS["lik_cache_append"].items() if isinstance(v, P)}
    assert call(L, "lik_cache_append", T=0) == LIK_OK
    assert call(L, "lik_cache_append", num_blocks=0, **no) == LIK_OK
    no = {k: None for k, v in ARGS["lik_cache_attention"].items() if isinstance(v, P)}
    assert call(L, "lik_cache_attention", T=0, num_blocks=0, **no) == LIK_OK
    no = {k: None for k, v in ARGS["lik_verify_rows"].items() if isinstance(v, P)}
    assert call(L, "lik_verify_rows", R=0, **no) == LIK_OK


@pytest.mark.parametrize("name", sorted(ARGS))
def test_a_sound_call_reaches_the_device_check(L, name):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; the pointers are not real")
    assert call(L, name) == LIK_ERR_UNSUPPORTED
    assert "device" in L.lik_last_error().decode()
    if name in ("lik_cache_append", "lik_cache_attention"):   # keys and values in one array
        assert call(L, name, v_cache=P(at(0).value + 2048), k_stride=4096,
                    v_stride=4096) == LIK_ERR_UNSUPPORTED
        assert "device" in L.lik_last_error().decode()


def test_binding_refuses_before_the_library(monkeypatch):
    def no_library():
        raise AssertionError("the library was reached")

    monkeypatch.setattr(_lib, "lib", no_library)
    i, f, f8 = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 64), torch.zeros(4, 2, 16, 64).to(_lib._F8)
    sc, table = torch.ones(4, 2), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        _lib.lik_cache_tables(i, i, table, i, i, 16, 4)
    with pytest.raises(ValueError, match="GPU"):
        _lib.lik_cache_append(f, f, i, f8, f8.mT.contiguous(), sc, sc)
    with pytest.raises(ValueError, match="GPU"):
        _lib.lik_cache_attention(f, i, i[:2], table, f8, f8.mT.contiguous(), sc, sc)
    with pytest.raises(ValueError, match="GPU"):
        _lib.lik_verify_rows(torch.zeros(3, 5), i, i[:2], i, i)


def test_binding_checks_shapes_strides_and_types():
    dev = torch.device("cpu")
    i = torch.zeros(6, dtype=torch.int32)
    assert _lib._ints(i, (6,), "x", dev) is i and _lib._ints(i[::2], (3,), "x", dev).stride() == (1,)
    for bad, msg in ((i[:5], "shape"), (i.long(), "int32")):
        with pytest.raises(ValueError, match=msg):
            _lib._ints(bad, (6,), "x", dev)
    with pytest.raises(ValueError, match="contiguous"):
        _lib._in_place(i[::2], (3,), "ring", dev)
    table = torch.zeros(3, 8, dtype=torch.int32)
    assert _lib._table(table[:, :5], 3, dev) == (5, 8)
    for bad in (table.long(), table[:2], i):
        with pytest.raises(ValueError, match="block_table"):
            _lib._table(bad, 3, dev)
    with pytest.raises(ValueError, match="overlap"):
        _lib._table(table[:1].expand(3, 8), 3, dev)
    kv = torch.zeros(5, 2, 2, 16, 64).to(_lib._F8)
    k, v, s = kv[:, 0], kv[:, 1].reshape(5, 2, 64, 16), torch.ones(5, 2)
    got = _lib._blocks(k, v, s, s, dev)
    assert got[4:] == (5, 2, 16, 64, 4096, 4096)
    assert _lib._blocks(k[:1], v[:1], s[:1], s[:1], dev)[8:] == (2048, 2048)
    bads = [(k.view(torch.uint8), v, s, s, "float8"), (k, v.mT, s, s, "shape"),
            (k, v.mT.contiguous().mT, s, s, "dense"), (k.transpose(0, 1), v, s, s, "shape"),
            (k, v, s[:4], s, "k_scale"), (k, v, s, s.half(), "v_scale"), (k, v, s, s.mT.contiguous().mT, "v_scale")]
    for a, b, c, d, msg in bads:
        with pytest.raises(ValueError, match=msg):
            _lib._blocks(a, b, c, d, dev)
    qkv = torch.zeros(4, 3, 2, 64)
    assert _lib._token_stride(qkv[:, 1], 2, 64, "k") == 384 and _lib._token_stride(qkv[:1, 1], 2, 64, "k") == 128
    for bad, msg in ((qkv[:, 1].transpose(0, 1), "shape"), (qkv[:, :, 0], "shape"),
                     (qkv[:1, 1].expand(4, 2, 64), "overlap"), (qkv.flatten(1)[:, ::3].view(4, 2, 64), "dense")):
        with pytest.raises(ValueError, match=msg):
            _lib._token_stride(bad, 2, 64, "k")
