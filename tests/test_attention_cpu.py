"""The attention operators without a GPU: the oracle's own pins, argument
checks of the binding, and the library's validation before any launch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attention_ref as ref

import w8a8_int8_quantized_rmsnorm_b200 as cr


@pytest.fixture(scope="module")
def lib():
    from w8a8_int8_quantized_rmsnorm_b200 import build, _capi
    build.build()
    return _capi.load()


# ------------------------------------------------------------------ oracle
def test_rotation_turns_pairs_and_keeps_the_rest():
    x = np.random.default_rng(0).standard_normal((3, 2, 64))
    table = ref.rope_table(9, 32)
    y, _ = ref.norm_rotate(x, None, table, [0, 4, 8], 0.0)
    assert np.array_equal(y[0], x[0])                       # position 0 turns nothing
    assert np.array_equal(y[..., 32:], x[..., 32:])         # past the rotation's width
    for i in range(16):
        z = (x[1, 0, i] + 1j * x[1, 0, i + 16]) * (float(table[4, i]) + 1j * float(table[4, i + 16]))
        assert abs(y[1, 0, i] - z.real) < 1e-12 and abs(y[1, 0, i + 16] - z.imag) < 1e-12


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    table = ref.rope_table(200, 64)
    dots = []
    for shift in (0, 7, 150):
        a, _ = ref.norm_rotate(q, None, table, [20 + shift], 0.0)
        b, _ = ref.norm_rotate(k, None, table, [3 + shift], 0.0)
        dots.append((a * b).sum())
    assert np.allclose(dots, dots[0], rtol=0, atol=1e-5)    # the table is fp32


def test_head_norm_of_a_constant_row():
    y, _ = ref.norm_rotate(np.full((1, 1, 64), -3.0), np.full(64, 0.5), ref.rope_table(1, 64), [0], 0.0)
    assert np.allclose(y, -1.5, rtol=0, atol=1e-12)


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((5, 8))
    o, _ = ref.attention(np.zeros((2, 8)), rng.standard_normal((5, 8)), v, 1.0,
                         np.array([[1, 1, 0, 0, 1], [0, 0, 0, 0, 0]], bool))
    assert np.allclose(o[0], v[[0, 1, 4]].mean(0))          # equal scores: the mean
    assert not o[1].any()                                   # sees nothing: zero
    k = np.eye(8)[:5]
    o, _ = ref.attention(np.eye(8)[3:4] * 1e4, k, v, 1.0, np.ones((1, 5), bool))
    assert np.allclose(o[0], v[3])                          # one key takes all
    v[4] = np.nan
    o, _ = ref.attention(np.ones((1, 8)), k, v, 1.0, np.arange(5)[None] < 4)
    assert np.isfinite(o).all()


def test_packed_rows_see_their_own_past_only():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 7, 2, 8))
    o, _ = ref.packed_attention(q, k, v, [0, 3, 7], [0, 3, 7], 1.0, True)
    assert np.allclose(o[0], v[0]) and np.allclose(o[3], v[3])
    k2, v2 = k.copy(), v.copy()
    k2[6], v2[6] = 9, 9
    o2, _ = ref.packed_attention(q, k2, v2, [0, 3, 7], [0, 3, 7], 1.0, True)
    assert np.array_equal(o[:6], o2[:6]) and not np.allclose(o[6], o2[6])


# ------------------------------------------------------------------ library
def _p(v):
    return ctypes.c_void_p(v)


A = _p(0x10000)


def _append(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, tokens=4, hq=4, hkv=1, d=128, rope=A, rows=8, dim=128, pos=A,
             slots=A, qn=None, kn=None, eps=1e-6, qo=A, qos=512, ko=None, kos=0, kc=A, vc=A, sk=None, sv=None, pages=3,
             page=16)
    assert not set(kw) - set(a)
    return lib.convrot_rope_append(*(a | kw).values(), None)


def test_append_validation(lib):
    for bad in (dict(tokens=-1), dict(hq=0), dict(hkv=3), dict(hq=1025, hkv=1), dict(page=0), dict(page=24),
                dict(page=8192), dict(pages=-1), dict(rows=0), dict(dim=8), dict(dim=24), dict(dim=144), dict(qs=504),
                dict(qs=516), dict(ks=64), dict(vs=120), dict(qos=8), dict(ko=A, kos=64), dict(qn=A, eps=-1.0),
                dict(kn=A, eps=float("nan")), dict(tokens=(1 << 24) + 1)):
        assert _append(lib, **bad) == 2, bad
    assert _append(lib, d=96) == 4
    assert _append(lib, d=256, qs=1024, ks=256, vs=256, qos=1024) == 4
    for name in ("q", "k", "v", "rope", "pos", "slots", "qo", "kc", "vc"):
        assert _append(lib, **{name: None}) == 1, name
        assert _append(lib, **{name: _p(0x10002)}) == 3, name
    assert _append(lib, sk=A) == 1 and _append(lib, sv=A) == 1   # one scale without the other
    assert _append(lib, sk=_p(0x10004), sv=A) == 3
    assert _append(lib, qn=_p(0x10004)) == 3
    assert _append(lib, tokens=0, q=None, kc=None) == 0


def _prompt(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, tokens=4, kv=4, hq=4, hkv=1, d=128, cuq=A, cuk=A, seqs=2, scale=0.1,
             causal=1, out=_p(0x20000), os=512)
    assert not set(kw) - set(a)
    return lib.convrot_attention_prompt(*(a | kw).values(), None)


def test_prompt_validation(lib):
    for bad in (dict(tokens=-1), dict(kv=-1), dict(seqs=-1), dict(hkv=3), dict(hq=0), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=508), dict(ks=64), dict(vs=0), dict(os=256)):
        assert _prompt(lib, **bad) == 2, bad
    assert _prompt(lib, d=80) == 4
    for name in ("q", "k", "v", "cuq", "cuk", "out"):
        assert _prompt(lib, **{name: None}) == 1, name
        assert _prompt(lib, **{name: _p(0x10002)}) == 3, name
    for name in "qkv":                                            # in place is refused
        assert _prompt(lib, **{name: _p(0x20000)}) == 4
    assert _prompt(lib, tokens=0, q=None) == 0 and _prompt(lib, seqs=0, q=None) == 0


def _decode(lib, **kw):
    a = dict(q=A, qs=512, seqs=4, hq=4, hkv=1, d=128, kc=A, vc=A, sk=None, sv=None, pages=3, page=16, table=A, ts=5,
             cols=5, lens=A, scale=0.1, out=A, os=512, ws=None, wb=0)
    assert not set(kw) - set(a)
    return lib.convrot_attention_decode(*(a | kw).values(), None)


def test_decode_validation(lib):
    for bad in (dict(seqs=-1), dict(hkv=3), dict(pages=-1), dict(page=0), dict(page=40), dict(ts=4), dict(cols=-1),
                dict(scale=0.0), dict(qs=256), dict(os=516)):
        assert _decode(lib, **bad) == 2, bad
    assert _decode(lib, d=32) == 4
    for name in ("q", "kc", "vc", "table", "lens", "out"):
        assert _decode(lib, **{name: None}) == 1, name
        assert _decode(lib, **{name: _p(0x10002)}) == 3, name
    assert _decode(lib, sk=A) == 1
    assert _decode(lib, ws=_p(0x10010), wb=1 << 30) == 3
    assert _decode(lib, pages=1 << 21, page=4096, hkv=1, hq=1, qs=128, os=128) == 4  # rows of a TMA map: 31 bits
    assert _decode(lib, seqs=0, q=None) == 0


# ------------------------------------------------------------------ binding
def _raises(match, fn, *args, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*args, **kw)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(*shape)


def test_append_operands():
    T, Hq, Hkv, D = 3, 4, 2, 64
    slots = torch.zeros(T, dtype=torch.int64)
    cache = bf(5, Hkv, 16, D)
    ok = [bf(T, Hq, D), bf(T, Hkv, D), bf(T, Hkv, D), f32(9, 64), i32(T), slots, cache, cache.clone()]

    def call(match, at=None, new=None, **kw):
        args = list(ok)
        if at is not None:
            args[at] = new
        _raises(match, cr.convrot_rope_append, *args, **kw)

    call("must be a CUDA tensor")
    call("q must be torch.bfloat16", 0, f32(T, Hq, D))
    call("q must have 3 dimensions", 0, bf(T, Hq * D))
    call("k must have 3 rows", 1, bf(T + 1, Hkv, D))
    call("k must have 64 elements", 1, bf(T, Hkv, 128))
    call("v must have 2 heads", 2, bf(T, Hkv + 1, D))
    call("contiguous heads", 0, bf(T, D, Hq).transpose(1, 2))
    call("contiguous heads", 0, bf(1, Hq, D).expand(T, Hq, D))
    call("rope must be torch.float32", 3, bf(9, 64))
    call("positions must be torch.int32", 4, slots)
    call("slots must have shape", 5, slots[:2])
    call("k_cache must be torch.int8", k_scale=f32(5, Hkv, 16), v_scale=f32(5, Hkv, 16))
    call("v_cache must have shape", 7, bf(4, Hkv, 16, D))
    call("q_norm must have shape", q_norm=f32(Hq, D))
    call("q_out must have 4 heads", q_out=bf(T, Hkv, D))
    call("k_out must have 3 rows", k_out=bf(T + 1, Hkv, D))


def test_append_cache_heads():
    T, D = 3, 64
    slots, cache = torch.zeros(T, dtype=torch.int64), bf(5, 2, 16, D)
    for heads in (1, 4):
        _raises("k_cache must hold", cr.convrot_rope_append, bf(T, 4, D), bf(T, heads, D), bf(T, heads, D), f32(9, 64), i32(T),
                slots, cache, cache)
    _raises("k_cache must hold", cr.convrot_rope_append, bf(T, 4, 128), bf(T, 2, 128), bf(T, 2, 128), f32(9, 64), i32(T), slots,
            cache, cache)


def test_rope_table_matches_the_oracle():
    t = cr.rope_table(1000, 64, 1e4)
    assert t.dtype == torch.float32 and np.abs(t.numpy() - ref.rope_table(1000, 64, 1e4)).max() <= 2.0 ** -23


def test_attention_block_shapes():
    W = [torch.zeros(n, 512, dtype=torch.bfloat16) for n in (512, 128, 128)]
    with pytest.raises(ValueError, match="multiple of kv_heads"):
        cr.ConvRotAttention(*W, W[0], q_heads=8, kv_heads=3, rope=f32(4, 64))
    with pytest.raises(ValueError, match="Wk and Wv must have"):
        cr.ConvRotAttention(*W, W[0], q_heads=8, kv_heads=4, rope=f32(4, 64))
    with pytest.raises(ValueError, match="Wo must have"):
        cr.ConvRotAttention(*W, torch.zeros(512, 256, dtype=torch.bfloat16), q_heads=8, kv_heads=2, rope=f32(4, 64))


def test_prompt_operands():
    q, k, cu = bf(6, 4, 64), bf(6, 2, 64), i32(3)
    f = cr.convrot_attention_prompt
    _raises("must be a CUDA tensor", f, q, k, k, cu)
    _raises("v must have 6 rows", f, q, k, bf(5, 2, 64), cu)
    _raises("k must have 64 elements", f, q, bf(6, 2, 128), k, cu)
    _raises("cu_seqlens must be torch.int32", f, q, k, k, cu.long())
    _raises("cu_seqlens_k is needed", f, q, bf(7, 2, 64), bf(7, 2, 64), cu)
    _raises("cu_seqlens_k must have shape", f, q, k, k, cu, i32(4))
    _raises("one offset more", f, q, k, k, i32(0))
    _raises("out must have 4 heads", f, q, k, k, cu, out=bf(6, 2, 64))


def test_decode_operands():
    q, cache, table, lens = bf(3, 4, 64), bf(5, 2, 16, 64), i32(3, 4), i32(3)
    f = cr.convrot_attention_decode
    _raises("must be a CUDA tensor", f, q, cache, cache, table, lens)
    _raises("q has 64 elements per head, the cache 128", f, q, bf(5, 2, 16, 128), bf(5, 2, 16, 128), table, lens)
    _raises("block_table must be", f, q, cache, cache, table.long(), lens)
    _raises("block_table must have shape", f, q, cache, cache, table[:2], lens)
    _raises("contiguous rows", f, q, cache, cache, i32(4, 3).t(), lens)
    _raises("seq_lens must have shape", f, q, cache, cache, table, i32(4))
    _raises("k_scale must have shape", f, q, cache.to(torch.int8), cache.to(torch.int8), table, lens, k_scale=f32(5, 2),
            v_scale=f32(5, 2))
    _raises("v_scale must be a torch.Tensor", f, q, cache.to(torch.int8), cache.to(torch.int8), table, lens,
            k_scale=f32(5, 2, 16))


# ------------------------------------------------------------------ slots
def test_slots_of_tokens_the_table_has_no_place_for():
    """Indices outside the block table are not followed (on a GPU they would end
    the process): padding is not stored, a token without a place is past every
    cache, where the append leaves it out and reports it."""
    cache = cr.PagedKVCache.__new__(cr.PagedKVCache)
    cache.page_size = 16
    table = torch.tensor([[3, 1], [0, -1]], dtype=torch.int32)

    def slots(sequence, position, table=table):
        return cache.slots(table, torch.tensor(sequence), torch.tensor(position, dtype=torch.int32)).tolist()

    assert slots([0, 0, 0, 1, 1], [0, 15, 16, 5, 15]) == [48, 63, 16, 5, 15]
    assert all(s < 0 for s in slots([1, 1, 0, 1, -1, -1], [16, 31, -1, -16, 0, 99]))
    most = 2 ** 31 * 4096          # no cache has a slot so far
    assert all(s >= most for s in slots([0, 1, 2, 7, 0], [32, 1 << 30, 0, 5, 2 ** 31 - 1]))
    empty = torch.empty(2, 0, dtype=torch.int32)
    assert [s >= most for s in slots([0, 1, 2], [0, 5, 0], empty)] == [True] * 3
    assert slots([0, -1], [-1, 3], empty) == [-1, -1] and slots([], []) == []


# ------------------------------------------------------------------ results on inputs
def test_decode_results_on_queries(lib):
    """In place or apart; anything between is refused.  Every arrangement of two
    to five rows against their bytes one by one.  (The calls have no workspace,
    so that none of them launches.)"""
    rng = np.random.default_rng(0)
    width, kinds = 2 * 128, set()
    for _ in range(3000):
        n = int(rng.integers(1, 6))
        sq, so = (int(x) for x in rng.choice([128, 136, 264, 384, 520], 2))
        if rng.random() < 0.5:
            so = sq
        q = 1 << 20
        out = q + 16 * int(rng.integers(-150, 150)) if rng.random() < 0.9 else q
        taken = [set().union(*(range(p + 2 * s * i, p + 2 * s * i + width, 16) for i in range(n))) for p, s in ((q, sq), (out, so))]
        shares = bool(taken[0] & taken[1]) and not (q == out and (sq == so or n == 1))
        st = _decode(lib, q=_p(q), qs=sq, out=_p(out), os=so, seqs=n, hq=1, hkv=1)
        assert (st == 4) == shares and st in (4, 5, 7), (n, sq, so, out - q)
        kinds.add((shares, sq == so, q < out))
    assert len(kinds) == 8


def test_append_results_on_inputs(lib):
    """q_out may be q and k_out may be k; nothing else may share memory."""
    at = dict(q=0x100000, k=0x200000, v=0x300000, qo=0x400000, ko=0x500000, kc=0x600000, vc=0x700000)
    ok = {n: _p(p) for n, p in at.items()} | dict(kos=128)

    def status(**kw):
        return _append(lib, **(ok | kw))

    for out, stride, inputs in (("qo", "qos", ("k", "v", "ko")), ("ko", "kos", ("q", "v", "qo"))):
        for name in inputs:
            assert status(**{out: _p(at[name])}) == 4 and status(**{out: _p(at[name] + 16)}) == 4
    assert status(qo=_p(at["q"] + 16)) == 4 and status(qo=_p(at["q"]), qos=520) == 4
    assert status(ko=_p(at["k"] + 16)) == 4 and status(ko=_p(at["k"]), kos=136) == 4
    assert status(vc=_p(at["kc"])) == 4 and status(vc=_p(at["kc"] + 3 * 16 * 128 * 2 - 16)) == 4
    scales = dict(sk=_p(0x800000), sv=_p(0x800000))
    assert status(**scales) == 4 and status(sk=_p(0x800000), sv=_p(0x800000 + 3 * 16 * 4 - 16)) == 4


def test_prompt_results_on_inputs(lib):
    for name, wide in (("q", 512), ("k", 128), ("v", 128)):
        for off in (16, -16, 4 * 2 * wide - 16, 16 - 4 * 2 * 512):       # four rows of each, four of the result
            assert _prompt(lib, **{name: _p(0x20000 - off)}) == 4, (name, off)


# ------------------------------------------------------------------ scales
def test_scales_that_leave_fp32(lib):
    """scores are held times log2(e): a scale that overflows by that would make
    every result NaN."""
    most = 3.4028234663852886e38
    for scale in (most, most / 1.4426):
        assert _prompt(lib, scale=scale) == 2 and _decode(lib, scale=scale) == 2
    assert _decode(lib, scale=most / 1.443, out=_p(0x20000)) in (5, 7)      # (without a workspace: no launch)
