"""The attention operators on the GPU against the float64 oracle: append with
rotation, prompt attention and single-token attention over a paged cache.

Tolerances are the oracle's bounds of the kernels' arithmetic
(oracle/attention_ref.py): half a bf16 step per rounding plus the fp32 terms.
Queries are drawn four times as wide as keys, so that a few keys carry most of
a row's weight and a wrong key shows.
"""
import numpy as np
import pytest
import torch

from oracle import attention_ref as ref
from tests import _tol

pytestmark = pytest.mark.gpu

U, BF16 = ref.U, ref.BF16
TINY = 2.0 ** -134      # half a step of bfloat16's subnormals
TINY32 = 2.0 ** -149    # a step of fp32's


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import w8a8_int8_quantized_rmsnorm_b200 as m
    m.lib()
    return m


def f64(t):
    return t.detach().float().cpu().double().numpy()


def randn(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def within(got, want, tol, what=""):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}, worst "
                           f"{np.max(np.abs(got - want) / np.maximum(tol, 1e-300))} times the bound")


# ------------------------------------------------------------------ append
def append_case(seed, T, Hq, Hkv, D, rot, page, i8, norm, pad=0, spare=2, rows=50):
    fused = randn(seed, T, (Hq + 2 * Hkv) * D)
    q, k, v = fused.split([Hq * D, Hkv * D, Hkv * D], 1)
    pages = (T + page - 1) // page + spare
    g = torch.Generator().manual_seed(seed + 1)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T:
        slots[0] = pages * page - 1
        slots = torch.where(torch.arange(T) >= T - pad, -1, slots)
        slots[(slots == pages * page - 1) & (torch.arange(T) > 0)] = -1
    shape = (pages, Hkv, page, D)
    c = dict(q=q.view(T, Hq, D), k=k.view(T, Hkv, D), v=v.view(T, Hkv, D),
             rope=torch.from_numpy(ref.rope_table(rows, rot)).cuda(),
             positions=torch.randint(0, rows, (T,), generator=g, dtype=torch.int32).cuda(), slots=slots.cuda())
    if i8:
        c |= dict(k_cache=torch.randint(-127, 128, shape, generator=g, dtype=torch.int16).to(torch.int8).cuda(),
                  v_cache=torch.randint(-127, 128, shape, generator=g, dtype=torch.int16).to(torch.int8).cuda(),
                  k_scale=torch.rand(shape[:3], generator=g).cuda(), v_scale=torch.rand(shape[:3], generator=g).cuda())
    else:
        c |= dict(k_cache=randn(seed + 2, *shape), v_cache=randn(seed + 3, *shape))
    if norm:
        c |= dict(q_norm=torch.randn(D, generator=g).cuda() * 0.1, k_norm=torch.randn(D, generator=g).cuda() * 0.1)
    return c


def check_append(c, before, q_out, k_out, eps=1e-6):
    rope, pos, slots = c["rope"].cpu().numpy(), c["positions"].cpu().numpy(), c["slots"].cpu().numpy()
    w = {x: None if c.get(x) is None else f64(c[x]) for x in ("q_norm", "k_norm")}
    q, qe = ref.norm_rotate(f64(before["q"]), w["q_norm"], rope, pos, eps)
    k, ke = ref.norm_rotate(f64(before["k"]), w["k_norm"], rope, pos, eps)
    v = f64(before["v"])
    within(f64(q_out), q, BF16 * np.abs(q) + 2 * qe + TINY, "q")
    if k_out is not None:
        within(f64(k_out), k, BF16 * np.abs(k) + 2 * ke + TINY, "k")
    page = c["k_cache"].shape[2]
    live = slots >= 0
    at = slots[live]
    for name, y, err in (("k", k, ke), ("v", v, 0 * v)):
        new, old = c[name + "_cache"].cpu(), before[name + "_cache"].cpu()
        rows = f64(new)[at // page, :, at % page]
        if c.get("k_scale") is None:
            within(rows, y[live], BF16 * np.abs(y[live]) + 2 * err[live] + TINY, name + " cache")
            if name == "v":
                assert np.array_equal(rows, y[live])
        else:
            scale = c[name + "_scale"].cpu().double().numpy()[at // page, :, at % page]
            y2, e2 = y[live].reshape(-1, y.shape[-1]), err[live].reshape(-1, y.shape[-1])
            amax = np.abs(y2).max(1)
            ratio = e2.max(1) / np.where(amax > 0, amax, 1)
            s = amax / 127
            assert np.all(np.abs(scale.reshape(-1) - s) <= s * _tol.scale_rel_tol(ratio, False) + TINY32), name + " scales"
            z = y2 / np.where(s > 0, s, 1)[:, None]
            _tol.check_codes(rows.reshape(z.shape), np.rint(z), z, _tol.int8_code_window(ratio), name)
        # every other row of the cache is as it was
        keep = np.ones(new.shape[0] * page, bool)
        keep[at] = False
        flat = [x.view(torch.uint8 if x.dtype == torch.int8 else torch.int16).transpose(1, 2).flatten(0, 1).numpy()
                for x in (new, old)]
        assert np.array_equal(flat[0][keep], flat[1][keep]), name + " cache: a row that is no slot changed"
        if c.get("k_scale") is not None:
            sc = [x.cpu().transpose(1, 2).flatten(0, 1).numpy() for x in (c[name + "_scale"], before[name + "_scale"])]
            assert np.array_equal(sc[0][keep], sc[1][keep])


def run_append(cr, c, k_out=True, **kw):
    before = {n: t.clone() for n, t in c.items()}
    ko = torch.empty(c["k"].shape, dtype=torch.bfloat16, device="cuda") if k_out is True else k_out
    q, k = cr.convrot_rope_append(**c, k_out=ko, **kw)
    torch.cuda.synchronize()
    assert cr.convrot_device_status() == 0
    return before, q, k


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page", [
    (1, 32, 8, 128, 128, 16), (1, 1, 1, 64, 64, 16), (3, 5, 1, 64, 32, 48), (37, 8, 2, 128, 64, 16),
    (130, 14, 2, 64, 16, 64), (300, 4, 4, 128, 128, 128), (33, 7, 7, 128, 16, 32), (1000, 32, 8, 128, 128, 64),
    (9000, 2, 1, 64, 64, 4096)])
def test_append(cr, T, Hq, Hkv, D, rot, page, norm, i8):
    c = append_case(T + Hq, T, Hq, Hkv, D, rot, page, i8, norm, pad=T // 5)
    before, q, k = run_append(cr, c)
    check_append(c, before, q, k)


def test_append_in_place_and_without_rotated_keys(cr):
    c = append_case(5, 70, 8, 2, 128, 128, 16, False, True)
    before = {n: t.clone() for n, t in c.items()}
    q, k = cr.convrot_rope_append(**c, q_out=c["q"], k_out=c["k"])
    assert q.data_ptr() == c["q"].data_ptr() and k.data_ptr() == c["k"].data_ptr()
    check_append(c, before, q, k)
    assert torch.equal(c["v"], before["v"])
    c = append_case(6, 70, 8, 2, 128, 128, 16, True, False)
    before, q, k = run_append(cr, c, k_out=None)
    assert k is None
    check_append(c, before, q, None)


def test_append_one_norm_only(cr):
    c = append_case(7, 21, 4, 2, 64, 64, 16, False, True)
    c["q_norm"] = None
    before = {n: None if t is None else t.clone() for n, t in c.items()}
    ko = torch.empty_like(c["k"].contiguous())
    q, k = cr.convrot_rope_append(**c, k_out=ko)
    check_append(c, before, q, k)


def test_append_extreme_rows_int8(cr):
    """A zero row (scale 0), rows far below and far above one, and a row with a
    NaN, whose scale says so."""
    c = append_case(8, 6, 2, 1, 64, 64, 16, True, False)
    k = c["k"].clone()
    k[0] = 0
    k[1] = k[1].float() * 2.0 ** -120
    k[2] = k[2].float() * 2.0 ** 100
    k[3] = k[3].float() * 1e-38
    c["k"] = k
    before, q, ko = run_append(cr, c)
    check_append(c, before, q, ko)
    c["k"][4, 0, 3] = float("nan")
    run_append(cr, c)
    page = c["k_cache"].shape[2]
    at = int(c["slots"][4])
    assert torch.isnan(c["k_scale"][at // page, 0, at % page])


def test_append_unrotated_part_keeps_infinities(cr):
    c = append_case(9, 3, 2, 1, 128, 64, 16, False, False)
    c["k"] = c["k"].clone()
    c["k"][1, 0, 100] = float("inf")
    before, q, ko = run_append(cr, c)
    assert torch.isinf(ko[1, 0, 100]) and torch.isfinite(ko).sum() == ko.numel() - 1


def test_append_reports_indices_outside(cr):
    """A position or slot outside its tensor: the token is left out, the others
    are as ever, and the device status says so."""
    for name, bad in (("positions", 50), ("positions", -1), ("slots", 10 ** 9)):
        c = append_case(10, 40, 4, 2, 64, 64, 16, False, False)
        c[name][7] = bad
        before = {n: t.clone() for n, t in c.items()}
        qo, ko = torch.zeros_like(c["q"].contiguous()), torch.zeros_like(c["k"].contiguous())
        cr.convrot_rope_append(**c, q_out=qo, k_out=ko)
        assert cr.convrot_device_status() == 2
        assert cr.convrot_device_status() == 0
        assert not qo[7].any() and not ko[7].any()
        keep = torch.arange(40) != 7
        c2 = {n: t[keep] if n in ("q", "k", "v", "positions", "slots") else t for n, t in c.items()}
        b2 = {n: t[keep] if n in ("q", "k", "v", "positions", "slots") else t for n, t in before.items()}
        check_append(c2, b2, qo[keep], ko[keep])


# ------------------------------------------------------------------ prompt
def prompt_case(seed, lens_q, lens_k, Hq, Hkv, D, spare=0):
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (lens_q, lens_k))
    T, Tk = int(cu_q[-1]) + spare, int(cu_k[-1]) + spare
    return (randn(seed, T, Hq, D, std=4.0), randn(seed + 1, Tk, Hkv, D), randn(seed + 2, Tk, Hkv, D), cu_q, cu_k)


def check_prompt(cr, q, k, v, cu_q, cu_k, causal=True, scale=None, out=None):
    got = cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda(),
                                      causal=causal, scale=scale, out=out)
    torch.cuda.synchronize()
    assert cr.convrot_device_status() == 0
    o, tol = ref.packed_attention(f64(q), f64(k), f64(v), cu_q, cu_k, q.shape[2] ** -0.5 if scale is None else scale,
                                  causal)
    n = cu_q[-1]
    within(f64(got)[:n], o[:n], tol[:n], "prompt")
    return got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([1], 1, 1, 64), ([1], 32, 8, 128), ([2], 4, 1, 128), ([31], 8, 2, 64), ([64], 4, 1, 128), ([65], 4, 1, 128),
    ([127], 2, 2, 128), ([128], 1, 1, 128), ([129], 3, 1, 128), ([255, 256, 257], 1, 1, 64), ([300], 5, 1, 128),
    ([1, 1, 1, 1], 8, 8, 64), ([5, 0, 300, 64, 0], 8, 2, 128), ([0, 0], 2, 1, 64), ([511], 16, 2, 64),
    ([40] * 9, 14, 2, 128), ([770], 6, 2, 128), ([90], 128, 1, 64), ([70], 200, 1, 128), ([1200, 3], 2, 1, 128)])
def test_prompt(cr, lens, Hq, Hkv, D, causal):
    check_prompt(cr, *prompt_case(sum(lens) + Hq, lens, lens, Hq, Hkv, D), causal=causal)


@pytest.mark.parametrize("n,Hq,Hkv,D", [(150, 4, 2, 64), (64, 2, 1, 128), (33, 8, 8, 128)])
def test_prompt_many_sequences(cr, n, Hq, Hkv, D):
    """More sequences than a warp has lanes, empty ones among them."""
    lens = [(i * 29) % 41 if i % 3 else 0 for i in range(n)]
    lens[-1] = 0
    check_prompt(cr, *prompt_case(n, lens, lens, Hq, Hkv, D))


def test_prompt_overlapping_offsets_end(cr):
    """Offsets that go back and forth are no pack: reported, nothing hangs, and
    nothing outside the rows is written."""
    q, k, v, _, _ = prompt_case(12, [640], [640], 1, 1, 64)
    big = torch.full((660, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for n in (3, 2001):
        cu = torch.tensor([0, 640] * n, dtype=torch.int32, device="cuda")
        cr.convrot_attention_prompt(q, k, v, cu, out=big[:640])
        assert cr.convrot_device_status() == 2 and cr.convrot_device_status() == 0
        assert (big[640:] == 7).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_with_keys_of_another_length(cr, D, causal):
    """More keys than queries (a prompt's continuation), fewer (leading rows see
    nothing and are zero), and none at all."""
    lens_q, lens_k = [3, 130, 200, 17, 64, 1], [300, 257, 40, 0, 64, 129]
    got = check_prompt(cr, *prompt_case(1, lens_q, lens_k, 4, 2, D), causal=causal)
    assert not got[350:].view(torch.int16)[-82:-65].any()           # the sequence without keys
    if causal:
        assert not got[133:133 + 160].any()


def test_prompt_strided_operands_and_untouched_rows(cr):
    """q, k, v as column views of one fused buffer, out with rows further apart;
    rows behind the last sequence stay as they were."""
    T, Hq, Hkv, D = 400, 8, 2, 128
    fused = randn(3, T, (Hq + 2 * Hkv) * D)
    q, k, v = (x.view(T, -1, D) for x in fused.split([Hq * D, Hkv * D, Hkv * D], 1))
    big = torch.full((T, Hq * D + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, :Hq * D].view(T, Hq, D)
    cu = np.array([0, 150, 333], np.int32)
    check_prompt(cr, q, k, v, cu, cu, out=out)
    assert (big[333:] == 7).all() and (big[:, Hq * D:] == 7).all()
    first = np.array([20, 150, 333], np.int32)                      # rows before the first sequence, too
    big.fill_(7.0)
    got = cr.convrot_attention_prompt(q, k, v, torch.from_numpy(first).cuda(), out=out)
    assert (big[:20] == 7).all() and not (got[20:333] == 7).all(-1).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.38e38])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 2, 2)])
def test_prompt_masked_places_do_not_leak(cr, bad, D, Hq, Hkv):
    """Keys and values that a row does not see, of later positions, of other
    sequences and of rows behind the last one, may be anything."""
    lens = [200, 1, 150]
    q, k, v, cu, _ = prompt_case(4, lens, lens, Hq, Hkv, D, spare=30)
    k[180:201], v[180:201] = bad, bad      # seen by rows 180.. of the first sequence and by the second
    k[351:], v[351:] = bad, bad
    got = f64(cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda()))
    o, tol = ref.packed_attention(f64(q)[:351], f64(k)[:351], f64(v)[:351], cu, cu, D ** -0.5, True)
    ok = np.r_[0:180, 201:351]
    within(got[ok], o[ok], tol[ok], "rows that do not see them")
    if bad != bad:
        assert np.isnan(got[180:201]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_nan_in_one_element_of_a_seen_value(cr, D):
    """It reaches that element of the rows that see it, and nothing else."""
    q, k, v, cu, _ = prompt_case(5, [230], [230], 4, 2, D)
    clean = v.clone()
    v[100, 1, 5] = float("nan")
    got = f64(cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda()))
    o, tol = ref.packed_attention(f64(q), f64(k), f64(clean), cu, cu, D ** -0.5, True)
    hit = np.zeros(got.shape, bool)
    hit[100:, 2:, 5] = True
    assert np.isnan(got[hit]).all()
    within(got[~hit], o[~hit], tol[~hit], "the others")


def test_prompt_scores_of_minus_infinity_and_large_scores(cr):
    q, k, v, cu, _ = prompt_case(6, [160], [160], 2, 1, 128)
    q[:, :, 0], k[:, :, 0] = 300.0, 0.0
    k[5:40, :, 0] = -3e38                     # their scores are -inf: they take no part
    k[100] = k[100].float() * 100             # scores of a thousand and more
    got = f64(cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda()))
    see = np.tril(np.ones((160, 160), bool))
    see[:, 5:40] = False
    o, tol = np.zeros(got.shape), np.zeros(got.shape)
    for h in range(2):
        o[:, h], tol[:, h] = ref.attention(f64(q)[:, h], f64(k)[:, 0], f64(v)[:, 0], 128 ** -0.5, see)
    within(got, o, tol, "prompt")


def test_prompt_scale_and_repeatability(cr):
    q, k, v, cu, _ = prompt_case(8, [190, 77], [190, 77], 4, 2, 64)
    a = check_prompt(cr, q, k, v, cu, cu, scale=0.01)
    b = check_prompt(cr, q, k, v, cu, cu, scale=0.01)
    assert torch.equal(a, b)
    check_prompt(cr, q, k, v, cu, cu, scale=3.0)


def test_prompt_reports_offsets_outside(cr):
    q, k, v, cu, _ = prompt_case(9, [50, 60], [50, 60], 2, 1, 64)
    good = check_prompt(cr, q, k, v, cu, cu)
    out = torch.zeros_like(good)
    cu_k = torch.tensor([0, 50, 111], dtype=torch.int32, device="cuda")   # one past the keys
    cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda(), cu_k, out=out)
    assert cr.convrot_device_status() == 2 and cr.convrot_device_status() == 0
    assert torch.equal(out[:50], good[:50]) and not out[50:].any()
    cu_q = torch.tensor([0, 50, 200], dtype=torch.int32, device="cuda")
    out.zero_()
    cr.convrot_attention_prompt(q, k, v, cu_q, torch.from_numpy(cu).cuda(), out=out)
    assert cr.convrot_device_status() == 2
    assert torch.equal(out[:50], good[:50]) and not out[50:].any()


def test_prompt_larger_packs_agree_with_single_prompts(cr):
    """A row's result does not depend on what it is packed with."""
    lens = [1, 700, 33, 1025, 256, 90]
    q, k, v, cu, _ = prompt_case(10, lens, lens, 8, 2, 128)
    whole = cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda())
    for a, b in zip(cu, cu[1:]):
        one = cr.convrot_attention_prompt(q[a:b], k[a:b], v[a:b], torch.tensor([0, b - a], dtype=torch.int32).cuda())
        assert torch.equal(whole[a:b], one)


# ------------------------------------------------------------------ decode
def decode_case(seed, lens, Hq, Hkv, D, page, i8, fill=float("nan"), spare=2):
    """A cache whose rows past every sequence's end hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages, cols = sum(need) + spare, max(need + [1]) + 1
    perm = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), cols), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    shape = (pages, Hkv, page, D)
    live = torch.zeros(pages, page, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(need[i]):
            live[table[i, j], :max(0, min(page, n - j * page))] = True
    keep = live[:, None, :].expand(shape[:3])
    c = dict(q=randn(seed + 1, len(lens), Hq, D, std=4.0))
    if i8:
        for x in "kv":
            codes = torch.randint(-127, 128, shape, generator=g, dtype=torch.int16).to(torch.int8)
            scale = torch.rand(shape[:3], generator=g) * 0.02 + 0.005
            scale[~keep] = fill
            c |= {x + "_cache": codes.cuda(), x + "_scale": scale.cuda()}
    else:
        for i, x in enumerate("kv"):
            t = torch.randn(shape, generator=g).to(torch.bfloat16)
            t[~keep] = fill
            c[x + "_cache"] = t.cuda()
    return c | dict(block_table=table.cuda(), seq_lens=torch.tensor(lens, dtype=torch.int32).cuda())


def oracle_decode(c, lens, scale=None):
    s = [None if c.get(x) is None else c[x].cpu().double().numpy() for x in ("k_scale", "v_scale")]
    return ref.paged_attention(f64(c["q"]), f64(c["k_cache"]), f64(c["v_cache"]), *s, c["block_table"].cpu().numpy(),
                               lens, c["q"].shape[2] ** -0.5 if scale is None else scale)


def check_decode(cr, c, lens, **kw):
    got = cr.convrot_attention_decode(**c, **kw)
    torch.cuda.synchronize()
    assert cr.convrot_device_status() == 0
    o, tol = oracle_decode(c, lens, kw.get("scale"))
    within(f64(got), o, tol, "decode")
    return got


LENS = [[1], [0], [15, 16, 17, 0, 1], [63, 64, 65, 127, 128, 129], [1000], [5, 3000, 0, 70, 1, 250]]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 16), (4, 4, 64, 64), (5, 1, 128, 48), (16, 2, 64, 32),
                                           (9, 1, 64, 128), (20, 1, 128, 16), (14, 2, 128, 1024), (6, 3, 64, 16)])
@pytest.mark.parametrize("lens", LENS, ids=[str(x)[:20] for x in LENS])
def test_decode(cr, lens, Hq, Hkv, D, page, i8):
    """Rows past a sequence's end, unused pages and unused table entries hold
    NaN or nonsense and must not matter."""
    check_decode(cr, decode_case(sum(lens) + Hq, lens, Hq, Hkv, D, page, i8), lens)


@pytest.mark.parametrize("i8", [False, True])
def test_decode_long_and_many(cr, i8):
    check_decode(cr, decode_case(1, [20011], 4, 1, 128, 64, i8), [20011])
    lens = [(i * 37) % 190 for i in range(333)]
    check_decode(cr, decode_case(2, lens, 4, 2, 64, 16, i8, fill=float("inf")), lens)


def test_decode_strided_operands(cr):
    lens = [70, 5, 130]
    c = decode_case(3, lens, 8, 2, 128, 16, False)
    fused = torch.zeros(3, 12 * 128, dtype=torch.bfloat16, device="cuda")
    fused[:, :1024] = c["q"].flatten(1)
    c["q"] = fused[:, :1024].view(3, 8, 128)
    wide = torch.full((3, 40), -9, dtype=torch.int32, device="cuda")
    wide[:, :c["block_table"].shape[1]] = c["block_table"]
    c["block_table"] = wide[:, :c["block_table"].shape[1]]
    big = torch.full((3, 8 * 128 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    check_decode(cr, c, lens, out=big[:, :1024].view(3, 8, 128), scale=0.05)
    assert (big[:, 1024:] == 7).all()


def test_decode_infinite_scores(cr):
    lens = [90]
    c = decode_case(4, lens, 2, 1, 64, 16, False, fill=0.0)
    c["q"][..., 0] = 300.0
    c["k_cache"][..., 0] = 0.0
    first = int(c["block_table"][0, 0])
    c["k_cache"][first, 0, 3:9, 0] = -3e38                  # scores of -inf
    got = f64(cr.convrot_attention_decode(**c))
    c2 = dict(c, k_cache=c["k_cache"].clone())
    rows = np.ones((1, 90), bool)
    rows[0, 3:9] = False
    k = ref.cache_rows(f64(c2["k_cache"]), None, c["block_table"].cpu().numpy()[0], 90)[:, 0]
    v = ref.cache_rows(f64(c["v_cache"]), None, c["block_table"].cpu().numpy()[0], 90)[:, 0]
    k[3:9, 0] = 0
    for h in range(2):
        o, tol = ref.attention(f64(c["q"])[0, h][None], k, v, 64 ** -0.5, rows)
        within(got[0, h], o[0], tol[0], "decode")


def test_decode_reports_pages_and_lengths_outside(cr):
    lens = [70, 40, 33]
    c = decode_case(5, lens, 4, 2, 64, 16, False)
    good = check_decode(cr, c, lens)
    for bad in (-1, 10 ** 6):
        d = dict(c, block_table=c["block_table"].clone())
        d["block_table"][1, 1] = bad
        got = cr.convrot_attention_decode(**d)
        assert cr.convrot_device_status() == 2 and cr.convrot_device_status() == 0
        assert torch.equal(got[[0, 2]], good[[0, 2]]) and torch.isfinite(got).all()
    for bad in (-3, 10 ** 6):
        d = dict(c, seq_lens=c["seq_lens"].clone())
        d["seq_lens"][0] = bad
        got = cr.convrot_attention_decode(**d)
        assert cr.convrot_device_status() == 2 and cr.convrot_device_status() == 0
        assert torch.equal(got[1:], good[1:]) and not got[0].any()


def test_decode_is_repeatable_and_batch_independent_in_value(cr):
    lens = [3000, 1, 700, 64]
    c = decode_case(6, lens, 8, 2, 128, 32, False)
    a = check_decode(cr, c, lens)
    for _ in range(3):
        assert torch.equal(a, cr.convrot_attention_decode(**c))


@pytest.mark.parametrize("i8", [False, True])
def test_cache_offsets_past_32_bits(cr, i8):
    """Pages whose rows start past 2^31 elements (and past 2^32 bytes)."""
    Hkv, page, D, lens = 8, 64, 128, [100, 64]
    pages = (1 << 31) // (Hkv * page * D) + 6
    shape = (pages, Hkv, page, D)
    dt = torch.int8 if i8 else torch.bfloat16
    c = dict(k_cache=torch.zeros(shape, dtype=dt, device="cuda"), v_cache=torch.zeros(shape, dtype=dt, device="cuda"))
    if i8:
        c |= dict(k_scale=torch.zeros(shape[:3], device="cuda"), v_scale=torch.zeros(shape[:3], device="cuda"))
    table = torch.tensor([[pages - 1, pages - 3], [pages - 4, 0]], dtype=torch.int32)
    T, Hq = sum(lens), 16
    q, k, v = randn(1, T, Hq, D, std=4.0), randn(2, T, Hkv, D), randn(3, T, Hkv, D)
    run = np.concatenate([np.arange(n) for n in lens])
    seq = np.repeat([0, 1], lens)
    slots = torch.from_numpy(table.numpy()[seq, run // page].astype(np.int64) * page + run % page)
    rope = torch.from_numpy(ref.rope_table(200, D)).cuda()
    ko = torch.empty_like(k)
    cr.convrot_rope_append(q, k, v, rope, torch.from_numpy(run.astype(np.int32)).cuda(), slots.cuda(), **c, k_out=ko)
    mine = {x: t[pages - 4:].clone() for x, t in c.items()}
    assert not any(t[:pages - 4].any() for t in c.values())
    small = table - (pages - 4)
    got = cr.convrot_attention_decode(q[:2], block_table=table.cuda(), seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(), **c)
    near = dict(mine, q=q[:2], block_table=small.clamp_min(0), seq_lens=None)
    o, tol = oracle_decode(near, lens)
    assert cr.convrot_device_status() == 0
    within(f64(got), o, tol, "decode")
    if not i8:
        page_of = small.numpy()[seq, run // page]
        assert torch.equal(mine["v_cache"].cpu()[page_of, :, run % page], v.cpu())
        assert torch.equal(mine["k_cache"].cpu()[page_of, :, run % page], ko.cpu())


# ------------------------------------------------------------------ streams and graphs
def test_other_streams_at_the_same_time(cr):
    """Calls on two streams at once, each with results of its own."""
    cases = [decode_case(20 + i, [2500, 31], 8, 2, 128, 16, bool(i)) for i in range(2)]
    want = [cr.convrot_attention_decode(**c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cr.convrot_attention_decode(**cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])


def test_two_captured_graphs_replayed_at_the_same_time(cr):
    """Graphs captured one after another on the same stream and replayed on two
    others share no scratch memory; replays see new inputs and lengths."""
    cases = [decode_case(30 + i, [2600, 31, 900], 8, 2, 128, 16, bool(i)) for i in range(2)]
    outs, graphs = [], []
    for c in cases:
        cr.convrot_attention_decode(**c)
    torch.cuda.synchronize()
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cr.convrot_attention_decode(**c))
        graphs.append(g)
    for new in ([2600, 31, 900], [1, 0, 333]):
        for c in cases:
            c["seq_lens"].copy_(torch.tensor(new, dtype=torch.int32))
            c["q"].copy_(c["q"].flip(0))
        want = [cr.convrot_attention_decode(**c) for c in cases]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in cases]
        for _ in range(20):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert cr.convrot_device_status() == 0


def test_captured_append_and_prompt(cr):
    c = append_case(40, 64, 8, 2, 128, 128, 16, False, True)
    q, k, v, cu, _ = prompt_case(41, [60, 200], [60, 200], 4, 2, 64)
    cu = torch.from_numpy(cu).cuda()
    ko = torch.empty(c["k"].shape, dtype=torch.bfloat16, device="cuda")
    cr.convrot_rope_append(**c, k_out=ko), cr.convrot_attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qo, _ = cr.convrot_rope_append(**c, k_out=ko)
        o = cr.convrot_attention_prompt(q, k, v, cu)
    c["q"].copy_(c["q"].flip(0))
    c["slots"].copy_(c["slots"].flip(0))
    q.copy_(q.flip(0))
    cu.copy_(torch.tensor([0, 130, 260]))
    before = {n: t.clone() for n, t in c.items()}
    g.replay()
    torch.cuda.synchronize()
    check_append(c, before, qo, ko)
    ref_o, tol = ref.packed_attention(f64(q), f64(k), f64(v), [0, 130, 260], [0, 130, 260], 64 ** -0.5, True)
    within(f64(o), ref_o, tol, "replayed prompt")


def test_decode_refuses_a_short_workspace(cr):
    import ctypes
    c = decode_case(51, [70], 8, 2, 128, 16, False)
    need = cr.convrot_attention_decode_workspace_bytes(1, 8, 2, 128)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out = torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    for p, n, want in ((None, need, 7), (ws.data_ptr(), need - 1, 7), (ws.data_ptr() + 16, need, 3), (ws.data_ptr(), need, 0)):
        st = cr.lib().convrot_attention_decode(
            c["q"].data_ptr(), 1024, 1, 8, 2, 128, c["k_cache"].data_ptr(), c["v_cache"].data_ptr(), None, None,
            c["k_cache"].shape[0], 16, c["block_table"].data_ptr(), c["block_table"].shape[1], c["block_table"].shape[1],
            c["seq_lens"].data_ptr(), 0.1, out.data_ptr(), 1024, p, n, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert st == want
        assert (out == 7).all() == (want != 0)


def test_decode_leaves_its_workspace_zero(cr):
    """The linears' contract: a Workspace may serve both."""
    ws = cr.Workspace()
    for lens in ([5000, 3], [64 * 7] * 40, [1]):
        c = decode_case(50, lens, 8, 2, 128, 16, False)
        check_decode(cr, c, lens, workspace=ws)
        assert not ws.buf.any()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 16), (64, 8, 4, 64)])
def test_attention_block_prompts_then_tokens(cr, D, Hq, Hkv, page, i8):
    """ConvRotAttention over packed prompts, then two decode steps of all
    sequences: the wiring against the operators one by one, the operators
    against the oracle, each on the inputs it got."""
    hidden, lens = 512, [70, 3, 129]
    W = [randn(60 + i, n, hidden, std=0.05) for i, n in enumerate((Hq * D, Hkv * D, Hkv * D))]
    Wo = randn(63, hidden, Hq * D, std=0.05)
    g = torch.Generator().manual_seed(1)
    norms = [torch.randn(D, generator=g).cuda() * 0.1 for _ in range(2)]
    rope = cr.rope_table(200, D, device="cuda")
    layer = cr.ConvRotAttention(*W, Wo, q_heads=Hq, kv_heads=Hkv, rope=rope, norm_w=torch.zeros(hidden).cuda(),
                                q_norm=norms[0], k_norm=norms[1])
    need = [-(-(n + 2) // page) for n in lens]
    cache = cr.PagedKVCache(sum(need) + 1, Hkv, D, page_size=page, int8=i8)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    perm, at = torch.randperm(sum(need) + 1, generator=g), 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    table = table.cuda()
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()

    def pieces(x, pos, slots, rotated):
        q, k, v = (t.unflatten(1, (-1, D)).clone() for t in layer.qkv(x))
        c = dict(q=q, k=k, v=v, rope=rope, positions=pos, slots=slots, q_norm=norms[0], k_norm=norms[1],
                 k_cache=cache.k.clone(), v_cache=cache.v.clone())
        if i8:
            c |= dict(k_scale=cache.k_scale.clone(), v_scale=cache.v_scale.clone())
        before = {n: t.clone() for n, t in c.items()}
        qo, ko = cr.convrot_rope_append(**c, k_out=torch.empty_like(k) if rotated else None)
        check_append(c, before, qo, ko)
        return c, qo, ko

    def same_cache(c):
        assert torch.equal(cache.k, c["k_cache"]) and torch.equal(cache.v, c["v_cache"])
        if i8:
            assert torch.equal(cache.k_scale, c["k_scale"]) and torch.equal(cache.v_scale, c["v_scale"])

    x = randn(64, sum(lens), hidden)
    slots = cache.slots(table, seq, pos)
    c, q, k = pieces(x, pos, slots, True)
    o = cr.convrot_attention_prompt(q, k, c["v"], cu)
    want, tol = ref.packed_attention(f64(q), f64(k), f64(c["v"]), cu.tolist(), cu.tolist(), D ** -0.5, True)
    within(f64(o), want, tol, "prompt")
    y = layer.prompt(x, cu, pos, slots, cache)
    assert y.shape == (sum(lens), hidden) and torch.equal(y, layer.o(o.flatten(1)))
    same_cache(c)
    for step in range(2):
        x = randn(65 + step, len(lens), hidden)
        now = torch.tensor([n + step for n in lens], dtype=torch.int32).cuda()
        slots = cache.slots(table, torch.arange(len(lens)).cuda(), now)
        c, q, _ = pieces(x, now, slots, False)
        a = dict(q=q, k_cache=c["k_cache"], v_cache=c["v_cache"], block_table=table, seq_lens=now + 1)
        if i8:
            a |= dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
        o = check_decode(cr, a, (now + 1).tolist())
        y = layer.decode(x, now, slots, cache, table, now + 1)
        assert torch.equal(y, layer.o(o.flatten(1)))
        same_cache(c)
    assert cr.convrot_device_status() == 0


def test_decode_step_agrees_with_the_prompt_s_last_row(cr):
    """The last row of a prompt's attention and the same token decoded over the
    cache are the same sum: both within their bounds of the oracle's value."""
    n, Hq, Hkv, D, page = 300, 8, 2, 128, 16
    c = append_case(70, n, Hq, Hkv, D, D, page, False, False, rows=n)
    c["positions"] = torch.arange(n, dtype=torch.int32).cuda()
    pages = c["k_cache"].shape[0]
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2))[None].int()
    run = torch.arange(n)
    c["slots"] = (table[0, run // page].long() * page + run % page).cuda()
    ko = torch.empty(n, Hkv, D, dtype=torch.bfloat16, device="cuda")
    q, k = cr.convrot_rope_append(**c, k_out=ko)
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    a = cr.convrot_attention_prompt(q, k, c["v"], cu)[-1]
    b = cr.convrot_attention_decode(q[-1:], c["k_cache"], c["v_cache"], table.cuda(),
                                    torch.tensor([n], dtype=torch.int32).cuda())[0]
    o, tol = ref.packed_attention(f64(q[-1:]), f64(k), f64(c["v"]), [0, 1], [0, n], D ** -0.5, True)
    within(f64(a), o[0], tol[0], "prompt")
    within(f64(b), o[0], tol[0], "decode")


# ------------------------------------------------------------------ the ends of the ranges
def test_empty_calls(cr):
    """No tokens, no sequences, no keys at all."""
    q, k = randn(1, 5, 4, 64), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, none = torch.tensor([0, 3, 5], dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    assert not cr.convrot_attention_prompt(q, k, k, cu, none).any()
    assert not cr.convrot_attention_prompt(q, k, k, cu, none, causal=False).any()
    out = torch.full_like(q, 7.0)
    cr.convrot_attention_prompt(q, q, q, torch.zeros(1, dtype=torch.int32).cuda(), out=out)   # no sequence
    assert (out == 7).all()
    assert cr.convrot_attention_prompt(q[:0], k, k, none).shape == (0, 4, 64)
    c = append_case(1, 4, 4, 2, 64, 64, 16, False, False)
    c = {n: t[:0] if n in ("q", "k", "v", "positions", "slots") else t for n, t in c.items()}
    before = c["k_cache"].clone()
    assert cr.convrot_rope_append(**c)[0].shape == (0, 4, 64) and torch.equal(before, c["k_cache"])
    d = decode_case(2, [5], 4, 2, 64, 16, False)
    assert cr.convrot_attention_decode(d["q"][:0], d["k_cache"], d["v_cache"], d["block_table"][:0],
                                       d["seq_lens"][:0]).shape == (0, 4, 64)
    assert cr.convrot_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_one_key_head_for_very_many(cr, D):
    check_prompt(cr, *prompt_case(3, [19, 2], [19, 2], 1024, 1, D))
    check_decode(cr, decode_case(4, [33, 200], 1024, 1, D, 32, True), [33, 200])
    c = append_case(5, 9, 1000, 25, D, D, 16, True, True)
    before, q, k = run_append(cr, c)
    check_append(c, before, q, k)


def test_prompts_on_two_streams_at_once(cr):
    cases = []
    for i, lens in enumerate(([700, 3, 130], [1025, 64])):
        q, k, v, cu, _ = prompt_case(70 + i, lens, lens, 8, 2, 128 if i else 64)
        cases.append((q, k, v, torch.from_numpy(cu).cuda()))
    want = [cr.convrot_attention_prompt(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cr.convrot_attention_prompt(*cases[i]))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)
    assert cr.convrot_device_status() == 0


def test_long_prompt_rows(cr):
    """Rows spread over a long prompt: many tiles, references raised on the way."""
    n, Hq, Hkv, D = 5003, 4, 1, 128
    q, k, v, cu, _ = prompt_case(80, [n], [n], Hq, Hkv, D)
    k[n // 2:] = k[n // 2:].float() * 3          # later keys score far higher
    got = f64(cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda()))
    K, V = f64(k)[:, 0], f64(v)[:, 0]
    for t in (0, 1, 63, 64, 127, 128, 1000, n // 2 - 1, n // 2, n // 2 + 1, 4095, 4096, n - 2, n - 1):
        for h in range(Hq):
            o, tol = ref.attention(f64(q[t])[h][None], K, V, D ** -0.5, np.arange(n)[None] <= t)
            within(got[t, h], o[0], tol[0], f"row {t} head {h}")

# ------------------------------------------------------------------ many blocks per CTA
def long_decode_case(seed, lens, Hq, Hkv, D, page, i8):
    """Contexts of thousands of keys, made on the GPU; keys of the later half of
    every page row score three times as high as the others."""
    g = torch.Generator("cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(need)), -7, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    shape = (pages, Hkv, page, D)
    c = dict(q=(torch.randn(len(lens), Hq, D, generator=g, device="cuda") * 2).to(torch.bfloat16), block_table=table,
             seq_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    wide = torch.zeros(pages, dtype=torch.bool, device="cuda")
    for i, n in enumerate(need):
        wide[table[i, n // 2:n].long()] = True
    for x in "kv":
        if i8:
            c[x + "_cache"] = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
            c[x + "_scale"] = torch.rand(shape[:3], generator=g, device="cuda") * 0.02 + 0.005
        else:
            c[x + "_cache"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    c["k_scale" if i8 else "k_cache"][wide] *= 3
    return c


def oracle_rows(c, lens, b, h):
    """The oracle's (o, tol) of one head of one sequence."""
    n, page = lens[b], c["k_cache"].shape[2]
    kv = h // (c["q"].shape[1] // c["k_cache"].shape[1])
    at = torch.arange(n, device="cuda")
    where = (c["block_table"][b].long()[at // page], torch.full_like(at, kv), at % page)
    k, v = (c[x][where].double().cpu().numpy() for x in ("k_cache", "v_cache"))
    vs = None
    if c.get("k_scale") is not None:
        vs = c["v_scale"][where].double().cpu().numpy()
        k, v = k * c["k_scale"][where].double().cpu().numpy()[:, None], v * vs[:, None]
    o, tol = ref.attention(f64(c["q"])[b, h][None], k, v, c["q"].shape[2] ** -0.5, np.ones((1, n), bool), vs)
    return o[0], tol[0]


LONG = [(32, 8, 128, 16), (64, 8, 128, 48), (16, 4, 64, 64), (16, 2, 64, 128), (20, 1, 128, 16)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page", LONG)
def test_decode_many_blocks_per_cta(cr, Hq, Hkv, D, page, i8):
    """Stretches of dozens of blocks: every ring slot taken again and again,
    several batches of pages per sequence, references raised on the way."""
    rng = np.random.default_rng(Hq + D)
    seqs = 400 // Hkv
    lens = [int(n) for n in rng.integers(1, 6000, seqs)]
    lens[:3] = [6000, 1, 5953]
    c = long_decode_case(seqs, lens, Hq, Hkv, D, page, i8)
    got = cr.convrot_attention_decode(**c)
    assert cr.convrot_device_status() == 0
    got = f64(got)
    assert np.isfinite(got).all()
    for b in [0, 1, 2, seqs - 1] + [int(x) for x in rng.integers(3, seqs, 12)]:
        for h in {0, Hq - 1, int(rng.integers(Hq))}:
            o, tol = oracle_rows(c, lens, b, h)
            within(got[b, h], o, tol, f"sequence {b} head {h}")


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,page", LONG)
def test_decode_heads_do_not_touch_one_another(cr, Hq, Hkv, D, page, i8):
    """A head's result depends, bit by bit, on its own query alone: other
    queries of its group, and what other kernels left in shared memory, move
    nothing."""
    lens = [3000 - 17 * i for i in range(160 // Hkv)]
    c = long_decode_case(7, lens, Hq, Hkv, D, page, i8)
    want = cr.convrot_attention_decode(**c)
    group = Hq // Hkv
    first = torch.arange(Hq, device="cuda") % group == 0
    other = dict(c, q=torch.where(first[:, None], c["q"], (c["q"].float() * 8).to(torch.bfloat16)))
    got = cr.convrot_attention_decode(**other)
    assert torch.equal(got[:, first], want[:, first])
    noise = long_decode_case(8, lens, 16, 1, 128, 16, not i8)
    noise["q"] *= 30
    p = prompt_case(9, [700], [700], 8, 2, 128)
    for i in range(6):
        if i % 2:
            cr.convrot_attention_decode(**noise)
        else:
            cr.convrot_attention_prompt(*(x * 100 for x in p[:3]), torch.from_numpy(p[3]).cuda())
        assert torch.equal(cr.convrot_attention_decode(**c), want)
    assert cr.convrot_device_status() == 0


# ------------------------------------------------------------------ pages that cannot be read
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_pages_that_cannot_be_read_are_left_out(cr, page, i8):
    """Keys of a page outside the cache take no part; a sequence none of whose
    pages can be read is 0, within one CTA's stretch and over many."""
    for lens in ([40, 16, 9, 300], [9000], [1, 9000, 5]):
        c = decode_case(11, lens, 4, 2, 64, page, i8)
        good = check_decode(cr, c, lens)
        for row in range(len(lens)):
            d = dict(c, block_table=c["block_table"].clone())
            d["block_table"][row] = -1
            got = cr.convrot_attention_decode(**d)
            assert cr.convrot_device_status() == 2 and cr.convrot_device_status() == 0
            assert not got[row].any(), "a sequence without a page that can be read"
            keep = [i for i in range(len(lens)) if i != row]
            assert torch.equal(got[keep], good[keep])
    lens = [200]
    c = decode_case(12, lens, 4, 2, 64, page, i8)
    table = c["block_table"].clone()
    table[0, 1] = 10 ** 6
    got = f64(cr.convrot_attention_decode(**dict(c, block_table=table)))
    assert cr.convrot_device_status() == 2
    see = np.ones((1, 200), bool)
    see[0, page:2 * page] = False
    s = [None if c.get(x) is None else c[x].cpu().double().numpy() for x in ("k_scale", "v_scale")]
    rows = c["block_table"].cpu().numpy()[0]
    k, v = ref.cache_rows(f64(c["k_cache"]), s[0], rows, 200), ref.cache_rows(f64(c["v_cache"]), s[1], rows, 200)
    at = np.arange(200)
    for h in range(4):
        vs = None if s[1] is None else s[1][rows[at // page], :, at % page][:, h // 2]
        o, tol = ref.attention(f64(c["q"])[0, h][None], k[:, h // 2], v[:, h // 2], 64 ** -0.5, see, vs)
        within(got[0, h], o[0], tol[0], f"head {h}")


def test_decode_only_scores_of_minus_infinity(cr):
    """Keys that are there and all score -inf: the softmax has no value, and
    the row is NaN, not the 0 of a sequence without keys."""
    for lens in ([40], [9000]):
        c = decode_case(13, lens, 2, 1, 64, 16, False, fill=0.0)
        c["q"][..., 0] = 300.0
        c["k_cache"][..., 0] = -3e38
        assert torch.isnan(cr.convrot_attention_decode(**c)).all()


# ------------------------------------------------------------------ many units per CTA
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (32, 4, 64), (40, 8, 64), (8, 8, 128)])
def test_prompt_many_units_per_cta(cr, Hq, Hkv, D, causal):
    """Hundreds of units of one to eleven key tiles, so that CTAs take over one
    unit after another: the same bits as each prompt's heads alone, where every
    unit has a CTA of its own, and sampled rows within the oracle's bounds."""
    group = Hq // Hkv
    lens = [1333, 1, 700, 64, 65, 1025, 128, 300, 999, 17, 1280, 450]
    if group == 1:
        lens = lens * 3
    q, k, v, cu, _ = prompt_case(90 + Hq, lens, lens, Hq, Hkv, D)
    units = sum(-(-n // (2 * (128 // group))) for n in lens) * Hkv
    assert units > 300
    whole = cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda(), causal=causal)
    for _ in range(3):
        assert torch.equal(whole, cr.convrot_attention_prompt(q, k, v, torch.from_numpy(cu).cuda(), causal=causal))
    for a, b in zip(cu[:12], cu[1:]):
        one = torch.tensor([0, b - a], dtype=torch.int32).cuda()
        for h in range(Hkv):
            mine = slice(h * group, (h + 1) * group)
            got = cr.convrot_attention_prompt(q[a:b, mine], k[a:b, h:h + 1], v[a:b, h:h + 1], one, causal=causal)
            assert torch.equal(whole[a:b, mine], got)
    assert cr.convrot_device_status() == 0
    rng = np.random.default_rng(Hq)
    for s in rng.integers(0, len(lens), 8):
        a, n, h = int(cu[s]), lens[s], int(rng.integers(Hq))
        i = int(rng.integers(n))
        see = np.arange(n)[None] <= (i if causal else n)
        o, tol = ref.attention(f64(q[a + i, h])[None], f64(k[a:a + n, h // group]), f64(v[a:a + n, h // group]), D ** -0.5, see)
        within(f64(whole[a + i, h]), o[0], tol[0], f"sequence {s} row {i} head {h}")


# ------------------------------------------------------------------ slots
def test_append_at_slots_the_table_has_no_place_for(cr):
    """Padding is not stored; a token past its sequence's pages is left out and
    reported; the others are as ever."""
    cache = cr.PagedKVCache(6, 2, 64, page_size=16)
    table = torch.tensor([[4, 1], [0, -1]], dtype=torch.int32).cuda()
    seq, pos = torch.tensor([0, 0, 1, 1, -1, 0]).cuda(), torch.tensor([0, 31, 3, 20, 5, 7], dtype=torch.int32).cuda()
    c = append_case(14, 6, 4, 2, 64, 64, 16, False, False, rows=50)
    c |= dict(k_cache=cache.k, v_cache=cache.v, positions=pos, slots=cache.slots(table, seq, pos))
    before, q, k = run_append(cr, c)               # nothing to report: padding and a page that is not there
    check_append(c, before, q, k)
    pos = pos.clone()
    pos[1], seq[2] = 32, 9
    c |= dict(positions=pos, slots=cache.slots(table, seq, pos))
    before = {n: t.clone() for n, t in c.items()}
    q, k = torch.zeros_like(q), torch.zeros_like(k)
    cr.convrot_rope_append(**c, q_out=q, k_out=k)
    assert cr.convrot_device_status() == 2 and cr.convrot_device_status() == 0
    assert not q[1:3].any() and not k[1:3].any()
    keep = torch.tensor([0, 3, 4, 5])
    pick = lambda d: {n: t[keep] if n in ("q", "k", "v", "positions", "slots") else t for n, t in d.items()}
    check_append(pick(c), pick(before), q[keep], k[keep])


# ------------------------------------------------------------------ results beside inputs
def test_results_beside_and_in_place_of_inputs(cr):
    """Results in columns of the buffer that holds the inputs, and a decode in
    place: the same bits as results of their own, nothing else touched."""
    T, Hq, Hkv, D = 150, 8, 2, 64
    wide = randn(15, T, (2 * Hq + 2 * Hkv) * D)
    q, k, v, out = (x.view(T, -1, D) for x in wide.split([Hq * D, Hkv * D, Hkv * D, Hq * D], 1))
    before = wide.clone()
    cu = torch.tensor([0, 90, T], dtype=torch.int32).cuda()
    want = cr.convrot_attention_prompt(q, k, v, cu)
    assert cr.convrot_attention_prompt(q, k, v, cu, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, want) and torch.equal(wide[:, :(Hq + 2 * Hkv) * D], before[:, :(Hq + 2 * Hkv) * D])
    for bad in (q, wide[:, D:(Hq + 1) * D].view(T, Hq, D), wide[:, (Hq + 1) * D:(2 * Hq + 1) * D].view(T, Hq, D)):
        with pytest.raises(cr.ConvRotError, match="UNSUPPORTED"):
            cr.convrot_attention_prompt(q, k, v, cu, out=bad)
    c = append_case(16, T, Hq, Hkv, D, D, 16, False, True)
    with pytest.raises(cr.ConvRotError, match="UNSUPPORTED"):
        cr.convrot_rope_append(**c, q_out=c["q"], k_out=c["q"][:, 1:1 + Hkv])
    with pytest.raises(cr.ConvRotError, match="UNSUPPORTED"):
        cr.convrot_rope_append(**(c | dict(v_cache=c["k_cache"])))
    lens = [300, 4, 0, 7000]
    d = decode_case(17, lens, Hq, Hkv, D, 16, False)
    want = cr.convrot_attention_decode(**d)
    assert cr.convrot_attention_decode(**d, out=d["q"]) is d["q"] and torch.equal(d["q"], want)
    with pytest.raises(cr.ConvRotError, match="UNSUPPORTED"):
        cr.convrot_attention_decode(**(d | dict(q=d["q"][:3], block_table=d["block_table"][:3], seq_lens=d["seq_lens"][:3])),
                                    out=d["q"][1:])
    assert cr.convrot_device_status() == 0


# ------------------------------------------------------------------ workspaces and graphs
def workspace_calls(cr, i):
    """A call that takes a Workspace, and one that needs a larger one."""
    if i == 2:
        g = torch.Generator().manual_seed(3)
        X, W = (torch.randint(-127, 128, (n, 12288), generator=g, dtype=torch.int16).to(torch.int8).cuda() for n in (768, 6400))
        return (lambda ws: cr.convrot_int8_gemm_s32(X[:16].contiguous(), W[:4096].contiguous(), workspace=ws),
                lambda ws: cr.convrot_int8_gemm_s32(X, W, workspace=ws))
    small, big = (decode_case(100 + h, [3000, 70], h, 1, 128, 16, bool(i)) for h in (2, 16))
    return lambda ws: cr.convrot_attention_decode(**small, workspace=ws), lambda ws: cr.convrot_attention_decode(**big, workspace=ws)


@pytest.mark.parametrize("i", range(3))
def test_workspace_captured_before_any_call(cr, i):
    """Eager calls between a capture and its first replay, a second graph
    replayed before the first, and replays after either."""
    f, _ = workspace_calls(cr, i)
    want = f(cr.Workspace())
    ws, graphs, outs = cr.Workspace(), [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f(ws))
    for _ in range(2):
        assert torch.equal(f(ws), want)
        for g, o in reversed(list(zip(graphs, outs))):
            o.zero_()
            g.replay()
            assert torch.equal(o, want)
    assert cr.convrot_device_status() == 0


@pytest.mark.parametrize("i", range(3))
def test_workspace_that_grows_behind_a_captured_graph(cr, i):
    """The graph goes on using the buffer that it was captured with."""
    f, larger = workspace_calls(cr, i)
    ws = cr.Workspace()
    want = f(ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(ws)
    size = ws.buf.numel()
    want_larger = larger(ws)
    assert ws.buf.numel() > size
    taken = [torch.full((size,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(8)]   # what was freed, if it was
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(larger(ws), want_larger)
    assert all((t == 0x55).all() for t in taken) and cr.convrot_device_status() == 0


def test_decode_refuses_a_workspace_of_another_device(cr):
    c = decode_case(52, [70], 8, 2, 128, 16, False)
    ws = cr.Workspace()
    ws.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="the workspace is on cuda:1"):
        cr.convrot_attention_decode(**c, workspace=ws)


# ------------------------------------------------------------------ values near the end of fp32
def test_decode_int8_values_near_the_end_of_the_range(cr):
    """A key whose probability, against a reference 2^7.5 below its score, times
    its value's scale lies above 2^126: its share of the result is there."""
    seqs, n, page, D = 700, 256, 16, 64        # two blocks each, several sequences to a CTA
    k, v = (torch.zeros(n // page, 1, page, D, dtype=torch.int8) for _ in range(2))
    ks, vs = torch.full((n // page, 1, page), 1e-3), torch.full((n // page, 1, page), 1e30)
    at = 200 // page, 0, 200 % page
    k[at][0], ks[at] = 127, 7.5 * np.log(2) / 127
    v[at], vs[at] = 1, 6e35
    v[at][0] = 127                             # this element's sum itself leaves fp32
    q = torch.zeros(seqs, 1, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    table = torch.arange(n // page, dtype=torch.int32).repeat(seqs, 1)
    got = cr.convrot_attention_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), torch.full((seqs,), n, dtype=torch.int32).cuda(),
                                      k_scale=ks.cuda(), v_scale=vs.cuda(), scale=1.0)
    rows = [x.double().numpy().reshape(n, D) * s.double().numpy().reshape(n, 1) for x, s in ((k, ks), (v, vs))]
    o, tol = ref.attention(f64(q[0]), rows[0], rows[1], 1.0, np.ones((1, n), bool), vs.double().numpy().reshape(n))
    assert o[0, 1] > 2e35
    for b in range(seqs):
        within(f64(got)[b, 0, 1:], o[0, 1:], tol[0, 1:], f"sequence {b}")


# ------------------------------------------------------------------ the block, captured and padded
@pytest.mark.parametrize("warm", [False, True])
@pytest.mark.parametrize("i8", [False, True])
def test_attention_block_captured_and_padded(cr, i8, warm):
    """A prompt and a token step of ConvRotAttention as captured graphs, with and
    without calls before the capture, over batches padded to a fixed size:
    replays with other tokens, pages and lengths are the eager calls' bits."""
    Hq, Hkv, D, hidden, page, rows = 8, 2, 128, 512, 16, 256
    W = [randn(160 + i, n, hidden, std=0.05) for i, n in enumerate((Hq * D, Hkv * D, Hkv * D))]
    Wo = randn(163, hidden, Hq * D, std=0.05)

    def layer():
        return cr.ConvRotAttention(*W, Wo, q_heads=Hq, kv_heads=Hkv, rope=cr.rope_table(300, D, device="cuda"),
                                   norm_w=torch.zeros(hidden).cuda())

    def batch(seed, lens):
        """Tokens of whole prompts padded to `rows`, and one token each padded to 8."""
        g = torch.Generator().manual_seed(seed)
        need = [-(-(n + 1) // page) for n in lens]
        perm, at = torch.randperm(40, generator=g).int(), 0
        table = torch.full((8, 16), -1, dtype=torch.int32)
        for i, n in enumerate(need):
            table[i, :n], at = perm[at:at + n], at + n
        pad = rows - sum(lens)
        seq = torch.cat([torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)), torch.full((pad,), -1)])
        pos = torch.cat([torch.arange(n) for n in lens] + [torch.zeros(pad, dtype=torch.int64)]).int()
        cu = torch.tensor([0] + lens + [0] * (8 - len(lens))).cumsum(0).int()
        n = torch.tensor(lens + [0] * (8 - len(lens)), dtype=torch.int32)
        live = torch.arange(8) < len(lens)
        s = cr.PagedKVCache.slots
        cache = cr.PagedKVCache.__new__(cr.PagedKVCache)
        cache.page_size = page
        b = dict(x=randn(seed, rows, hidden).cpu(), cu=cu, pos=pos, slots=s(cache, table, seq, pos), x1=randn(seed + 1, 8, hidden).cpu(),
                 pos1=n, slots1=s(cache, table, torch.where(live, torch.arange(8), -1), n), table=table,
                 lens1=torch.where(live, n + 1, 0).int())
        return {k: t.cuda() for k, t in b.items()}

    def step(layer, cache, b):
        return (layer.prompt(b["x"], b["cu"], b["pos"], b["slots"], cache),
                layer.decode(b["x1"], b["pos1"], b["slots1"], cache, b["table"], b["lens1"]))

    batches = [(200, [70, 3, 129]), (300, [1]), (400, [17, 16, 15, 40, 100, 1, 2])]
    eager, want = layer(), []
    for seed, lens in batches:
        cache = cr.PagedKVCache(40, Hkv, D, page_size=page, int8=i8)
        y, y1 = step(eager, cache, batch(seed, lens))
        assert torch.isfinite(y[:sum(lens)]).all() and torch.isfinite(y1).all() and not y1[len(lens):].any()
        want.append((y, y1, cache))
    mine, held = layer(), batch(*batches[0])
    cache = cr.PagedKVCache(40, Hkv, D, page_size=page, int8=i8)
    if warm:
        step(mine, cache, held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(mine, cache, held)
    for i in (2, 0, 1, 2):
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            if t is not None:
                t.zero_()
        for k, t in batch(*batches[i]).items():
            held[k].copy_(t)
        graph.replay()
        n = sum(batches[i][1])
        assert torch.equal(out[0][:n], want[i][0][:n]) and torch.equal(out[1], want[i][1])
        assert torch.equal(cache.k, want[i][2].k) and torch.equal(cache.v, want[i][2].v)
    assert cr.convrot_device_status() == 0


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 48), (128, 48), (128, 80), (128, 112)])
def test_append_rotation_widths_between(cr, D, rot, i8):
    """Widths that end inside a lane's share of the head."""
    c = append_case(D + rot, 50, 6, 3, D, rot, 48, i8, True, pad=7)
    before, q, k = run_append(cr, c)
    check_append(c, before, q, k)


def test_rows_far_apart(cr):
    """Row strides with which offsets pass 2^32 elements: the bits of the same
    rows side by side."""
    T, stride, Hq, Hkv, D = 1030, 1 << 22, 8, 2, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    q, k, v, out = (big.as_strided((T, h, D), (stride, D, 1), at) for h, at in ((Hq, 0), (Hkv, 2048), (Hkv, 4096), (Hq, 8192)))
    near = [randn(20 + i, *x.shape) for i, x in enumerate((q, k, v))]
    for x, y in zip((q, k, v), near):
        x.copy_(y)
    cu = torch.tensor([0, 500, T], dtype=torch.int32).cuda()
    assert torch.equal(cr.convrot_attention_prompt(q, k, v, cu, out=out), cr.convrot_attention_prompt(*near, cu))
    rope, pos = cr.rope_table(T, D, device="cuda"), torch.arange(T, dtype=torch.int32).cuda()
    slots = torch.randperm(70 * 16, generator=torch.Generator().manual_seed(1))[:T].cuda()
    caches = [cr.PagedKVCache(70, Hkv, D, page_size=16) for _ in range(2)]
    far = cr.convrot_rope_append(q, k, v, rope, pos, slots, caches[0].k, caches[0].v, q_out=out)[0]
    assert torch.equal(far, cr.convrot_rope_append(*near, rope, pos, slots, caches[1].k, caches[1].v)[0])
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    g = torch.Generator().manual_seed(2)
    table = torch.randint(0, 70, (T, 3), generator=g, dtype=torch.int32).cuda()
    lens = torch.randint(0, 49, (T,), generator=g, dtype=torch.int32).cuda()
    args = caches[0].k, caches[0].v, table, lens
    assert torch.equal(cr.convrot_attention_decode(q, *args, out=out), cr.convrot_attention_decode(near[0], *args))
    assert cr.convrot_device_status() == 0
