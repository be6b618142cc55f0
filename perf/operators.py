"""Cases, plain forms and 64-bit values of the attention operators.

Three operators stand between the q/k/v projection and the o projection of a
decoder layer (32 query heads x 128, 8 key/value heads x 128, hidden 4096):

* append: per-head RMSNorm (optional) and position rotation of q and k, and the
  write of k and v into a paged cache (bf16, or int8 with one fp32 scale per
  token and head);
* prompt: causal attention over whole prompts, packed one after another;
* decode: attention of one new token per sequence over the paged cache.

A case is a dict of plain values; its sequence lengths follow from the case
alone, its inputs from the case and a seed.
"""
import math
import random

import torch

own = False

THETA = 1e6      # base of the rotation's angles
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence being decoded: one token per layer and step, latency only
        dict(name="append_1_token", op="append", kind="tokens", tokens=1, pad=0, ctx=900, hq=32, hkv=8, d=128,
             rot=128, page=16, cache="bf16", norm=False),
        # a decode batch padded to 256 rows for a captured graph (the last 19 rows have no slot), int8 cache
        dict(name="append_256_tokens_int8", op="append", kind="tokens", tokens=256, pad=19, ctx=4000, hq=32, hkv=8,
             d=128, rot=128, page=64, cache="int8", norm=True),
        # 34 text-encoder prompts of different lengths, packed; the rotated keys go to the attention too
        dict(name="append_34_prompts", op="append", kind="prompts", seqs=34, lo=16, hi=300, hq=32, hkv=8, d=128,
             rot=128, page=16, cache="bf16", norm=True),
        # the longest single prompt of the token sweep
        dict(name="append_prompt_8192", op="append", kind="prompts", seqs=1, lo=8192, hi=8192, hq=32, hkv=8, d=128,
             rot=128, page=64, cache="bf16", norm=False),
        # 34 text-encoder prompts, packed: every sequence ends inside a tile
        dict(name="prompt_34_short", op="prompt", seqs=34, lo=16, hi=300, hq=32, hkv=8, d=128),
        # one prompt of the decoder layer's 2048 tokens
        dict(name="prompt_2048", op="prompt", seqs=1, lo=2048, hi=2048, hq=32, hkv=8, d=128),
        # very different lengths in one pack, narrow heads in groups of eight
        dict(name="prompt_packed_d64", op="prompt", seqs=12, lo=1, hi=1333, hq=32, hkv=4, d=64),
        # the longest prompt of the token sweep
        dict(name="prompt_8192", op="prompt", seqs=1, lo=8192, hi=8192, hq=32, hkv=8, d=128),
        # one short conversation: latency only
        dict(name="decode_1x777", op="decode", seqs=1, lo=777, hi=777, hq=32, hkv=8, d=128, page=16, cache="bf16"),
        # one long context: all of the GPU has to work on eight key/value heads
        dict(name="decode_1x131071", op="decode", seqs=1, lo=131071, hi=131071, hq=32, hkv=8, d=128, page=64,
             cache="bf16"),
        # a serving batch with contexts of every length
        dict(name="decode_64_ragged", op="decode", seqs=64, lo=1, hi=8192, hq=32, hkv=8, d=128, page=32, cache="bf16"),
        # the same with twice the sequences on an int8 cache
        dict(name="decode_128_ragged_int8", op="decode", seqs=128, lo=1, hi=8192, hq=32, hkv=8, d=128, page=64,
             cache="int8"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "prompt", "decode"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([g for g in (1, 2, 4, 5, 8) if g * hkv <= 32])
    if op == "prompt":
        total = _log(rng, 8, 8192)                  # tokens of the whole pack
        seqs = _log(rng, 1, min(64, total))
        hi = max(1, total // seqs)
        return dict(op=op, seqs=seqs, lo=max(1, hi - rng.randrange(hi)), hi=hi, hq=hq, hkv=hkv, d=d)
    page = rng.choice([16, 32, 48, 64, 128])
    cache = rng.choice(["bf16", "int8"])
    if op == "append":
        rot = rng.choice([d, d, d // 2, 32])
        norm = rng.random() < 0.5
        if rng.random() < 0.5:
            tokens = _log(rng, 1, 512)
            return dict(op=op, kind="tokens", tokens=tokens, pad=rng.randrange(1 + tokens // 4), ctx=_log(rng, 1, 32768),
                        hq=hq, hkv=hkv, d=d, rot=rot, page=page, cache=cache, norm=norm)
        total = _log(rng, 8, 8192)
        seqs = _log(rng, 1, min(64, total))
        hi = max(1, total // seqs)
        return dict(op=op, kind="prompts", seqs=seqs, lo=max(1, hi - rng.randrange(hi)), hi=hi, hq=hq, hkv=hkv, d=d,
                    rot=rot, page=page, cache=cache, norm=norm)
    seqs = _log(rng, 1, 128)
    hi = _log(rng, 1, min(131072, (1 << 19) // seqs))
    return dict(op=op, seqs=seqs, lo=max(1, hi - rng.randrange(hi)), hi=hi, hq=hq, hkv=hkv, d=d, page=page, cache=cache)


def _lengths(case):
    """The sequences' lengths: lo and hi are among them, the rest lie between."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["lo"], case["hi"]))
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n[0] = case["hi"]
    if len(n) > 1:
        n[1] = case["lo"]
    return n


def _append_sequences(case):
    """(lengths, first positions) of the runs of new tokens of an append."""
    if case["kind"] == "prompts":
        n = _lengths(case)
        return n, [0] * len(n)
    rng = random.Random("%d %d" % (case["tokens"], case["ctx"]))
    live = case["tokens"] - case["pad"]
    return [1] * live, [rng.randrange(case["ctx"]) for _ in range(live)]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    per = 1 if case.get("cache") == "int8" else 2
    scales = 4 if per == 1 else 0
    if case["op"] == "append":
        n, first = _append_sequences(case)
        live = sum(n)
        t = live + case.get("pad", 0)
        angles = len({f + i for f, m in zip(first, n) for i in range(m)})
        out_k = hkv * d * 2 if case["kind"] == "prompts" else 0
        return {"bytes": t * ((hq + hkv) * d * 2 + hq * d * 2 + out_k + 12) + live * hkv * (d * 2 + 2 * (d * per + scales))
                + angles * case["rot"] * 4, "flops": t * (hq + hkv) * d * 8}
    n = _lengths(case)
    if case["op"] == "prompt":
        return {"bytes": sum(n) * (2 * hq + 2 * hkv) * d * 2, "flops": 4 * d * hq * sum(m * (m + 1) // 2 for m in n)}
    return {"bytes": sum(n) * hkv * 2 * (d * per + scales) + 2 * len(n) * hq * d * 2 + sum(-(-m // case["page"]) for m in n) * 4,
            "flops": 4 * d * hq * sum(n)}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _keys(gen, t, h, d):
    """Keys with a few channels that are larger than the others, as projections give them."""
    k = torch.randn(t, h, d, generator=gen, device="cuda")
    k[:, :, 3::37] *= 4.0
    return k.to(torch.bfloat16)


def _pages(case, need, gen):
    """A cache's block table: `need` pages for each sequence, in an order of chance."""
    most, total = max(need), sum(need)
    table = torch.zeros(len(need), most, dtype=torch.int32)
    perm = torch.randperm(total + 3, generator=gen, device="cuda").cpu().to(torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table.cuda(), total + 3


def _empty_cache(case, pages, gen):
    shape = (pages, case["hkv"], case["page"], case["d"])
    if case["cache"] == "int8":
        scale = [torch.rand(shape[:3], generator=gen, device="cuda") * 0.02 + 0.01 for _ in range(2)]
        codes = [(torch.randn(shape, generator=gen, device="cuda") * 40).round_().clamp_(-127, 127).to(torch.int8)
                 for _ in range(2)]
        return dict(k_cache=codes[0], v_cache=codes[1], k_scale=scale[0], v_scale=scale[1])
    return dict(k_cache=_normal(gen, *shape), v_cache=_normal(gen, *shape), k_scale=None, v_scale=None)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = dict(case=case, op=case["op"], scale=d ** -0.5)
    if case["op"] == "append":
        n, first = _append_sequences(case)
        pad = case.get("pad", 0)
        t = sum(n) + pad
        # the fused projection's output: q, k and v are column views of it
        fused = torch.cat([_normal(gen, t, hq * d), _keys(gen, t, hkv, d).reshape(t, -1), _normal(gen, t, hkv * d)], 1)
        q, k, v = fused.split([hq * d, hkv * d, hkv * d], 1)
        s |= dict(q=q.view(t, hq, d), k=k.view(t, hkv, d), v=v.view(t, hkv, d))
        page = case["page"]
        if case["kind"] == "prompts":
            table, pages = _pages(case, [-(-m // page) for m in n], gen)
            run = torch.cat([torch.arange(m) for m in n])
            seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
            pos = run
            slots = table.cpu()[seq, run // page].long() * page + run % page
        else:  # the page that each sequence is filling
            pages = len(n) + 3
            pos = torch.tensor(first + [0] * pad)
            mine = torch.randperm(pages, generator=gen, device="cuda")[:len(n)].cpu()
            slots = torch.cat([mine * page + torch.tensor(first) % page, torch.full((pad,), -1)]).long()
        s |= _empty_cache(case, pages, gen)
        far = int(pos.max()) + 1
        inv = THETA ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * inv
        s |= dict(rope=torch.cat([angle.cos(), angle.sin()], 1).float(), positions=pos.int().cuda(), slots=slots.cuda(),
                  q_norm=None, k_norm=None)
        if case["norm"]:
            s |= dict(q_norm=_normal(gen, d, std=0.1, dtype=torch.float32), k_norm=_normal(gen, d, std=0.1, dtype=torch.float32))
        s["k_out"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda") if case["kind"] == "prompts" else None
        return s
    n = _lengths(case)
    if case["op"] == "prompt":
        t = sum(n)
        cu = torch.tensor([0] + n).cumsum(0).int().cuda()
        v = _normal(gen, t, hkv * d).view(t, hkv, d)
        return s | dict(q=_normal(gen, t, hq, d), k=_keys(gen, t, hkv, d), v=v, cu=cu)
    table, pages = _pages(case, [-(-m // case["page"]) for m in n], gen)
    s |= _empty_cache(case, pages, gen)
    return s | dict(q=_normal(gen, len(n), hq, d), table=table, lens=torch.tensor(n, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ plain forms
def _norm_rotate(x, weight, rope, positions):
    """RMSNorm with (1 + w) per head where there is a weight; then the first R dimensions turn, each with the one R / 2 above it."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (1 + weight)
    half = rope.shape[1] // 2
    turn = rope[positions.long()][:, None]
    cos, sin = turn[..., :half], turn[..., half:]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1)


def _store(cache, scale, x, page, off):
    """Writes the rows x [tokens, heads, d], given in 32 bits, at their places of a cache."""
    if scale is None:
        cache[page, :, off] = x.to(cache.dtype)
        return
    s = x.abs().amax(-1) / 127
    cache[page, :, off] = torch.where(s[..., None] > 0, x / s[..., None], 0).round().clamp(-127, 127).to(torch.int8)
    scale[page, :, off] = s


def _values(cache, scale):
    """What a cache stands for: int8 codes times their scales, as the bf16 values that a cache of that type would hold."""
    return cache if scale is None else (cache * scale[..., None]).to(torch.bfloat16)


def _plain_append(s):
    q = _norm_rotate(s["q"], s["q_norm"], s["rope"], s["positions"])
    k = _norm_rotate(s["k"], s["k_norm"], s["rope"], s["positions"])
    page = s["k_cache"].shape[2]
    live = s["slots"] >= 0
    at = s["slots"][live]
    _store(s["k_cache"], s["k_scale"], k[live], at // page, at % page)
    _store(s["v_cache"], s["v_scale"], s["v"][live].float(), at // page, at % page)
    return q.to(torch.bfloat16), k.to(torch.bfloat16) if s["k_out"] is not None else None


def _softmax_(x):
    """exp(x - max) over the last dimension, over its sum; in place."""
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    return x


def _plain_prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"]
    t, hq, d = q.shape
    hkv = k.shape[1]
    at = torch.arange(t, device=q.device)
    seq = torch.bucketize(at, cu[1:].long(), right=True)
    seen = (seq[:, None] == seq) & (at[:, None] >= at)
    q = q.float().view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    p = (q @ k.float().permute(1, 2, 0)).view(hq, t, t)
    p *= s["scale"]
    _softmax_(p.masked_fill_(~seen, -math.inf))
    o = p.view(hkv, -1, t) @ v.float().transpose(0, 1)
    return o.view(hq, t, d).transpose(0, 1).to(torch.bfloat16).contiguous()


def _plain_decode(s):
    q, table, lens = s["q"], s["table"].long(), s["lens"]
    b, hq, d = q.shape
    hkv, page = s["k_cache"].shape[1:3]

    def gather(cache, scale):
        x = cache[table].float() if scale is None else cache[table] * scale[table][..., None]
        return x.transpose(1, 2).reshape(b, hkv, -1, d)

    q = q.float().view(b, hkv, hq // hkv, d)
    p = q @ gather(s["k_cache"], s["k_scale"]).transpose(2, 3)
    p *= s["scale"]
    seen = torch.arange(p.shape[-1], device=q.device) < lens[:, None]
    _softmax_(p.masked_fill_(~seen[:, None, None], -math.inf))
    return (p @ gather(s["v_cache"], s["v_scale"])).view(b, hq, d).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import w8a8_int8_quantized_rmsnorm_b200 as cr
        if s["op"] == "prompt":
            return cr.convrot_attention_prompt(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"])
        if s["op"] == "decode":
            return cr.convrot_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                               k_scale=s["k_scale"], v_scale=s["v_scale"], scale=s["scale"])
        q, k = cr.convrot_rope_append(s["q"], s["k"], s["v"], s["rope"], s["positions"], s["slots"], s["k_cache"],
                                      s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"], q_norm=s["q_norm"],
                                      k_norm=s["k_norm"], eps=EPS, k_out=s["k_out"])
    else:
        if s["op"] == "prompt":
            return _plain_prompt(s)
        if s["op"] == "decode":
            return _plain_decode(s)
        q, k = _plain_append(s)
    return dict(q=q, k=k, k_cache=_values(s["k_cache"], s["k_scale"]), v_cache=_values(s["v_cache"], s["v_scale"]))


# ------------------------------------------------------------------ 64 bits
def _exact_append(s):
    case, page = s["case"], s["case"]["page"]
    half = case["rot"] // 2
    turn = s["rope"].double()[s["positions"].long()]
    factor = torch.complex(turn[:, :half], turn[:, half:])[:, None]

    def rotated(x, w):
        x = x.double().clone()
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * (w.double() + 1)
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * factor
        x[..., :half], x[..., half:2 * half] = z.real, z.imag
        return x

    def written(cache, scale, x):
        if scale is not None:
            cache = cache.double() * scale.double().unsqueeze(-1)
            s_new = x.abs().max(-1, keepdim=True).values / 127
            x = s_new * torch.round(x / s_new.clamp_min(1e-300))
        out = cache.double().transpose(1, 2).flatten(0, 1)
        live = s["slots"] >= 0
        out[s["slots"][live]] = x[live]
        return out.view(-1, page, case["hkv"], case["d"]).transpose(1, 2)

    q, k = rotated(s["q"], s["q_norm"]), rotated(s["k"], s["k_norm"])
    return dict(q=q, k=k if s["k_out"] is not None else None, k_cache=written(s["k_cache"], s["k_scale"], k),
                v_cache=written(s["v_cache"], s["v_scale"], s["v"].double()))


def _exact_prompt(s):
    q, k, v = (s[x].double() for x in "qkv")
    cu, group = s["cu"].tolist(), q.shape[1] // k.shape[1]
    out = torch.empty_like(q)
    for a, b in zip(cu, cu[1:]):
        future = torch.ones(b - a, b - a, dtype=torch.bool, device=q.device).triu(1)
        for h in range(q.shape[1]):
            x = torch.einsum("id,jd->ij", q[a:b, h], k[a:b, h // group]) * s["scale"]
            out[a:b, h] = torch.softmax(x.masked_fill(future, -math.inf), 1) @ v[a:b, h // group]
    return out


def _exact_decode(s):
    q, out = s["q"].double(), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    group = q.shape[1] // s["k_cache"].shape[1]
    for i, n in enumerate(s["lens"].tolist()):
        mine = s["table"][i].long()[:-(-n // s["case"]["page"])]

        def rows(cache, scale):
            x = cache[mine].double()
            if scale is not None:
                x *= scale[mine].double().unsqueeze(-1)
            return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n].repeat_interleave(group, 0)

        x = torch.einsum("hd,hjd->hj", q[i], rows(s["k_cache"], s["k_scale"])) * s["scale"]
        out[i] = torch.einsum("hj,hjd->hd", torch.softmax(x, 1), rows(s["v_cache"], s["v_scale"]))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "prompt": _exact_prompt, "decode": _exact_decode}[case["op"]](s)
