"""CPU reference of the attention operators in numpy float64.

Test infrastructure: position rotation and per-head norm, the rows a paged
cache holds, and softmax attention over an explicit set of visible keys.  It
shares no code with the CUDA path.
"""
import numpy as np

U = 2.0 ** -24      # unit roundoff of fp32
BF16 = 2.0 ** -8    # half a step of bfloat16, relative to the value


def rope_table(rows, dim, theta=1e4):
    """fp32 [rows, dim]: cosines, then sines, of position * theta^(-2i / dim)."""
    angle = np.arange(rows)[:, None] * theta ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def norm_rotate(x, weight, table, positions, eps):
    """x [tokens, heads, D] -> (y, E): the normed and rotated rows, and a bound on
    the error that the same arithmetic in fp32 may make in each element.

    fp32 roundings: the sum of D squares goes through at most D / 8 + 5 adds
    and the root halves its error, then the root, the quotient, three factors
    and the rotation's two roundings, each relative to |a| + |b| at most:
    D / 16 + 12 <= 20 unit roundoffs for D <= 128.
    """
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 + np.asarray(weight, np.float64))
    half = table.shape[1] // 2
    t = np.asarray(table, np.float64)[positions]
    c, s = t[:, None, :half], t[:, None, half:]
    a, b = x[..., :half], x[..., half:2 * half]
    y = np.concatenate([a * c - b * s, a * s + b * c, x[..., 2 * half:]], -1)
    size = np.abs(a) + np.abs(b)
    return y, 20 * U * np.concatenate([size, size, np.abs(x[..., 2 * half:])], -1)


def attention(q, k, v, scale, visible, v_scale=None):
    """One head's rows: q [n, D], k, v [m, D], visible bool [n, m] ->
    (o [n, D], tol [n, D]).

    tol bounds what a kernel may be off that holds scores, sums and outputs in
    fp32 and rounds the probabilities and the result to bf16 once each:
    * a score's dot product of D terms: 2 D unit roundoffs (twice, for a
      matrix unit that does not round to nearest) of scale * sum |q k|, which
      moves a probability by as much relative to itself, in the numerator and
      in the sum;
    * exp2: 2^-12 relative; the probability's rounding: 2^-8;
    * sums of m terms in fp32: m unit roundoffs;
    * the result's rounding: 2^-8 of the result;
    * with v_scale [m] (int8 caches, v = code * scale): each query element is
      off by half a step of a 16-bit grid, max|q| / 32512 / 2, which moves a
      score by scale * sum |k| times that; each probability times its scale is
      off by half a step of such a grid of the largest among 32 neighbours,
      instead of half a step of bf16, which multiplies its key's |code|.
    """
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, d = q.shape
    m = k.shape[0]
    o, tol = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    for i in range(n):
        see = np.flatnonzero(visible[i])
        if not len(see):
            continue
        s = (k[see] @ q[i]) * scale
        p = np.exp(s - s.max())
        p /= p.sum()
        o[i] = p @ v[see]
        ds = 2 * d * U * scale * (np.abs(k[see]) @ np.abs(q[i])).max()
        grid = 0.0
        if v_scale is not None:
            ds += scale * np.abs(q[i]).max() / 65024 * np.abs(k[see]).sum(1).max()
            w = p * v_scale[see]
            code = np.abs(v[see]) / np.where(v_scale[see] > 0, v_scale[see], 1)[:, None]
            for a in range(0, len(see), 32):
                grid = grid + w[a:a + 32].max() / 65024 * code[a:a + 32].sum(0)
        rel = (BF16 if v_scale is None else 0.0) + 2.0 ** -12 + 2 * ds + m * U
        tol[i] = (1 + BF16) * (rel * (p @ np.abs(v[see])) + grid) + BF16 * np.abs(o[i])
    return o, tol


def packed_attention(q, k, v, cu_q, cu_k, scale, causal):
    """q [T, Hq, D], k, v [Tk, Hkv, D] -> (o, tol), rows of no sequence NaN."""
    o, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    group = q.shape[1] // k.shape[1]
    for a, b, c, e in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        lq, lk = b - a, e - c
        see = np.ones((lq, lk), bool)
        if causal:
            see = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq
        for h in range(q.shape[1]):
            o[a:b, h], tol[a:b, h] = attention(q[a:b, h], k[c:e, h // group], v[c:e, h // group], scale, see)
    return o, tol


def cache_rows(cache, scale, table, n):
    """The first n rows [n, heads, D] of a sequence whose pages are `table`."""
    page = cache.shape[2]
    at = np.arange(n)
    rows = np.asarray(cache, np.float64)[np.asarray(table)[at // page], :, at % page]
    if scale is not None:
        rows = rows * np.asarray(scale, np.float64)[np.asarray(table)[at // page], :, at % page][..., None]
    return rows


def paged_attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale):
    """One row per sequence: q [B, Hq, D] -> (o, tol)."""
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    group = q.shape[1] // k_cache.shape[1]
    page = k_cache.shape[2]
    for b, n in enumerate(lens):
        at = np.arange(n)
        s = None if v_scale is None else np.asarray(v_scale, np.float64)[np.asarray(table[b])[at // page], :, at % page]
        k = cache_rows(k_cache, k_scale, table[b], n)
        v = cache_rows(v_cache, v_scale, table[b], n)
        for h in range(q.shape[1]):
            o[b, h], tol[b, h] = (x[0] for x in attention(q[b, h][None], k[:, h // group], v[:, h // group], scale,
                                                          np.ones((1, n), bool), None if s is None else s[:, h // group]))
    return o, tol
