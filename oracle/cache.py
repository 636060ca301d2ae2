"""fp64 oracle of the 8-bit key/value cache: storing tokens, reading them back and
causal softmax attention over them, in plain numpy loops over sequences, heads and
pages.  Independent of the CUDA library; used by the tests only.

A cache is a dict: "k", "v" uint8 codes [num_pages,Hkv,page,d] and "k_scale",
"v_scale" float64 [num_pages,Hkv].
"""
import math

import numpy as np

TOP, LOW = 448.0, -126


def _decode(code):
    s, e, m = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
    return -x if s else x


E4M3 = np.array([_decode(c) for c in range(256)])


def round_e4m3(x):
    """The code of the e4m3 number nearest to each x (|x| <= 448; ties to the even code)."""
    x = np.asarray(x, dtype=np.float64)
    a, grid = np.abs(x), E4M3[:127]
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    take = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return (take + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(amax):
    """Least e >= LOW with amax <= TOP * 2^e."""
    e = LOW
    while amax > math.ldexp(TOP, e):
        e += 1
    return e


def write(cache, table, k, v, start, count):
    """A copy of the cache with tokens start[b] .. start[b] + count[b] - 1 stored."""
    out = {n: a.copy() for n, a in cache.items()}
    page = cache["k"].shape[2]
    for name, x in (("k", k), ("v", v)):
        codes, scales = out[name], out[name + "_scale"]
        for b, (s, n) in enumerate(zip(start, count)):
            for p in range(s // page, -(-(s + n) // page)) if n else ():
                lo, hi = max(s, p * page), min(s + n, (p + 1) * page)
                at = table[b][p]
                for h in range(x.shape[1]):
                    new = np.asarray(x[b, h, lo - s:hi - s], dtype=np.float64)
                    finite = np.isfinite(new)
                    scale = math.ldexp(1.0, exponent(np.max(np.abs(new), where=finite, initial=0.0)))
                    if lo > p * page:
                        old = scales[at, h]
                        scale = max(scale, old)
                        if scale > old:
                            rows = codes[at, h, :lo - p * page]
                            rows[:] = round_e4m3(E4M3[rows] * (old / scale))
                    scales[at, h] = scale
                    new = np.where(np.isnan(new), 0.0, np.clip(new / scale, -TOP, TOP))
                    codes[at, h, lo - p * page:hi - p * page] = round_e4m3(new)
    return out


def tokens(cache, name, pages, h, first, last):
    """Tokens first .. last - 1 of kv head h of the sequence in `pages`, [last - first, d]."""
    page, d = cache[name].shape[2:]
    t = np.arange(first, last)
    at = np.asarray(pages)[t // page] if last > first else np.zeros(0, dtype=np.int64)
    return E4M3[cache[name][at, h, t % page]] * cache[name + "_scale"][at, h][:, None]


def attend(cache, table, q, kv_len, q_len, scale):
    """o, lse and, for bounds on the rounding of both, sum_j p_ij |v_j| / sum_j p_ij, the
    largest sum_c |q_c k_jc| * |scale| of a row and the largest |v| it sees.  Rows at and behind
    q_len[b] are zero."""
    q = np.asarray(q, dtype=np.float64)
    B, Hq, N, d = q.shape
    G = Hq // cache["k"].shape[1]
    o, size = np.zeros_like(q), np.zeros_like(q)
    lse, dots, top = np.zeros(q.shape[:3]), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    for b in range(B):
        for h in range(Hq):
            k = tokens(cache, "k", table[b], h // G, 0, kv_len[b])
            v = tokens(cache, "v", table[b], h // G, 0, kv_len[b])
            for i in range(q_len[b]):
                n = kv_len[b] - q_len[b] + i + 1
                if n <= 0:
                    lse[b, h, i] = -np.inf
                    continue
                s = (k[:n] @ q[b, h, i]) * scale
                m = s.max()
                p = np.exp(s - m)
                o[b, h, i] = p @ v[:n] / p.sum()
                size[b, h, i] = p @ np.abs(v[:n]) / p.sum()
                lse[b, h, i] = m + math.log(p.sum())
                dots[b, h, i] = (np.abs(k[:n]) @ np.abs(q[b, h, i])).max() * abs(scale)
                top[b, h, i] = np.abs(v[:n]).max()
    return o, lse, size, dots, top
