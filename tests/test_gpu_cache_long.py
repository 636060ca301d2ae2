"""Attention over long caches: what a row's sums keep of a million small weights.  Sequences
of 2^18 tokens and more on a few pages that their tables repeat, so that a distinct page and how
often a row sees it give the result in 64 bits.

Bounds.  Scores and the exponential as in _cache_cases.  The sum of a row's weights: steps
of at most 32 additions from zero, put together with what each addition lost (2^-23 of each
step) and then across lanes, blocks and warps: less than 64 roundings of 2^-24.  A weight enters
the product with V as fp16: off by 2^-11 of itself or, where that is less, by 2^-25 of the 2^7
that stand for the row's largest.  The products' sums cut off: a step of 16 tokens adds 17 numbers,
each cut off at the last place of the sum or below, 2^-23 of it, and a chain has at most 16384
tokens (prompts) or 4096; the chains and parts are then added in fp32, no more than 600 of them.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc

from _cache_cases import filled_cache, ints, normal, to_device

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
PAGE = 128


def cut_off(rows):
    return (16384 if rows > 32 else 4096) / 16 * 17 * 2.0 ** -23 + 600 * 2.0 ** -24


def attend_pages(cache, pages, q, kv, scale, chain):
    """o, lse and their bounds for rows q [N,d], the last N of kv tokens in the full pages `pages`
    of one kv head; `chain`: what the products' sums may lose."""
    k, v = (oc.E4M3[cache[n][:, 0]] * cache[n + "_scale"][:, 0, None, None] for n in "kv")  # [P,page,d]
    # a weight times its page's scale is what is rounded
    least = 2.0 ** -32 * cache["v_scale"][:, 0].max() / cache["v_scale"][:, 0, None]
    N, d = q.shape
    o, lse, o_tol, lse_tol = np.zeros((N, d)), np.zeros(N), np.zeros((N, d)), np.zeros(N)
    for i in range(N):
        n = kv - N + i + 1
        times = np.zeros(k.shape[:2])                      # how often the row sees each token
        for page, c in zip(*np.unique(pages[:n // PAGE], return_counts=True)):
            times[page] += c
        if n % PAGE:
            times[pages[n // PAGE], :n % PAGE] += 1
        s = (k @ q[i]) * scale
        m = s[times > 0].max()
        p = np.where(times > 0, np.exp(np.minimum(s - m, 0)), 0)
        l = (times * p).sum()
        o[i] = np.einsum("pt,ptd->d", times * p, v) / l
        lse[i] = m + math.log(l)
        dots = (np.abs(k) @ np.abs(q[i]))[times > 0].max() * abs(scale)
        weight = np.expm1(2 * (d + 8) * 2.0 ** -24 * dots) + 2.0 ** -16 + 64 * 2.0 ** -24
        off = times * ((2 * weight + chain) * p + np.maximum(2.0 ** -11 * p, least))
        o_tol[i] = np.einsum("pt,ptd->d", off, np.abs(v)) / l
        lse_tol[i] = weight + 2.0 ** -22 * abs(lse[i])
    return o, lse, o_tol, lse_tol


def check(la, cache, table, q, scale, kv=None):
    """Sequences whose tables repeat a few pages; q [G,N,d] the same for every sequence."""
    B, n = table.shape
    kv = kv or n * PAGE
    G, N, d = q.shape
    x = q[None].expand(B, -1, -1, -1).contiguous().to(DEV)
    lse = torch.zeros(x.shape[:3], device=DEV)
    o = la.la_cache_attend(x, to_device(la, cache, DEV), torch.from_numpy(table).to(DEV), ints([kv] * B, DEV),
                           lse=lse, scale=scale)
    assert la.la_device_status() == (0, 0)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    half = torch.finfo(q.dtype).eps / 2
    for g in range(G):
        want, want_lse, o_tol, lse_tol = attend_pages(cache, table[0], q[g].double().numpy(), kv, scale,
                                                      cut_off(G * N))
        off = np.abs(lse[:, g] - want_lse) / lse_tol
        assert off.max() <= 1, f"lse {off.max():.2f} of the bound"
        off = np.abs(o[:, g] - want) / (o_tol * (1 + half) + half * np.abs(want))
        assert off.max() <= 1, f"o {off.max():.2f} of the bound, {np.abs(o[:, g] - want).max():.2e}"


def some_pages(count, d, seed):
    """A cache of `count` full pages."""
    cache, table = filled_cache([count * PAGE], 1, PAGE, d, seed)
    return {n: a[table[0]] for n, a in cache.items()}


SHAPES = [(1, 1, 64), (4, 4, 64), (4, 8, 128), (1, 40, 64), (1, 40, 128), (2, 200, 64)]   # G, N, d


@pytest.mark.parametrize("G,N,d", SHAPES)
@pytest.mark.parametrize("log_n,gap", [(20, 20.3), (18, 24.5), (20, 24.5), (20, 0.585)])
def test_a_large_weight_and_a_million_small_ones(la, G, N, d, log_n, gap):
    """One key 2^gap above all others, every value 1: o is 1 and lse tells the others' share.  More
    sequences than blocks, so that each sequence is one block's."""
    B = 300 if G * N <= 32 else 160
    cache = {n: np.zeros((2, 1, PAGE, d), np.uint8) for n in "kv"}
    cache |= {n + "_scale": np.ones((2, 1)) for n in "kv"}
    cache["k"][0, 0, 0] = oc.round_e4m3(np.ones(d))
    cache["v"][:] = oc.round_e4m3(1.0)
    table = np.ones((B, 2 ** log_n // PAGE), dtype=np.int32)
    table[:, 0] = 0
    check(la, cache, table, torch.ones(G, N, d).half(), gap * math.log(2) / d)


@pytest.mark.parametrize("G,N,d", SHAPES)
@pytest.mark.parametrize("B,log_n", [(1, 23), (3, 20)])
def test_long_sequences_split_over_the_gpu(la, G, N, d, B, log_n):
    """Chains that end inside a block's share, of units cut between blocks and of whole ones; a length
    that ends inside a page."""
    cache = some_pages(5, d, G + N)
    table = np.random.default_rng(N).integers(0, 5, (1, 2 ** log_n // PAGE)).astype(np.int32).repeat(B, 0)
    check(la, cache, table, (normal(N, G, N, d) * 1.5).half(), d ** -0.5, kv=2 ** log_n - 77)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_maximum_that_grows_from_chain_to_chain(la, dtype):
    """Scores that rise by 2^10 and more along the sequence, so that the sums put by are relative to
    smaller maxima than those that follow, and values whose scales grow too."""
    d, parts = 64, 6
    cache = some_pages(parts, d, 3)
    per = 300                      # pages of a kind in a row: more than two chains of prompts, nine of tokens
    table = np.repeat(np.arange(parts), per).astype(np.int32)[None].repeat(160, 0)
    for p in range(parts):
        cache["v_scale"][p] *= 2.0 ** (2 * p)
        cache["k"][p, 0, :, 0] = oc.round_e4m3(np.full(PAGE, p / 8) / cache["k_scale"][p, 0])
    for G, N in ((1, 1), (4, 8), (1, 64)):
        q = normal(N, G, N, d)
        q[..., 0] = 400.0          # 400 / 8 * d ** -0.5: 2^9 from each kind to the next
        check(la, cache, table, q.to(dtype), d ** -0.5)
