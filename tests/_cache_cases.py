"""Inputs and bounds of the 8-bit cache tests."""
import numpy as np
import torch

from oracle import cache as oc

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FILL = 0x7F  # e4m3's NaN: what no call may let into a result


def pages_of(lengths, page, seed, spare=2, width=None):
    """A table [B, width] of distinct pages in a random order (-1 behind each sequence's) and num_pages."""
    need = [-(-n // page) for n in lengths]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lengths), width or max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def empty_cache(num_pages, Hkv, page, d):
    """Codes that are NaN and scales that are NaN: a call that uses one shows it."""
    shape = (num_pages, Hkv, page, d)
    return {"k": np.full(shape, FILL, np.uint8), "v": np.full(shape, FILL, np.uint8),
            "k_scale": np.full(shape[:2], np.nan), "v_scale": np.full(shape[:2], np.nan)}


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def filled_cache(lengths, Hkv, page, d, seed, k_size=1.0, v_size=1.0, width=None):
    """A cache that holds lengths[b] tokens of each sequence, rows behind them NaN, and its table.
    Blocks differ in size by powers of two, so scales do."""
    table, num = pages_of(lengths, page, seed, width=width)
    cache = empty_cache(num, Hkv, page, d)
    longest = max(max(lengths), 1)
    rng = np.random.default_rng(seed + 1)
    for name, size in (("k", k_size), ("v", v_size)):
        for b, n in enumerate(lengths):
            for p in range(-(-n // page)):
                rows = min(page, n - p * page)
                x = rng.standard_normal((Hkv, rows, d)) * size * 2.0 ** rng.integers(-2, 2, (Hkv, 1, 1))
                for h in range(Hkv):
                    e = oc.exponent(np.abs(x[h]).max())
                    cache[name + "_scale"][table[b, p], h] = 2.0 ** e
                    cache[name][table[b, p], h, :rows] = oc.round_e4m3(x[h] / 2.0 ** e)
    assert longest >= 1
    return cache, table


def to_device(la, cache, dev):
    t = [torch.from_numpy(cache[n].copy()).to(dev).view(torch.float8_e4m3fn) for n in "kv"]
    s = [torch.from_numpy(cache[n + "_scale"]).float().to(dev) for n in "kv"]
    return la.la_cache(*t, *s)


def from_device(cache):
    k, v, ks, vs = cache
    return {"k": k.view(torch.uint8).cpu().numpy(), "v": v.view(torch.uint8).cpu().numpy(),
            "k_scale": ks.double().cpu().numpy(), "v_scale": vs.double().cpu().numpy()}


def same_cache(got, ref):
    for n in ref:
        np.testing.assert_array_equal(got[n], ref[n], err_msg=n)


def ints(v, dev):
    return torch.tensor(list(v), dtype=torch.int32, device=dev)


# Bounds of the attention, from its arithmetic.
#   scores   a dot product of d exact products (q of 11 bits, codes of 4) summed in fp32, and a
#            few factors: off by at most (d + 8) 2^-24 sum |q_c k_c| scale.  The score and
#            the row's maximum enter the exponent, so a weight is off by twice that, plus one
#            fp32 rounding of the exponent's argument, at most 2^-24 of the scores' size
#   weights  2^-16 for the exponential, and rounded to fp16 for the product with V: 2^-11 of
#            each, or for those too small 2^-25 of a weight of 2^7 at least at the maximum: 2^-32
#   o        rounded to its type; sums in fp32: n 2^-24 at most
def attend_bounds(ref, n, d, dtype):
    o, lse, size, dots, top = ref
    score = 2 * (d + 8) * 2.0 ** -24 * dots
    weight = np.expm1(score) + 2.0 ** -16 + n * 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    tiny = float(torch.finfo(dtype).tiny) * 2.0 ** -8   # half a step of the subnormals, or more
    o_tol = (2 * weight[..., None] + 2.0 ** -11) * size + n * 2.0 ** -32 * top[..., None]
    return o_tol * (1 + half) + half * np.abs(o) + tiny, weight + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def assert_attend(got_o, got_lse, ref, n, d, dtype, what=""):
    o_tol, lse_tol = attend_bounds(ref, n, d, dtype)
    g = got_o.double().cpu().numpy()
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    off = np.abs(g - ref[0]) / o_tol
    assert off.max() <= 1, f"{what}: {off.max():.2f} of the bound at {np.unravel_index(off.argmax(), off.shape)}"
    if got_lse is not None:
        g = got_lse.double().cpu().numpy()
        np.testing.assert_array_equal(np.isneginf(g), np.isneginf(ref[1]), err_msg=what)
        fine = np.isfinite(ref[1])
        off = np.abs(g[fine] - ref[1][fine]) / lse_tol[fine]
        assert not off.size or off.max() <= 1, f"{what}: lse {off.max():.2f} of the bound"
