"""Attention over pages whose scales differ by many powers of two: early rows of a prompt see
only pages that are small beside those of later rows.

Bounds: those of _cache_cases, and where a page's scale is under 2^-22 of the largest one's, 2^-32 of
that for each value of the page: in o as it is (o is a mean of them), in a score times |q| and the
call's factor."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

from _cache_cases import filled_cache, ints, normal, to_device

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def check(la, cache, table, q, kv, nq, scale, off_k, off_v):
    """off_k, off_v: what a value of a key or a value may be off by beside the usual."""
    B, Hq, N, d = q.shape
    x = q.double().numpy()
    ref, ref_lse, size, dots, top = oc.attend(cache, table, x, kv, nq, scale)
    lse = torch.zeros(B, Hq, N, device=DEV)
    o = torch.zeros_like(q, device=DEV)
    la.la_cache_attend(q.to(DEV), to_device(la, cache, DEV), torch.from_numpy(table).to(DEV), ints(kv, DEV),
                       q_len=ints(nq, DEV), o=o, lse=lse, scale=scale)
    assert la.la_device_status() == (0, 0)
    score = (d + 8) * 2.0 ** -24 * dots + off_k * np.abs(x).sum(-1) * abs(scale)
    weight = np.expm1(2 * score) + 2.0 ** -16 + max(kv) * 2.0 ** -24
    half = torch.finfo(q.dtype).eps / 2
    tol = (2 * weight[..., None] + 2.0 ** -11) * size + max(kv) * 2.0 ** -32 * top[..., None] + off_v
    tol = tol * (1 + half) + half * np.abs(ref) + float(torch.finfo(q.dtype).tiny) * 2.0 ** -8
    off = np.abs(o.double().cpu().numpy() - ref) / tol
    assert off.max() <= 1, f"o {off.max():.3g} of the bound at {np.unravel_index(off.argmax(), off.shape)}"
    fine = np.isfinite(ref_lse)
    off = np.abs(lse.double().cpu().numpy() - ref_lse)[fine] / (weight + 2.0 ** -22 * np.abs(ref_lse))[fine]
    assert off.max() <= 1, f"lse {off.max():.3g} of the bound"


@pytest.mark.parametrize("d,G,page", [(64, 1, 16), (128, 2, 16), (64, 4, 64)])
@pytest.mark.parametrize("log_r", [-14, -16, -20, -22, -25, -28, -30, -33])
def test_small_values_before_large_ones(la, d, G, page, log_r):
    """A prompt's first 64 rows see values 2^log_r beside those of the rows after them."""
    n = 200
    cache, table = filled_cache([n, 40], 1, page, d, 3 - log_r)
    for p in range(64 // page):
        cache["v_scale"][table[0, p]] *= 2.0 ** log_r
    largest = max(cache["v_scale"][t, 0] for t in table[0])
    q = normal(2, 2, G, n, d).bfloat16()
    check(la, cache, table, q, [n, 40], [n, 40], d ** -0.5, 0, 2.0 ** -32 * largest if log_r < -18 else 0)


@pytest.mark.parametrize("d,G,page", [(64, 1, 16), (128, 2, 16), (64, 4, 64)])
@pytest.mark.parametrize("log_r", [-14, -16, -20, -22, -25, -28])
def test_small_keys_before_large_ones(la, d, G, page, log_r):
    """The same of the keys.  The large ones are large where the queries are zero, so that the small ones
    decide everywhere."""
    n = 200
    cache, table = filled_cache([n, 40], 1, page, d, 5 - log_r)
    small = 64 // page
    cache["k"][table[0, :small], :, :, 0] = 0
    for p in range(small, table.shape[1]):
        rows = min(page, n - p * page)
        cache["k"][table[0, p], :, :rows, 1:] = 0
    q = normal(2, 2, G, n, d).bfloat16()
    q[0, :, :, 0] = 0
    for p in range(small):
        cache["k_scale"][table[0, p]] *= 2.0 ** log_r
    cache["k_scale"][table[1, :-(-40 // page)]] *= 2.0 ** log_r
    largest = max(cache["k_scale"][t, 0] for t in table[0])
    # scales differ by 2^4 among pages of a kind
    check(la, cache, table, q, [n, 40], [n, 40], d ** -0.5 * 2.0 ** -log_r,
          2.0 ** -32 * largest if log_r < -18 else 0, 0)


@pytest.mark.parametrize("N", [1, 12, 40])
@pytest.mark.parametrize("name", ["k_scale", "v_scale", "k", "v"])
def test_a_page_that_was_never_written_shows(la, N, name):
    """NaN in a page's scale, or in a code: the rows that see it are NaN, not something finite."""
    cache, table = filled_cache([70, 70], 1, 16, 64, 4)
    bad = cache[name]
    if name in "kv":
        bad[table[0, 1], 0, 3, 5] = 0x7F
    else:
        bad[table[0, 1], 0] = np.nan
    q = normal(2, 2, 2, N, 64).half().to(DEV)
    o = la.la_cache_attend(q, to_device(la, cache, DEV), torch.from_numpy(table).to(DEV), ints([70, 70], DEV))
    seen = o[0].isnan().any(-1)
    assert seen.all() and torch.isfinite(o[1]).all()
    la.la_device_status()
