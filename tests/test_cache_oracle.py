"""Pins of the 8-bit cache's oracle, on the CPU: the number format, the scale, growth of a
page's scale, and attention against closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc

from _cache_cases import empty_cache, filled_cache


def test_e4m3_values_are_torchs():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oc.E4M3, ref)


def test_rounding_is_to_nearest_even():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.02,
                        (oc.E4M3[:126] + oc.E4M3[1:127]) / 2, oc.E4M3[:127], [0.0, 2.0 ** -10]])
    ref = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    x = x.astype(np.float32)
    np.testing.assert_array_equal(oc.E4M3[oc.round_e4m3(x)], ref)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (np.nextafter(448.0, 449), 1), (224.0, -1), (1.0, -8),
                                    (1.75, -8), (1.76, -7), (0.0, -126), (3.0e38, 120)])
def test_scale_exponent(amax, e):
    assert oc.exponent(amax) == e
    assert amax <= math.ldexp(448.0, e) and (e == -126 or amax > math.ldexp(448.0, e - 1))


def test_growth_rounds_older_codes_once():
    cache = empty_cache(1, 1, 16, 64)
    k = np.full((1, 1, 1, 64), 1.0)
    c = oc.write(cache, [[0]], k, k, [0], [1])
    assert c["k_scale"][0, 0] == 2.0 ** -8 and oc.E4M3[c["k"][0, 0, 0, 0]] == 256
    c = oc.write(c, [[0]], k * 100, k, [1], [1])
    assert c["k_scale"][0, 0] == 2.0 ** -2 and oc.E4M3[c["k"][0, 0, 0, 0]] == 4
    assert c["v_scale"][0, 0] == 2.0 ** -8
    assert (c["k"][0, 0, 2:] == 0x7F).all()


def test_attention_closed_forms():
    """Equal keys: the mean of the values seen; one token: its value; none: zero."""
    cache, table = filled_cache([20], 2, 16, 64, 3)
    cache["k"][:] = 0
    q = np.ones((1, 4, 3, 64))
    o, lse, *_ = oc.attend(cache, table, q, [20], [3], 0.125)
    v = oc.tokens(cache, "v", table[0], 1, 0, 20)
    np.testing.assert_allclose(o[0, 2, 0], v[:18].mean(0), rtol=1e-12, atol=1e-15)
    np.testing.assert_allclose(lse[0, 0], np.log([18, 19, 20]), rtol=1e-12)
    o, lse, *_ = oc.attend(cache, table, q, [2], [3], 0.125)
    assert (o[0, :, 0] == 0).all() and np.isneginf(lse[0, :, 0]).all()
    np.testing.assert_allclose(o[0, 2, 1], v[0], rtol=1e-14)


def test_split_invariance():
    """Two halves joined by their logarithms are the whole."""
    cache, table = filled_cache([40], 1, 16, 64, 4)
    q = np.random.default_rng(1).standard_normal((1, 1, 1, 64))
    o, lse, *_ = oc.attend(cache, table, q, [40], [1], 0.3)
    o1, l1, *_ = oc.attend(cache, table, q, [16], [1], 0.3)
    rest = table[:, 1:]
    o2, l2, *_ = oc.attend(cache, rest, q, [24], [1], 0.3)
    w1, w2 = np.exp(l1 - lse)[..., None], np.exp(l2 - lse)[..., None]
    np.testing.assert_allclose(o1 * w1 + o2 * w2, o, rtol=1e-10, atol=1e-12)
