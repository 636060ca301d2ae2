"""Attention whose scores are so large that fp32 holds them to whole numbers only, or to multiples of
2^50: a row is then its best key's value wherever that key is best by more than the scores' rounding."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

from _cache_cases import filled_cache, ints, normal, to_device

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("G,N", [(1, 1), (4, 4), (8, 4), (1, 40), (3, 150)])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("log_scale", [16, 20, 23, 24, 25, 26, 27, 28, 29, 30, 35, 50, 80])
def test_scores_far_beyond_one(la, G, N, d, dtype, log_scale):
    kv = [400, N]
    cache, table = filled_cache(kv, 1, 16, d, 5)
    q = normal(N + log_scale, 2, G, N, d).to(dtype)
    scale = 2.0 ** log_scale * (-1 if log_scale % 2 else 1)
    lse = torch.zeros(q.shape[:3], device=DEV)
    o = la.la_cache_attend(q.to(DEV), to_device(la, cache, DEV), torch.from_numpy(table).to(DEV), ints(kv, DEV),
                           lse=lse, scale=scale)
    assert la.la_device_status() == (0, 0)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    half, sure = torch.finfo(dtype).eps / 2, 0
    for b, n in enumerate(kv):
        k, v = (oc.tokens(cache, x, table[b], 0, 0, n) for x in "kv")
        for h in range(G):
            for i in range(N):
                x = q[b, h, i].double().numpy()
                s = (k[:n - N + i + 1] @ x) * scale
                # a score is off by (d + 8) 2^-24 of its terms, and by three roundings as it goes into the
                # exponent; 40 more: below fp16's weights
                off = (d + 16) * 2.0 ** -24 * (np.abs(k[:len(s)]) @ np.abs(x)).max() * abs(scale)
                best = s.argmax()
                rest = np.delete(s, best).max(initial=-np.inf)
                assert abs(lse[b, h, i] - s[best]) <= off + np.log(len(s))
                if s[best] - rest > 2 * off + 40:
                    sure += 1
                    want = v[best]
                    # the weight's own rounding, and of l: 2^-11 and 2^-15
                    tol = (half + 2.0 ** -11 + 2.0 ** -15) * np.abs(want) + 2.0 ** -32 * np.abs(v).max()
                    tol += float(torch.finfo(dtype).tiny) * 2.0 ** -8
                    assert (np.abs(o[b, h, i] - want) <= tol).all(), (b, h, i)
                else:   # some mean of the values
                    assert np.abs(o[b, h, i]).max() <= np.abs(v[:len(s)]).max() * (1 + 2.0 ** -7)
    assert sure > G * N
