"""The 8-bit key/value cache on the GPU against the fp64 oracle: storing (bit for bit),
reading back (bit for bit), attention of single tokens, a few tokens and prompts."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

from _cache_cases import (FILL, TYPES, assert_attend, attend_bounds, empty_cache, filled_cache,
                          from_device, ints, normal, pages_of, same_cache, to_device)

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def clean(la, flags=0):
    assert la.la_device_status()[1] == flags


# ------------------------------------------------------------------ storing
def write_both(la, cache, table, k, v, start, count, N=None):
    ref = oc.write(cache, table, k.double().numpy(), v.double().numpy(), start, count)
    dev = to_device(la, cache, DEV)
    la.la_cache_write(k.to(DEV), v.to(DEV), dev, torch.from_numpy(table).to(DEV), ints(start, DEV),
                      count=ints(count, DEV))
    same_cache(from_device(dev), ref)
    return ref, dev


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("N,start,count", [
    (1, [0, 5, 15, 16, 127], [1, 1, 1, 0, 1]),
    (3, [0, 14, 15, 126, 31], [3, 2, 3, 3, 1]),
    (4, [13, 0, 60, 62, 64], [4, 4, 4, 4, 0]),
    (5, [13, 0, 60, 62, 64], [5, 4, 5, 5, 0]),
    (200, [0, 1, 64, 127, 300], [200, 199, 17, 129, 1]),
])
def test_write_is_the_oracles(la, dtype, page, d, N, start, count):
    Hkv = 3
    cache, table = filled_cache([s + n for s, n in zip(start, count)], Hkv, page, d, N + page)
    # sizes that grow the scale of some pages and not of others
    size = torch.exp2(normal(7, 5, Hkv, N, 1) * 2)
    k, v = (normal(N + d + i, 5, Hkv, N, d) * size for i in range(2))
    write_both(la, cache, table, k.to(TYPES[dtype]), v.to(TYPES[dtype]), start, count)
    clean(la)


def test_write_token_by_token_is_one_sequence_of_writes(la):
    """Forty tokens one at a time, each page's scale growing as it must."""
    B, Hkv, d, page, n = 2, 2, 64, 16, 40
    table, num = pages_of([n] * B, page, 1)
    ref = empty_cache(num, Hkv, page, d)
    dev = to_device(la, ref, DEV)
    k, v = (normal(i, B, Hkv, n, d) * torch.exp2(3 * normal(9, B, Hkv, n, 1)) for i in range(2))
    k, v = k.bfloat16(), v.bfloat16()
    start = torch.zeros(B, dtype=torch.int32, device=DEV)
    for t in range(n):
        kt, vt = k[:, :, t:t + 1].contiguous(), v[:, :, t:t + 1].contiguous()
        ref = oc.write(ref, table, kt.double().numpy(), vt.double().numpy(), [t] * B, [1] * B)
        la.la_cache_write(kt.to(DEV), vt.to(DEV), dev, torch.from_numpy(table).to(DEV), start)
        start += 1
    same_cache(from_device(dev), ref)


@pytest.mark.parametrize("N", [2, 40])
def test_write_of_zeros_extremes_and_nonfinite(la, N):
    B, Hkv, d, page = 4, 1, 64, 16
    table, num = pages_of([N] * B, page, 2)
    k = normal(1, B, Hkv, N, d)
    k[0] = 0
    k[1] *= 1e38 / 4
    k[2] *= 1e-38
    v = normal(2, B, Hkv, N, d)
    ref, _ = write_both(la, empty_cache(num, Hkv, page, d), table, k, v, [0] * B, [N] * B)
    assert ref["k_scale"][table[0, 0], 0] == 2.0 ** -126
    clean(la)
    v[0, 0, 0, 0], v[1, 0, 1, 5], v[2, 0, N - 1, 63] = float("nan"), float("inf"), -float("inf")
    v[3, 0] = float("nan")
    write_both(la, empty_cache(num, Hkv, page, d), table, k, v, [0] * B, [N] * B)
    assert la.la_device_status() == (0, 4)
    clean(la)


@pytest.mark.parametrize("N", [1, 20])
def test_write_and_read_leave_bad_lengths_and_pages_out(la, N):
    B, Hkv, d, page = 6, 2, 64, 16
    table, num = pages_of([64] * B, page, 3)
    cache = empty_cache(num, Hkv, page, d)
    k = normal(5, B, Hkv, N, d).half()
    start, count = [0, -1, 64, 0, 64 - N + 1, 3], [N, N, 1, N + 1, N, 0]
    good = [N, 0, 0, 0, 0, 0]
    ref = oc.write(cache, table, k.double().numpy(), k.double().numpy(), [0] * B, good)
    dev = to_device(la, cache, DEV)
    t = torch.from_numpy(table).to(DEV)
    args = (k.to(DEV), k.to(DEV), dev, t, ints(start, DEV))
    la.la_cache_write(*args, count=ints(count, DEV))
    same_cache(from_device(dev), ref)
    assert la.la_device_status() == (0, 2)
    out = [torch.full_like(k, 7, device=DEV) for _ in "kv"]
    la.la_cache_read(dev, t, ints(start, DEV), *out, count=ints(count, DEV))
    assert (out[0][1:] == 7).all() and (out[0][0] != 7).any()
    assert la.la_device_status() == (0, 2)
    # a start out of range does not matter to a sequence without tokens
    la.la_cache_write(*args[:4], ints([-5] * B, DEV), count=ints([0] * B, DEV))
    clean(la)
    # pages out of range: not written, read as zeros
    bad = table.copy()
    bad[0, 0], bad[1, 0] = num, -1
    dev = to_device(la, cache, DEV)
    la.la_cache_write(k.to(DEV), k.to(DEV), dev, torch.from_numpy(bad).to(DEV), ints([0] * B, DEV))
    skip = oc.write(cache, table, k.double().numpy(), k.double().numpy(), [0, 0, 0, 0, 0, 0],
                    [0, 0, N, N, N, N])
    if N > page:   # their second pages are good
        for b in (0, 1):
            s, n = [0] * B, [0] * B
            s[b], n[b] = page, N - page
            part = np.zeros(k.shape)
            part[:, :, :N - page] = k.double().numpy()[:, :, page:]
            skip = oc.write(skip, table, part, part, s, n)
    same_cache(from_device(dev), skip)
    assert la.la_device_status() == (0, 2)
    la.la_cache_read(dev, torch.from_numpy(bad).to(DEV), ints([0] * B, DEV), *out)
    assert (out[0][:2, :, :page] == 0).all() and torch.isfinite(out[0]).all()
    assert la.la_device_status() == (0, 2)


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("page,d", [(16, 128), (32, 64), (64, 64), (128, 128)])
def test_read_is_the_oracles(la, dtype, page, d):
    Hkv, N = 3, 150
    start, count = [0, 1, 15, 16, 200], [150, 149, 64, 0, 1]
    cache, table = filled_cache([s + n for s, n in zip(start, count)], Hkv, page, d, 11 + page)
    dev = to_device(la, cache, DEV)
    out = [torch.full((5, Hkv, N, d), -3.0, dtype=TYPES[dtype], device=DEV) for _ in "kv"]
    got = la.la_cache_read(dev, torch.from_numpy(table).to(DEV), ints(start, DEV), *out,
                           count=ints(count, DEV))
    assert got[0] is out[0] and got[1] is out[1]
    for name, x in zip("kv", out):
        ref = torch.full((5, Hkv, N, d), -3.0, dtype=torch.float64)
        for b in range(5):
            for h in range(Hkv):
                ref[b, h, :count[b]] = torch.from_numpy(
                    oc.tokens(cache, name, table[b], h, start[b], start[b] + count[b]))
        assert torch.equal(x.cpu(), ref.to(TYPES[dtype])), name
    clean(la)


# ------------------------------------------------------------------ attention
def attend_both(la, cache, table, q, kv_len, q_len, scale=None, lse=True, workspace=None, what=""):
    B, Hq, N, d = q.shape
    ref = oc.attend(cache, table, q.double().numpy(), kv_len, q_len,
                    d ** -0.5 if scale is None else scale)
    dev = to_device(la, cache, DEV)
    o = torch.full_like(q, 5.0, device=DEV)
    e = torch.full(q.shape[:3], 5.0, device=DEV) if lse else None
    got = la.la_cache_attend(q.to(DEV), dev, torch.from_numpy(table).to(DEV), ints(kv_len, DEV),
                             q_len=ints(q_len, DEV), o=o, lse=e, scale=scale, workspace=workspace)
    assert got is o
    for b in range(B):     # rows behind the last query: as they were
        assert (o[b, :, q_len[b]:] == 5).all(), what
        assert not lse or (e[b, :, q_len[b]:] == 5).all(), what
        o[b, :, q_len[b]:] = 0
        if lse:
            e[b, :, q_len[b]:] = 0
    assert_attend(o, e, ref, max(max(kv_len), 1), d, q.dtype, what)
    clean(la)
    return o, e


SHAPES = [
    # G, d, page, dtype
    (1, 128, 64, "bf16"), (4, 128, 16, "fp16"), (3, 64, 32, "bf16"), (8, 64, 128, "fp16"),
    (16, 128, 128, "bf16"), (6, 64, 16, "fp16"), (32, 128, 32, "bf16"), (2, 64, 64, "bf16"),
]


@pytest.mark.parametrize("G,d,page,dtype", SHAPES)
@pytest.mark.parametrize("N", [1, 2, 5])
def test_tokens(la, G, d, page, dtype, N):
    """Decode: one and a few tokens, sequences from none to several hundred tokens."""
    Hkv = 2
    kv = [N, 1, 15, 16, 17, 64, 65, 129, 700, 0]
    nq = [min(N, 1 + b % N) for b in range(len(kv))]
    cache, table = filled_cache(kv, Hkv, page, d, G + d + page + N)
    q = normal(N + G, len(kv), Hkv * G, N, d).to(TYPES[dtype])
    attend_both(la, cache, table, q, kv, nq, what=f"{G} {d} {page} {dtype} {N}")


@pytest.mark.parametrize("G,N", [(1, 7), (2, 4), (8, 1), (9, 1), (3, 3), (1, 16), (17, 1), (1, 32), (1, 33)])
@pytest.mark.parametrize("d", [64, 128])
def test_numbers_of_rows(la, G, N, d):
    """Around 8, 16 and 32 rows, over tables that leave units whole and that do not; one row is NaN and
    changes no other."""
    kv, nq = [N + 140, N, 3, 610], [N, N, min(N, 3), max(1, N - 1)]
    cache, table = filled_cache(kv, 2, 32, d, G + N)
    wide = np.full((4, 300), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    q = normal(N, 4, 2 * G, N, d).half()
    lost = q.clone()
    lost[0, G, 0, d // 2] = float("nan")
    scale = -0.3 if d == 64 else d ** -0.5
    ref = oc.attend(cache, table, q.double().numpy(), kv, nq, scale)
    for t in (table, wide):
        attend_both(la, cache, t, q, kv, nq, scale=scale)
        got = torch.zeros_like(q, device=DEV)
        la.la_cache_attend(lost.to(DEV), to_device(la, cache, DEV), torch.from_numpy(t).to(DEV), ints(kv, DEV),
                           q_len=ints(nq, DEV), o=got, scale=scale)
        assert got[0, G, 0].isnan().all()
        got[0, G, 0] = torch.from_numpy(ref[0][0, G, 0]).half()
        assert_attend(got, None, ref, max(kv), d, q.dtype)


@pytest.mark.parametrize("G,d,page,dtype", SHAPES)
@pytest.mark.parametrize("N,past", [(40, [0, 3, 100, 129]), (130, [0, 1, 64, 250]), (300, [0, 20])])
def test_prompts(la, G, d, page, dtype, N, past):
    Hkv = 1 if G > 4 else 2
    nq = [N, N - 1, 1, N // 2][:len(past)]
    kv = [a + n for a, n in zip(past, nq)]
    cache, table = filled_cache(kv, Hkv, page, d, G + N)
    q = normal(N + G, len(kv), Hkv * G, N, d).to(TYPES[dtype])
    attend_both(la, cache, table, q, kv, nq, what=f"{G} {d} {page} {dtype} {N}")


@pytest.mark.parametrize("N", [1, 4, 50])
def test_rows_that_see_nothing_and_sequences_without_queries(la, N):
    """More queries than tokens: the first see none (o = 0, lse = -inf); q_len 0: nothing written."""
    kv, nq = [0, 1, N - 1, N, 70], [N, N, N, 0, 0]
    cache, table = filled_cache(kv, 2, 32, 64, N, width=3)
    q = normal(N, 5, 4, N, 64).bfloat16()
    o, lse = attend_both(la, cache, table, q, kv, nq)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("N", [1, 48])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sizes_of_scores_and_values(la, N, dtype):
    """Large and small q, k, v and scale factors: scores of hundreds, values near the type's ends."""
    kv = [200, 77]
    top = 2.0 ** 12 if dtype == "fp16" else 2.0 ** 100
    for q_size, k_size, v_size, scale in ((30, 1, 1, None), (1e-3, 1, top, None), (top, 1 / top, 1, 0.1),
                                          (1, 1, 2.0 ** -12, -0.2), (1, 2.0 ** -60, 1, 2.0 ** 58),
                                          (1, 1, 1, 0.0)):
        cache, table = filled_cache(kv, 2, 16, 64, 5, k_size=k_size, v_size=v_size)
        q = (normal(3, 2, 4, N, 64) * q_size).to(TYPES[dtype])
        attend_both(la, cache, table, q, kv, [N, N], scale=scale, what=f"{q_size} {k_size} {v_size}")


@pytest.mark.parametrize("N", [1, 40])
def test_a_far_larger_score_keeps_the_small_weights(la, N):
    """One key far above thousands of others whose weights add up."""
    n, d = 3000, 64
    cache, table = filled_cache([n], 1, 64, d, 6, k_size=1e-3, width=60)
    first = table[0, 0]
    cache["k"][first, 0, 0] = oc.round_e4m3(np.full(d, 256.0))
    cache["k_scale"][first, 0] = 2.0 ** -7      # the first key: all twos
    q = torch.full((1, 1, N, d), 0.9).half()
    attend_both(la, cache, table, q, [n], [N], what="sink")


@pytest.mark.parametrize("N", [1, 33])
def test_blocks_of_very_different_size(la, N):
    """Scales that differ by 2^40 from page to page: the small values vanish beside the large
    ones, and matter where only they are seen."""
    kv = [100, 16]
    cache, table = filled_cache(kv, 1, 16, 64, 8)
    for p in range(7):
        cache["v_scale"][table[0, p]] *= 2.0 ** (-40 if p % 2 else 0)
        cache["k_scale"][table[0, p]] *= 2.0 ** (-40 if p % 3 else 0)
    cache["v_scale"][table[1, 0]] *= 2.0 ** -100
    q = normal(1, 2, 2, N, 64).bfloat16()
    attend_both(la, cache, table, q, kv, [min(N, n) for n in kv])


def test_a_nan_query_stays_in_its_row(la):
    cache, table = filled_cache([90, 90], 2, 16, 64, 9)
    for N in (1, 40):
        q = normal(1, 2, 4, N, 64).bfloat16()
        dev = to_device(la, cache, DEV)
        args = (dev, torch.from_numpy(table).to(DEV), ints([90, 90], DEV))
        ref = la.la_cache_attend(q.to(DEV), *args)
        q[1, 2, N // 2, 3] = float("nan")
        got = la.la_cache_attend(q.to(DEV), *args)
        assert torch.isnan(got[1, 2, N // 2]).all()
        got[1, 2, N // 2] = ref[1, 2, N // 2]
        assert torch.equal(got, ref)
    clean(la)


@pytest.mark.parametrize("N", [1, 40])
def test_attend_leaves_bad_lengths_out_and_follows_no_bad_page(la, N):
    kv = [64, 64, 64, 64]
    cache, table = filled_cache(kv, 1, 16, 64, 10)
    dev = to_device(la, cache, DEV)
    q = normal(1, 4, 1, N, 64).bfloat16().to(DEV)
    t = torch.from_numpy(table).to(DEV)
    ref = la.la_cache_attend(q, dev, t, ints(kv, DEV))
    clean(la)
    o = torch.full_like(q, 5.0)
    la.la_cache_attend(q, dev, t, ints([65, -1, 64, 64], DEV), q_len=ints([N, 1, N + 1, N], DEV), o=o)
    assert (o[:3] == 5).all() and torch.equal(o[3], ref[3])
    assert la.la_device_status() == (0, 2)
    bad = table.copy()
    bad[0, 1], bad[1, 3], bad[2, 0] = len(cache["k"]), -1, 2 ** 31 - 1
    o = la.la_cache_attend(q, dev, torch.from_numpy(bad).to(DEV), ints(kv, DEV))
    assert torch.isfinite(o).all() and torch.equal(o[3], ref[3])
    assert la.la_device_status() == (0, 2)


def test_lengths_at_the_end_of_32_bits_are_left_out(la):
    """A table of 2^31 tokens: lengths whose sums would pass 32 bits are refused, not followed."""
    page, big = 128, 2 ** 31 - 1
    cache, _ = filled_cache([page], 1, page, 64, 21)
    dev = to_device(la, cache, DEV)
    t = torch.zeros(1, 2 ** 31 // page, dtype=torch.int32, device=DEV)
    for N in (1, 40):
        q = normal(1, 1, 1, N, 64).half().to(DEV)
        o = torch.full_like(q, 5.0)
        la.la_cache_attend(q, dev, t, ints([big], DEV), o=o)
        assert (o == 5).all() and la.la_device_status() == (0, 2)
        k = [torch.full_like(q, 5.0) for _ in "kv"]
        la.la_cache_read(dev, t, ints([big - 1], DEV), *k)
        assert (k[0] == 5).all() and la.la_device_status() == (0, 2)
        la.la_cache_write(*k, dev, t, ints([big - 1], DEV))
        assert la.la_device_status() == (0, 2)
    same_cache(from_device(dev), cache)


def test_two_captured_graphs_with_a_workspace_each(la):
    """Graphs captured from one call each, replayed in turn and together on two streams."""
    cache, table = filled_cache([3000, 2000], 1, 16, 64, 22)
    dev, t, lens = to_device(la, cache, DEV), torch.from_numpy(table).to(DEV), ints([3000, 2000], DEV)
    qs = [normal(i, 2, 4, N, 64).half().to(DEV) for i, N in enumerate((2, 60))]
    refs = [la.la_cache_attend(q, dev, t, lens) for q in qs]
    need = [la.la_cache_attend_workspace_bytes(2, 4, 1, q.shape[2], 64) for q in qs]
    work = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in need]
    outs, graphs, streams = [torch.zeros_like(q) for q in qs], [], [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for q, o, ws, s in zip(qs, outs, work, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            la.la_cache_attend(q, dev, t, lens, o=o, workspace=ws, stream=s)
        graphs.append(g)
    for rounds in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, ref in zip(outs, refs):
            assert torch.equal(o, ref)
    clean(la)


@pytest.mark.parametrize("N", [1, 64])
def test_shared_pages_and_the_same_bits(la, N):
    """Two sequences on the pages of one prompt; repeated calls give the same bits."""
    cache, table = filled_cache([500], 2, 32, 128, 12)
    table = np.concatenate([table, table])
    q = normal(2, 1, 8, N, 128).bfloat16().expand(2, -1, -1, -1).contiguous()
    o, lse = attend_both(la, cache, table, q, [500, 500], [N, N])
    assert torch.equal(o[0], o[1]) or N > 1
    for _ in range(3):
        again, e = attend_both(la, cache, table, q, [500, 500], [N, N])
        assert torch.equal(again, o) and torch.equal(e, lse)


def test_a_long_sequence_split_over_the_gpu(la):
    """One sequence over all SMs: long split, parts joined, against the oracle at every row."""
    n, d, G = 9000, 128, 4
    cache, table = filled_cache([n], 1, 64, d, 13)
    for N in (1, 3, 8, 20):
        q = (normal(N, 1, G, N, d) * 2).bfloat16()
        attend_both(la, cache, table, q, [n], [N], what=f"N {N}")


def test_workspace_of_the_caller(la):
    cache, table = filled_cache([700], 2, 16, 64, 14)
    q = normal(1, 1, 4, 1, 64).half()
    need = la.la_cache_attend_workspace_bytes(1, 4, 2, 1, 64)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    o, lse = attend_both(la, cache, table, q, [700], [1], workspace=ws)
    o2, lse2 = attend_both(la, cache, table, q, [700], [1])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    with pytest.raises(la.LAError) as e:
        attend_both(la, cache, table, q, [700], [1], workspace=ws[:need - 256].clone())
    assert e.value.code == 5


def test_workspace_sizes_of_calls_that_are_refused(la):
    for bad in ((1, 66, 2, 8, 64), (1, 256, 1, 1, 128), (4097, 4, 4, 8, 64), (1, 4, 2, 2 ** 31 - 1, 64),
                (4096, 1 << 20, 1 << 20, 1, 64)):
        assert la.la_cache_attend_workspace_bytes(*bad) == 0, bad
    assert la.la_cache_attend_workspace_bytes(4096, 64, 2, 2 ** 31 - 257, 64) > 0


def test_offsets_beyond_32_bits(la):
    """A pool of more than 2^32 codes: the pages used lie at its end."""
    page, Hkv, d, n = 128, 4, 128, 300
    pages = (2 ** 32 + 2 ** 28) // (Hkv * page * d)
    small, table = filled_cache([n], Hkv, page, d, 15)
    codes = [torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.ones(pages, Hkv, device=DEV) for _ in "kv"]
    far = table + pages - len(small["k"])
    for name, c, s in zip("kv", codes, scales):
        c[pages - len(small["k"]):] = torch.from_numpy(small[name]).to(DEV)
        s[pages - len(small["k"]):] = torch.from_numpy(small[name + "_scale"]).float().to(DEV)
    dev = la.la_cache(*(c.view(torch.float8_e4m3fn) for c in codes), *scales)
    t = torch.from_numpy(far).to(DEV)
    for N in (1, 70):
        q = normal(N, 1, 8, N, d).bfloat16()
        ref = oc.attend(small, table, q.double().numpy(), [n], [N], d ** -0.5)
        o = la.la_cache_attend(q.to(DEV), dev, t, ints([n], DEV))
        assert_attend(o, None, ref, n, d, q.dtype, f"N {N}")
    k = normal(5, 1, Hkv, 20, d).bfloat16()
    la.la_cache_write(k.to(DEV), k.to(DEV), dev, t, ints([n - 20], DEV))
    ref = oc.write(small, table, k.double().numpy(), k.double().numpy(), [n - 20], [20])
    out = [torch.empty(1, Hkv, n, d, device=DEV) for _ in "kv"]
    la.la_cache_read(dev, t, ints([0], DEV), *out)
    for name, x in zip("kv", out):
        for h in range(Hkv):
            np.testing.assert_array_equal(x[0, h].double().cpu().numpy(),
                                          oc.tokens(ref, name, table[0], h, 0, n))
    clean(la)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("G,Hkv,d,page", [(4, 2, 128, 64), (3, 1, 64, 16)])
def test_a_conversation(la, G, Hkv, d, page):
    """As a model uses them: a prompt in two pieces, tokens one at a time, ragged batch."""
    B, steps = 2, 6
    pieces = [[37, 70], [50, 1]]
    total = [sum(p[b] for p in pieces) + steps for b in range(B)]
    table, num = pages_of(total, page, 16)
    ref = empty_cache(num, Hkv, page, d)
    dev, t = to_device(la, ref, DEV), torch.from_numpy(table).to(DEV)
    held = [0] * B
    for step, n in enumerate(pieces + [[1] * B] * steps):
        N = max(n)
        q, k, v = (normal(100 * step + j, B, Hkv * (G if j == 0 else 1), N, d).bfloat16() for j in range(3))
        ref = oc.write(ref, table, k.double().numpy(), v.double().numpy(), held, n)
        la.la_cache_write(k.to(DEV), v.to(DEV), dev, t, ints(held, DEV), count=ints(n, DEV))
        held = [a + b for a, b in zip(held, n)]
        o = torch.zeros_like(q, device=DEV)
        la.la_cache_attend(q.to(DEV), dev, t, ints(held, DEV), q_len=ints(n, DEV), o=o)
        want = oc.attend(ref, table, q.double().numpy(), held, n, d ** -0.5)
        assert_attend(o, None, want, max(held), d, q.dtype, f"step {step}")
    same_cache(from_device(dev), ref)
    clean(la)


def test_hybrid_layers_in_a_captured_graph(la):
    """A lightning layer's decode step and a softmax layer's token on one stream, captured once and
    replayed with lengths that move on the device."""
    B, Hq, Hkv, d, page, n0, steps = 2, 8, 2, 128, 16, 30, 4
    cache, table = filled_cache([n0] * B, Hkv, page, d, 17, width=4)
    free = sorted(set(range(len(cache["k"]))) - set(table[table >= 0].tolist()))
    table[0, 2], table[1, 2] = free[:2]
    ref = {n: a.copy() for n, a in cache.items()}
    dev, t = to_device(la, cache, DEV), torch.from_numpy(table).to(DEV)
    S = torch.zeros(B, Hkv, d, d, device=DEV)
    q, k, v = (torch.zeros(B, h, d, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    lin, o = torch.zeros_like(q), torch.zeros_like(q)
    start = torch.full((B,), n0, dtype=torch.int32, device=DEV)
    length = start + 1
    s = torch.cuda.Stream()

    def work():
        la.la_decode_step(S, q, k, v, o=lin, stream=s)
        la.la_cache_write(k[:, :, None], v[:, :, None], dev, t, start, stream=s)
        la.la_cache_attend(q[:, :, None], dev, t, length, o=o[:, :, None], stream=s)

    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        work()
    for c, name in zip(dev, ("k", "v", "k_scale", "v_scale")):   # what the first call stored goes
        back = torch.from_numpy(cache[name])
        c.view(torch.uint8).copy_(back.to(DEV)) if name in "kv" else c.copy_(back.float().to(DEV))
    for i in range(steps):
        x = [normal(200 + 3 * i + j, *y.shape).bfloat16() for j, y in enumerate((q, k, v))]
        for y, z in zip((q, k, v), x):
            y.copy_(z)
        start.fill_(n0 + i)
        length.fill_(n0 + i + 1)
        g.replay()
        torch.cuda.synchronize()
        ref = oc.write(ref, table, x[1].double().numpy()[:, :, None], x[2].double().numpy()[:, :, None],
                       [n0 + i] * B, [1] * B)
        want = oc.attend(ref, table, x[0].double().numpy()[:, :, None], [n0 + i + 1] * B, [1] * B, d ** -0.5)
        assert_attend(o[:, :, None], None, want, n0 + i + 1, d, torch.bfloat16, f"step {i}")
    same_cache(from_device(dev), ref)
    clean(la)


def test_two_streams_at_once(la):
    """Calls on two streams without an order between them, each with a workspace of its own."""
    cache, table = filled_cache([900, 900], 2, 16, 128, 18)
    dev, t = to_device(la, cache, DEV), torch.from_numpy(table).to(DEV)
    lens = ints([900, 900], DEV)
    qs = [normal(i, 2, 8, N, 128).bfloat16().to(DEV) for i, N in enumerate((1, 100))]
    refs = [la.la_cache_attend(q, dev, t, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[torch.empty_like(q) for _ in range(10)] for q in qs]
    for i in range(10):
        for q, s, o in zip(qs, streams, outs):
            la.la_cache_attend(q, dev, t, lens, o=o[i], stream=s)
    torch.cuda.synchronize()
    for ref, o in zip(refs, outs):
        assert all(torch.equal(x, ref) for x in o)
    clean(la)


@pytest.mark.parametrize("G,Hkv,N", [(4, 2, 1), (5, 3, 4), (32, 1, 1), (7, 2, 9), (24, 1, 40), (1, 3, 200)])
def test_cut_units_are_whole_ones(la, G, Hkv, N):
    """The same call over a table of the sequences' own length (units whole, where short) and over
    one with room for far more (the general way)."""
    kv = [N + 100, N, N + 211, 1, 260]
    nq = [N, N, max(1, N - 1), 1, 1]
    cache, table = filled_cache(kv, Hkv, 16, 64, G)
    q = normal(N, 5, Hkv * G, N, 64).half()
    wide = np.full((5, 4096), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    attend_both(la, cache, table, q, kv, nq, what="short table")
    attend_both(la, cache, wide, q, kv, nq, what="wide table")


@pytest.mark.parametrize("d,G", [(64, 3), (128, 4)])
def test_many_short_units_for_each_block(la, d, G):
    """Ragged prompts of several users: a block works on three units and more, some of one key tile."""
    nq = [777, 400, 130, 61, 700, 256]
    kv = [n + past for n, past in zip(nq, [0, 37, 600, 300, 128, 0])]
    cache, table = filled_cache(kv, 4, 32, d, 20)
    q = normal(4, 6, 4 * G, 777, d).half()
    for b, n in enumerate(nq):   # the oracle takes some rows of each sequence
        q[b, :, n:] = 0
    dev, t = to_device(la, cache, DEV), torch.from_numpy(table).to(DEV)
    lse = torch.zeros(q.shape[:3], device=DEV)
    o = la.la_cache_attend(q.to(DEV), dev, t, ints(kv, DEV), q_len=ints(nq, DEV), lse=lse)
    for b, n in enumerate(nq):
        rows = sorted({0, 1, n - 1, n // 2, *range(40, n, 97)})
        for i in rows:
            ref = oc.attend(cache, table[b:b + 1], q[b:b + 1, :, i:i + 1].double().numpy(),
                            [kv[b] - n + i + 1], [1], d ** -0.5)
            assert_attend(o[b:b + 1, :, i:i + 1], lse[b:b + 1, :, i:i + 1], ref, kv[b], d, q.dtype,
                          f"sequence {b} row {i}")
    clean(la)


def test_a_large_batch(la):
    """More sequences than SMs, lengths all different."""
    B, d, page = 300, 64, 16
    kv = [1 + (37 * b) % 150 for b in range(B)]
    cache, table = filled_cache(kv, 1, page, d, 19)
    q = normal(3, B, 2, 1, d).half()
    attend_both(la, cache, table, q, kv, [1] * B)
