"""Refusals of the 8-bit cache's entry points, without a GPU: the C ABI before any device
call, and the binding before any library call."""
import ctypes

import pytest
import torch

from linear_attention_11_b200 import api

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
e4m3 = torch.float8_e4m3fn


def c_cache(**change):
    at = {"k_codes": 1 << 20, "v_codes": 2 << 20, "k_scale": 3 << 20, "v_scale": (3 << 20) + 4096,
          "num_pages": 4, "Hkv": 2, "page": 16, "d": 64}
    at |= change
    return api._la_cache(*(at[n] for n, _ in api._la_cache._fields_))


P = ctypes.c_void_p
K, V, T, S, C, Q, O = (P(n << 20) for n in (8, 9, 10, 11, 12, 16, 17))


def write(la, k=K, v=V, dtype=0, cache=None, table=T, start=S, count=C, B=1, N=8, max_pages=4, **c):
    cache = ctypes.byref(c_cache(**c)) if cache is None else cache
    return la.api.load_library().la_cache_write(k, v, dtype, cache, table, start, count, B, N,
                                                max_pages, None)


def read(la, k=K, v=V, dtype=0, table=T, start=S, B=1, N=8, max_pages=4, **c):
    return la.api.load_library().la_cache_read(ctypes.byref(c_cache(**c)), table, start, None, k, v,
                                               dtype, B, N, max_pages, None)


def attend(la, q=Q, dtype=0, table=T, kv_len=S, q_len=C, o=O, lse=None, B=1, Hq=4, N=8, max_pages=4,
           scale=0.125, **c):
    return la.api.load_library().la_cache_attend(q, dtype, ctypes.byref(c_cache(**c)), table, kv_len,
                                                 q_len, o, lse, B, Hq, N, max_pages, scale, None)


@pytest.mark.parametrize("call", [write, read, attend])
def test_shared_refusals(la, call):
    for change in (dict(k_codes=None), dict(v_codes=None), dict(k_scale=None), dict(v_scale=None),
                   dict(num_pages=0), dict(Hkv=0), dict(page=0), dict(d=0), dict(B=0), dict(N=0),
                   dict(max_pages=0), dict(N=1 << 31), dict(table=None), dict(k_codes=(1 << 20) + 8),
                   dict(k_scale=(3 << 20) + 2), dict(num_pages=1 << 31), dict(dtype=3),
                   dict(dtype=-1)):
        assert call(la, **change) == 1, change
    for change in (dict(page=8), dict(page=48), dict(page=256), dict(d=32), dict(d=96), dict(d=256)):
        assert call(la, **change) == 2, change


@pytest.mark.parametrize("call", [write, read])
def test_write_and_read_refusals(la, call):
    for change in (dict(k=None), dict(v=None), dict(start=None), dict(k=P((8 << 20) + 8)),
                   dict(start=P((11 << 20) + 2)), dict(k=P(1 << 20)), dict(v=P((2 << 20) + 64))):
        assert call(la, **change) == 1, change
    assert write(la, count=P((12 << 20) + 1)) == 1
    assert write(la, v_codes=(1 << 20) + 16) == 1          # codes over codes
    assert write(la, cache=ctypes.POINTER(api._la_cache)()) == 1
    assert read(la, v=K) == 1                              # k over v


def test_attend_refusals(la):
    for change in (dict(q=None), dict(o=None), dict(kv_len=None), dict(Hq=3), dict(Hq=0), dict(o=Q),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(q=P((16 << 20) + 2)),
                   dict(o=P(1 << 20)), dict(lse=O), dict(lse=P((20 << 20) + 2)),
                   dict(q_len=P((12 << 20) + 2))):
        assert attend(la, **change) == 1, change
    for change in (dict(dtype=2), dict(Hq=66), dict(B=4097)):
        assert attend(la, **change) == 2, change
    for bad in ((0, 4, 2, 8, 64), (1, 3, 2, 8, 64), (1, 4, 2, 0, 64), (1, 4, 2, 8, 96)):
        assert la.la_cache_attend_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ the binding
class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLib()
    monkeypatch.setattr(api, "load_library", lambda path=None: lib)
    monkeypatch.setattr(api, "_stream", lambda stream: None)
    monkeypatch.setattr(api, "_on_device", lambda t: getattr(t, "on_host", False) is False)
    return lib


def host(t):
    t.on_host = True
    return t


def parts(B=2, Hq=4, Hkv=2, N=3, d=64, page=16, pages=5, dtype=bf16):
    codes = torch.zeros(pages, Hkv, page, d, dtype=torch.uint8).view(e4m3)
    cache = api.la_cache(codes, codes.clone(), torch.ones(pages, Hkv), torch.ones(pages, Hkv))
    return (torch.zeros(B, Hq, N, d, dtype=dtype), torch.zeros(B, Hkv, N, d, dtype=dtype), cache,
            torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32))


def test_well_formed_calls_reach_the_library(fake):
    q, k, cache, table, n = parts()
    api.la_cache_write(k, k.clone(), cache, table, n)
    api.la_cache_write(k.float(), k.float(), cache, table, n, count=n)
    api.la_cache_read(cache, table, n, k.half(), k.half(), count=n)
    api.la_cache_attend(q, cache, table, n)
    api.la_cache_attend(q.half(), cache, table, n, q_len=n, lse=torch.zeros(2, 4, 3), scale=0.5)
    api.la_cache_attend(q, cache, table, n, workspace=torch.zeros(64, dtype=torch.uint8))
    assert [c[0] for c in fake.calls] == ["la_cache_write"] * 2 + ["la_cache_read"] + \
        ["la_cache_attend"] * 2 + ["la_cache_attend_ws"]
    assert fake.calls[3][1][-2] == 0.125 and fake.calls[4][1][-2] == 0.5
    assert [c[1][2] for c in fake.calls[:2]] == [0, 2] and fake.calls[4][1][1] == 1


def test_binding_refusals(fake):
    q, k, cache, table, n = parts()
    bad = [
        ("float8", lambda: api.la_cache_write(k, k, cache._replace(k_codes=cache.k_codes.view(torch.uint8)), table, n)),
        ("float32", lambda: api.la_cache_write(k, k, cache._replace(v_scale=cache.v_scale.double()), table, n)),
        ("num_pages", lambda: api.la_cache_write(k, k, cache._replace(v_scale=cache.v_scale[:4]), table, n)),
        ("int32", lambda: api.la_cache_write(k, k, cache, table.long(), n)),
        ("max_pages", lambda: api.la_cache_write(k, k, cache, table[0], n)),
        ("start must be", lambda: api.la_cache_write(k, k, cache, table, n[:1])),
        ("count must be", lambda: api.la_cache_write(k, k, cache, table, n, count=torch.zeros(3, dtype=torch.int32))),
        ("CUDA", lambda: api.la_cache_write(host(k.clone()), k, cache, table, n)),
        ("CUDA", lambda: api.la_cache_write(k, k, cache, table, host(n.clone()))),
        ("contiguous", lambda: api.la_cache_write(k.transpose(1, 2), k, cache, table, n)),
        ("expected k", lambda: api.la_cache_write(k, k[:, :, :2].contiguous(), cache, table, n)),
        ("expected k", lambda: api.la_cache_read(cache, table, n, k[:1], k[:1])),
        ("one type", lambda: api.la_cache_read(cache, table, n, k, k.half())),
        ("one type", lambda: api.la_cache_read(cache, table, n, k.double(), k.double())),
        ("bfloat16 or float16", lambda: api.la_cache_attend(q.float(), cache, table, n)),
        ("must be torch.bfloat16", lambda: api.la_cache_attend(q, cache, table, n, o=q.half())),
        ("expected q", lambda: api.la_cache_attend(q[..., :32].contiguous(), cache, table, n)),
        ("expected q", lambda: api.la_cache_attend(q, cache, table, n, o=q[:, :2].contiguous())),
        ("lse must be", lambda: api.la_cache_attend(q, cache, table, n, lse=torch.zeros(2, 4))),
        ("required", lambda: api.la_cache_attend(q, cache, table, None)),
        ("CUDA", lambda: api.la_cache_attend(q, cache, table, n, workspace=host(torch.zeros(64)))),
    ]
    for match, call in bad:
        with pytest.raises(ValueError, match=match):
            call()
    assert fake.calls == []


def test_sizes_beyond_a_grid_are_refused(la):
    """More pages or runs of tokens than a grid has blocks: an argument error, like other sizes."""
    N, Hkv = 2 ** 31 - 300, 2
    for B in (9, 64, 2 ** 20):
        assert write(la, N=N, B=B, Hkv=Hkv) == 1, B
    for B in (64, 2 ** 20):
        there = P((8 << 20) + B * Hkv * N * 64 * 2)   # v behind k
        assert read(la, N=N, B=B, Hkv=Hkv, v=there) == 1, B


def test_tables_and_lengths_that_the_call_would_write_over(la):
    """The kernels read them as they go: nothing that a call writes may lie over them."""
    over_codes, over_scale = P((1 << 20) + 256), P((3 << 20) + 4096)
    for at in (over_codes, over_scale):
        for name in ("table", "start", "count"):
            assert write(la, **{name: at}) == 1, name
    for name in ("table", "start"):
        for at in (K, P((9 << 20) + 1024)):
            assert read(la, **{name: at}) == 1, name
    for name in ("table", "kv_len", "q_len"):
        assert attend(la, **{name: P((17 << 20) + 64)}) == 1, name
        assert attend(la, lse=P(20 << 20), **{name: P((20 << 20) + 4)}) == 1, name
    assert write(la, table=P((1 << 20) - 12)) == 1   # its last entry


def test_a_table_or_codes_without_dimensions(fake):
    q, k, cache, table, n = parts()
    none = torch.zeros((), dtype=torch.int32)
    with pytest.raises(ValueError, match="max_pages"):
        api.la_cache_attend(q, cache, none, n)
    with pytest.raises(ValueError, match="max_pages"):
        api.la_cache_write(k, k, cache, none, n)
    with pytest.raises(ValueError, match="num_pages"):
        api.la_cache_read(cache._replace(k_codes=torch.zeros((), dtype=torch.uint8).view(e4m3)), table, n, k, k.clone())
    with pytest.raises(ValueError, match="start must be"):
        api.la_cache_write(k, k, cache, table, none)
    assert fake.calls == []
