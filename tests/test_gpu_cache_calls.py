"""Calls of the 8-bit cache's entry points that a program could make by mistake, or from two streams."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

from _cache_cases import attend_bounds, filled_cache, ints, normal, to_device

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_a_workspace_over_the_table_or_a_length(la):
    """Refused: the kernels read both while they write the workspace."""
    cache, table = filled_cache([700], 2, 16, 64, 14)
    dev, q = to_device(la, cache, DEV), normal(1, 1, 4, 1, 64).half().to(DEV)
    need = la.la_cache_attend_workspace_bytes(1, 4, 2, 1, 64)
    room = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
    t = room[need - 64:need - 64 + table.nbytes].view(torch.int32).view(table.shape)
    t.copy_(torch.from_numpy(table))
    length = room[1024:1028].view(torch.int32)
    length.fill_(700)
    ref = la.la_cache_attend(q, dev, t, length)
    for args in ((t, length.clone()), (t.clone(), length)):
        with pytest.raises(la.LAError) as e:
            la.la_cache_attend(q, dev, *args, workspace=room[:need])
        assert e.value.code == 5
    got = la.la_cache_attend(q, dev, t.clone(), ints([700], DEV), workspace=room[:need])
    assert torch.equal(got, ref) and la.la_device_status() == (0, 0)


@pytest.mark.parametrize("call", ["cache_attend", "forward", "forward_state", "decode_step", "decode_steps",
                                  "backward", "segment_state"])
def test_what_a_call_makes_is_its_streams(la, call):
    """An output that a call on another stream makes does not lie in memory that the current stream has
    just given back and may still be working on."""
    B, H, N, d = 2, 4, 1024, 128
    q, k, v = (normal(i, B, H, N, d).bfloat16().to(DEV) for i in range(3))
    S = torch.zeros(B, H, d, d, device=DEV)
    s = torch.cuda.Stream()
    if call == "cache_attend":
        cache, table = filled_cache([1100, 1030], H, 32, d, 1)
        dev, t, n = to_device(la, cache, DEV), torch.from_numpy(table).to(DEV), ints([1100, 1030], DEV)
        run = lambda stream: la.la_cache_attend(q, dev, t, n, stream=stream)  # noqa: E731
    elif call == "decode_step":
        one = [x[:, :, 0].contiguous() for x in (q, k, v)]
        run = lambda stream: la.la_decode_step(S.clone(), *one, stream=stream)  # noqa: E731
    elif call == "decode_steps":
        some = [x[:, :, :8].contiguous() for x in (q, k, v)]
        run = lambda stream: la.la_decode_steps(S.clone(), *some, stream=stream)  # noqa: E731
    elif call == "backward":
        run = lambda stream: la.la_backward(q, k, v, q, stream=stream)[0]  # noqa: E731
    elif call == "segment_state":
        run = lambda stream: la.la_segment_state(k, v, stream=stream)  # noqa: E731
    else:
        run = lambda stream: getattr(la, "la_" + call)(q, k, v, stream=stream)  # noqa: E731
    ref = run(None)
    torch.cuda.synchronize()
    freed = {ref.data_ptr()}
    keep, ref = ref.clone(), None
    for _ in range(4):                 # memory of this size that the current stream gave back
        x = torch.empty_like(keep)
        freed.add(x.data_ptr())
        del x
    torch.cuda.synchronize()
    o = run(s)
    torch.cuda.synchronize()
    assert torch.equal(o, keep)
    assert o.data_ptr() not in freed
    assert la.la_device_status() == (0, 0)


@pytest.mark.parametrize("G,N,d", [(4, 64, 128), (1, 1, 64), (4, 5, 128), (2, 300, 64)])
def test_sequences_on_the_same_pages(la, G, N, d):
    """Over a short table units are whole: two sequences on one prompt's pages, the same call in another
    batch and repeated calls give the same bits.  Over a long one they are cut by the whole batch's line:
    the same to what the order of fp32 sums and the reference maxima (weights are rounded relative to them)
    leave open, once for each of the two."""
    cache, table = filled_cache([500], 2, 32, d, 12)
    dev = to_device(la, cache, DEV)
    q = normal(2, 1, 2 * G, N, d).bfloat16().expand(2, -1, -1, -1).contiguous()
    short = torch.from_numpy(table).to(DEV).expand(2, -1).contiguous()
    wide = torch.full((2, 4096), -1, dtype=torch.int32, device=DEV)
    wide[:, :short.shape[1]] = short
    n = ints([500, 500], DEV)
    o = la.la_cache_attend(q.to(DEV), dev, short, n)
    assert torch.equal(o[0], o[1])
    assert torch.equal(la.la_cache_attend(q[:1].to(DEV), dev, short[:1], n[:1]), o[:1])
    ref = oc.attend(cache, table, q[:1].double().numpy(), [500], [N], d ** -0.5)
    cut = la.la_cache_attend(q.to(DEV), dev, wide, n)
    assert torch.equal(la.la_cache_attend(q.to(DEV), dev, wide, n), cut)
    bound = 2 * attend_bounds(ref, 500, d, q.dtype)[0][0]
    for x in (cut[0], cut[1]):
        assert (np.abs((x - o[0]).double().cpu().numpy()) <= bound).all()
    assert la.la_device_status() == (0, 0)
