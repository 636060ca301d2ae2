"""Calls of the 8-bit cache's entry points that a program could make by mistake, or from two streams."""
import pytest
import torch

from _cache_cases import filled_cache, ints, normal, to_device

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
