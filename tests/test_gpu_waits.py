"""The kernels' bounded waits run out where nothing arrives, say so in the status word and leave the
context usable."""
import pytest
import torch

from _cache_cases import filled_cache, ints, normal, to_device

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_both_kinds_of_wait_run_out(la):
    la.la_device_status()
    cache, table = filled_cache([70], 1, 16, 64, 1)
    dev, t = to_device(la, cache, DEV), torch.from_numpy(table).to(DEV)
    q = normal(1, 1, 1, 50, 64).half().to(DEV)
    ref = la.la_cache_attend(q, dev, t, ints([70], DEV))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    la.api.la_selftest_wait(5_000_000)
    end.record()
    assert la.la_device_status() == (4, 1)
    assert 5 < begin.elapsed_time(end) < 1000     # the flag's 5 ms, the barrier's thousand tries
    assert torch.equal(la.la_cache_attend(q, dev, t, ints([70], DEV)), ref)
    assert la.la_device_status() == (0, 0)
