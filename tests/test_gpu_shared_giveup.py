"""The prefix kernel of decode over shared prefixes gives up a wait that does not
end: with the test hook holding back one barrier arrival in every CTA, the call
returns after about 2 s with code 2 instead of hanging. Every role first lets
what it has in flight land, the CTAs give back their tensor memory, and the next
calls are right."""
import time

import pytest
import torch

from paged_kv_cache_255_gb300 import pagedattn as pa
from test_gpu_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


# one unit, long units that every CTA shares, and many units of both layouts
@pytest.mark.parametrize("sizes,blocks,Hq,Hkv,hm", [
    ([20], [9], 16, 1, False), ([128], [300], 64, 8, False), ([64, 60], [40, 90], 32, 4, True),
])
def test_a_held_arrival_is_reported_and_the_next_calls_are_right(sizes, blocks, Hq, Hkv, hm):
    b = Batch(sizes, blocks, [3, 40], Hq, Hkv, hm=hm)
    want = b.check()
    pa.debug_prefill_fault(1)
    try:
        t0 = time.time()
        b.run()
        torch.cuda.synchronize()
        dt = time.time() - t0
    finally:
        pa.debug_prefill_fault(0)
    assert pa.take_device_error() == 2
    assert 1.0 < dt < 30.0, dt
    for _ in range(3):
        assert torch.equal(b.check(), want)
