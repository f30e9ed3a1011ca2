"""The tcgen05 prefill kernel gives up with copies, products and launch-control
requests of many CTAs under way: the call returns with code 2, and the calls
after it give the bits of the calls before."""
import time

import pytest
import torch

from paged_kv_cache_255_gb300 import inputs
from paged_kv_cache_255_gb300 import pagedattn as pa
from test_gpu_prefill import _device, _gpu_step, _spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


# a few CTAs, and more than run at once: later ones are taken over or start when those have ended
@pytest.mark.parametrize("Hq,Hkv,lens", [(16, 2, [600, 40]), (32, 8, [900, 300, 700, 500, 900, 260, 640, 384])])
def test_a_held_arrival_is_reported_and_the_next_calls_are_right(Hq, Hkv, lens):
    pb = inputs.prefill_batch(_spec("giveup", Hq, Hkv, 16), seed=70, context_lens=lens,
                              chunk_lens=[min(n, 200) for n in lens])
    d = _device(pb)
    want = _gpu_step(pb, d)
    torch.cuda.synchronize()
    assert pa.take_device_error() == 0
    pa.debug_prefill_fault(1)
    try:
        t0 = time.time()
        _gpu_step(pb, d)
        torch.cuda.synchronize()
        dt = time.time() - t0
    finally:
        pa.debug_prefill_fault(0)
    assert pa.take_device_error() == 2
    assert 1.0 < dt < 60.0, dt
    for _ in range(3):
        assert torch.equal(_gpu_step(pb, d).view(torch.int16), want.view(torch.int16))
    assert pa.take_device_error() == 0
