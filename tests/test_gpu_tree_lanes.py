"""Decode over trees whose sequences all have the same number of units: side by side in lanes,
or, where that would leave CTAs without a share, in one."""
import numpy as np
import pytest

from paged_kv_cache_255_gb300 import pagedattn as pa
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


# units a sequence and KV head, of 16 tokens each: divisors of 152 and not, more than an eighth
# left over and less, more than 152
@pytest.mark.parametrize("units", [2, 9, 19, 22, 52, 64, 77, 152, 153])
@pytest.mark.parametrize("S", [1, 3])
def test_units_of_every_number(units, S):
    pa.take_device_error()
    rng = np.random.default_rng(units)
    nodes = rng.integers(16 * units - 15, 16 * units + 1, S)
    same = int(rng.integers(1, 1 << 40)) | 1
    b = Batch(rng.integers(0, 700, S), nodes, 32, 2, masks=lambda r, n: [same & (1 << n) - 1] * n, mask_words=3,
              seed=units)
    assert (b.run() == b.check()).all()
