"""Tables as wide as the token counts of decode over shared prefixes allow, on the
CPU: one more block is refused, whatever the lengths are, before any CUDA call."""
import pytest

from paged_kv_cache_255_gb300 import pagedattn as pa


@pytest.mark.parametrize("bs", [16, 64, 128, 256])
def test_tables_past_the_token_counts_are_refused(pa_lib, bs):
    def call(mb):       # no workspace: what the checks let through ends there, or at the missing GPU
        return pa_lib.pa_decode_shared(16, 16, 16, 16, mb, 16, 16, 16, 2, 0.1, 16, 2, 16, 8, 128, bs, 10, 0, None, 0,
                                       None)
    most = (2 ** 31 - 128) // bs
    assert call(most) in (pa.PA_ERR_WORKSPACE, pa.PA_ERR_CUDA)
    for mb in (most + 1, 2 ** 31 - 1):
        assert call(mb) == pa.PA_ERR_UNSUPPORTED
