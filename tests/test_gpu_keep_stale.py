"""Lists of kept tokens with what earlier drafts left behind their ends: nothing there is
followed, moved or recorded, also where a place of that number would lie behind the table."""
import numpy as np
import pytest
import torch

import blocks_ref
import tree_ref as ref
from paged_kv_cache_255_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


# Tables filled to their last token and in the middle of a larger buffer whose other words are
# no block ids, lists of 1024 places for drafts of 1 to 33 nodes.
@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("n,lead", [(1, []), (1, [0]), (2, [1]), (7, [0, 2, 5]), (33, [3, 4, 32]), (33, list(range(33)))])
@pytest.mark.parametrize("m", [64, 1000, 1024])
def test_what_stands_behind_the_end_is_nobodys(n, lead, m, hm):
    if len(lead) >= m:
        pytest.skip("no place behind the end")
    bs, Hkv, S, width = 16, 2, 3, 3
    rng = np.random.default_rng(n + m)
    NB = 2 + S * width
    big = np.full(4 * S * width, NB + 7, np.int32)
    tables = big[S * width:2 * S * width].reshape(S, width)
    tables[:] = 1 + rng.permutation(NB - 1)[:S * width].reshape(S, width)
    lens = np.full(S, bs * width, np.int32)
    starts = np.arange(S + 1, dtype=np.int32) * n
    refs = blocks_ref.counts(tables, lens, NB, bs)
    stale = np.where(np.arange(m) % 2, np.arange(m) // 2 % n, -1)       # -1, 0, -1, 1, ...
    kept = np.tile(stale, (S, 1)).astype(np.int32)
    kept[:, :len(lead)] = lead
    kept[:, len(lead)] = -1
    kept[1, len(lead) + 1:] = np.arange(m - len(lead) - 1) % n
    shape = (NB, Hkv, bs, D) if hm else (NB, bs, Hkv, D)
    pools = [rng.integers(0, 1 << 16, size=shape, dtype=np.uint16) for _ in range(2)]
    d_big, d_lens, d_starts, d_kept, d_refs = (torch.from_numpy(x.copy()).cuda() for x in (big, lens, starts, kept, refs))
    d_pools = [torch.from_numpy(p.view(np.int16).copy()).cuda().view(torch.bfloat16) for p in pools]
    d_tables = d_big[S * width:2 * S * width].view(S, width)
    pa.take_device_error()
    pa.keep_tokens(pa.CachePools(d_pools, head_major=hm), d_tables, d_lens, d_starts, d_kept, ref_counts=d_refs)
    assert ref.keep(pools, tables, lens, starts, kept, refs, bs, hm) == set()
    assert pa.take_device_error() == 0
    assert lens.tolist() == [bs * width - n + len(lead)] * S
    for got, want in ((d_big, big), (d_lens, lens), (d_refs, refs)):
        assert np.array_equal(got.cpu().numpy(), want)
    for p, x in zip(pools, d_pools):
        assert np.array_equal(x.view(torch.int16).cpu().numpy().view(np.uint16), p)
