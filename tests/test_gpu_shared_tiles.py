"""Decode over shared prefixes on long prefixes, where a lost, doubled or stale key
tile must show: coded keys and values, and the relative error of every row
(tile_codes)."""
import numpy as np
import pytest
import torch

import tile_codes as tc
from paged_kv_cache_255_gb300 import pagedattn as pa
from test_gpu_shared import Batch, reference

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


# on the prefix kernel: shares of many tiles, several shares a unit, pairs of query tiles in
# lanes; and packed prefixes: a few sequences of few heads
SHAPES = [
    (20, 3000, 16, 1, 16, False), (9, 2999, 16, 1, 16, False), (128, 1000, 16, 1, 16, False),
    (20, 701, 16, 1, 16, True), (64, 512, 32, 8, 64, True), (256, 300, 32, 8, 16, False), (300, 40, 8, 2, 256, False),
    (2, 2500, 2, 1, 16, False), (5, 1000, 16, 8, 16, False), (4, 180, 16, 8, 128, True),
]


@pytest.mark.parametrize("n,blocks,Hq,Hkv,bs,hm", SHAPES)
def test_coded_keys(n, blocks, Hq, Hkv, bs, hm):
    rng = np.random.default_rng(n + blocks)
    own = np.array([[3, 40, 700, 0, 129][i % 5] for i in range(n)])
    own_nb = -(-own // bs)
    width, NB = blocks + int(own_nb.max()), 2 + blocks + int(own_nb.sum())
    ids = 1 + rng.permutation(NB - 1)
    tables = np.full((n, width), NB + 5, np.int32)
    tables[:, :blocks] = ids[:blocks]
    at, place = blocks, np.zeros(NB, np.int64)              # place: the block's first token in its sequence
    place[ids[:blocks]] = np.arange(blocks) * bs
    for s in range(n):
        for j in range(own_nb[s]):
            tables[s, blocks + j] = ids[at]
            place[ids[at]] = (blocks + j) * bs
            at += 1
    # head h holds the codes of the tokens 16 * 7 h further on
    shift = 112 * torch.arange(Hkv, device="cuda")
    code = torch.stack(tc.coded_rows(width * bs + 112 * Hkv, "cuda"))
    t = torch.from_numpy(place).cuda()[:, None, None] + torch.arange(bs, device="cuda")[:, None] + shift
    kv = code[:, t]                                          # [2, NB, bs, Hkv, D]
    kv[:, ids[-1]] = float("nan")                            # a block of nobody
    if hm:
        kv = kv.transpose(2, 3).contiguous()
    q = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    dim = torch.arange(n * Hq, device="cuda").view(n, Hq) % D
    q.scatter_(2, dim[..., None], 400.0)                     # dim 127 meets no key: all count the same
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = torch.tensor(blocks * bs + own, **i32)
    args = (q, kv[0], kv[1], torch.tensor(tables, **i32), lens)
    groups = (torch.tensor([0, n], **i32), torch.tensor([blocks], **i32))
    outs = [pa.decode_shared(*args, *groups, D ** -0.5, head_major=hm) for _ in range(3)]
    assert pa.take_device_error() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    got = outs[0].double().view(n, Hkv, Hq // Hkv, D)
    for s in range(n):
        for h in range(Hkv):
            rows = code[:, 112 * h:112 * h + int(lens[s])]
            o, A = tc.attend(q.view(n, Hkv, -1, D)[s, h], rows[0], rows[1], D ** -0.5)
            assert ((got[s, h] - o).abs() <= tc.element_bound(o, A)).all(), (s, h)


@pytest.mark.parametrize("sizes,blocks,Hq,Hkv,own", [
    ([128], [1000], 16, 1, [3, 40]), ([20], [3000], 16, 1, [3, 40]), ([9], [2999], 16, 1, [3, 40]),
    ([256], [1100], 32, 8, [16, 700, 0]), ([64, 60], [300, 533], 16, 2, [300, 1]), ([4], [1000], 16, 8, [3, 90]),
    ([2], [2500], 2, 1, [1, 700]), ([50, 2], [400, 900], 32, 4, [9, 130]), ([3], [300], 8, 8, [6000]),
])
def test_relative_error_of_every_row(sizes, blocks, Hq, Hkv, own):
    b = Batch(sizes, blocks, own, Hq, Hkv)
    out = b.check()
    o, _ = reference(b.q, b.k, b.v, b.tables, b.lens, b.scale, b.bs, b.hm)
    err = tc.row_error(out, o)
    assert (err <= tc.ROW_REL).all(), err.max()
