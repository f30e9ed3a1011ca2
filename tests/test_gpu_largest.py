"""Rotations, trees and kept tokens at the largest numbers of tokens and sequences that they
are made for."""
import numpy as np
import pytest
import torch

import tile_codes as tc
import tree_ref as ref
from paged_kv_cache_255_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


@pytest.fixture(autouse=True)
def _no_error_left():
    pa.take_device_error()
    yield
    pa.take_device_error()


def test_rotation_of_16_million_tokens():
    # 2.1e9 elements on either side
    T = (1 << 24) + 5
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    q = torch.empty(T, 1, D, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    pos = torch.randint(0, 1 << 31, (T,), generator=gen, device="cuda").int()
    R, w = pa.Rotary(128), torch.randn(D, generator=gen, device="cuda").bfloat16()
    out, _ = pa.rotate(q, None, pos, R, q_weight=w)
    # every row is what a short call makes of it: sampled ones and both ends
    at = torch.cat([torch.randint(0, T, (50000,), generator=gen, device="cuda"), torch.arange(64, device="cuda"),
                    torch.arange(T - 64, T, device="cuda")])
    assert torch.equal(out[at], pa.rotate(q[at], None, pos[at], R, q_weight=w)[0])
    del q, out


def test_trees_of_70000_sequences():
    S, bs, Hq, blocks = 70000, 16, 4, 3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    rnd = lambda lo, hi, n: torch.randint(lo, hi, (n,), generator=gen, device="cuda")      # noqa: E731
    n, base = rnd(0, 4, S), rnd(0, 46, S)
    L = base + n
    starts = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), n.cumsum(0)])
    T = int(starts[-1])
    k, v = (torch.empty(S * blocks, bs, 1, D, device="cuda", dtype=torch.bfloat16).normal_(generator=gen) for _ in range(2))
    q = torch.empty(T, Hq, D, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    tables = torch.randperm(S * blocks, generator=gen, device="cuda").view(S, blocks)
    mask = rnd(0, 8, T)
    out = torch.full_like(q, 77.0)
    pa.decode_tree(q, k, v, tables.int(), L.int(), starts.int(), mask[:, None].contiguous(), D ** -0.5, out=out)
    assert pa.take_device_error() == 0
    t = torch.arange(blocks * bs, device="cuda")
    owner = torch.repeat_interleave(torch.arange(S, device="cuda"), n)
    for rows in torch.arange(T, device="cuda").split(20000):
        s = owner[rows]
        node = t - base[s][:, None]                                     # of each token of the table
        seen = ((node < 0) | (mask[rows][:, None] >> node.clamp(0, 3) & 1).bool()) & (t < L[s][:, None])
        K, V = (x[tables[s]].view(len(rows), -1, D).double() for x in (k, v))
        a = torch.einsum("rhd,rtd->rht", q[rows].double(), K) * D ** -0.5
        p = torch.softmax(a.masked_fill(~seen[:, None], -torch.inf), -1).nan_to_num(0.0)
        o, A = torch.einsum("rht,rtd->rhd", p, V), torch.einsum("rht,rtd->rhd", p, V.abs())
        assert ((out[rows].double() - o).abs() <= tc.element_bound(o, A)).all()


@pytest.mark.parametrize("hm", [False, True])
def test_keeping_tokens_of_65535_sequences(hm):
    S, bs, n = 65535, 16, 3
    rng = np.random.default_rng(6)
    NB = 2 * S + 1
    tables = (1 + rng.permutation(NB - 1)).reshape(S, 2).astype(np.int32)
    lens = rng.integers(17, 33, S).astype(np.int32)
    starts = np.arange(S + 1, dtype=np.int32) * n
    refs = np.ones(NB, np.int32)
    paths = np.array([[-1, 0, 1], [0, -1, 2], [1, -1, -1], [2, -1, 2], [0, 2, -1], [1, 2, -1], [0, 1, 2]], np.int32)
    kept = paths[rng.integers(0, len(paths), S)]
    pool = rng.integers(0, 1 << 16, size=(NB, 1, bs, D) if hm else (NB, bs, 1, D), dtype=np.uint16)
    d = [torch.from_numpy(x.copy()).cuda() for x in (tables, lens, starts, kept, refs)]
    x = torch.from_numpy(pool.view(np.int16).copy()).cuda().view(torch.bfloat16)
    pa.keep_tokens(pa.CachePools([x], head_major=hm), *d[:4], ref_counts=d[4])
    assert ref.keep([pool], tables, lens, starts, kept, refs, bs, hm) == set()
    assert pa.take_device_error() == 0
    for got, want in zip((d[0], d[1], d[4]), (tables, lens, refs)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(x.view(torch.int16).cpu().numpy().view(np.uint16), pool)
