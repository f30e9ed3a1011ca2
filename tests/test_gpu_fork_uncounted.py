"""Forks of rows whose owned entries name blocks that nobody counts. Such a
block is free, so the call may hand it to another fork: an entry that names it
is passed on, never copied from, and the counts do not depend on which thread
comes first. Expected values are written out, or follow from a loop over the
forks in order."""
import numpy as np
import pytest
import torch

from paged_kv_cache_255_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
BS = 16


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def run(tables, lens, refs, parents, children, head_major=False, pools=2):
    """(tables, lens, refs, pools before, pools after, code) of one call."""
    rng = np.random.default_rng(len(refs))
    shape = (len(refs), 2, BS, 128) if head_major else (len(refs), BS, 2, 128)
    before = [rng.integers(0, 1 << 15, size=shape, dtype=np.int16) for _ in range(pools)]
    dev = [torch.from_numpy(b.copy()).cuda().view(torch.bfloat16) for b in before]
    t, n, r = ints(tables), ints(lens), ints(refs)
    pa.take_device_error()
    pa.fork_blocks(pa.CachePools(dev, head_major=head_major), t, n, r, ints(parents), ints(children))
    code = pa.take_device_error()
    after = [d.view(torch.int16).cpu().numpy() for d in dev]
    return t.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy(), before, after, code


@pytest.mark.parametrize("head_major", [False, True])
def test_an_uncounted_last_block_is_passed_on(head_major):
    # row 0 owns blocks 5 and 2, 20 tokens; nobody counts block 2
    refs = [0, 1, 0, 1, 0, 1, 0]
    t, n, r, before, after, code = run([[5, 2], [0, 0]], [20, 0], refs, [0], [1], head_major)
    assert t.tolist() == [[5, 2], [5, 2]] and n.tolist() == [20, 20]
    assert r.tolist() == [0, 1, 1, 1, 0, 2, 0] and code == 5
    assert all(np.array_equal(b, a) for b, a in zip(before, after))


@pytest.mark.parametrize("head_major", [False, True])
def test_an_uncounted_last_block_is_handed_out_once(head_major):
    # block 2, row 0's uncounted last one, is the lowest free: row 3 gets it for row 1's block 3
    refs = [0, 1, 0, 1, 0, 1, 0]
    t, n, r, before, after, code = run([[5, 2], [3, 0], [0, 0], [0, 0]], [20, 9, 0, 0], refs, [0, 1], [2, 3],
                                       head_major)
    assert t.tolist() == [[5, 2], [3, 0], [5, 2], [2, 0]] and n.tolist() == [20, 9, 20, 9]
    assert r.tolist() == [0, 1, 2, 1, 0, 2, 0] and code == 5
    for b, a in zip(before, after):
        want = b.copy()
        if head_major:
            want[2, :, :9] = b[3, :, :9]
        else:
            want[2, :9] = b[3, :9]
        assert np.array_equal(a, want)


def test_counts_of_blocks_that_are_named_and_handed_out():
    # block 1 is a full block of row 0 and uncounted; rows 3 .. take 1, 2, 4 for row 1's block 3
    refs = [0, 0, 0, 1, 0, 0, 0, 0]
    t, n, r, _, _, code = run([[1, 0], [3, 0]] + [[0, 0]] * 5, [16, 7] + [0] * 5, refs, [1, 0, 1, 0, 1],
                              [2, 3, 4, 5, 6])
    assert t.tolist() == [[1, 0], [3, 0], [1, 0], [1, 0], [2, 0], [1, 0], [4, 0]]
    assert n.tolist() == [16, 7, 7, 16, 7, 16, 7]
    assert r.tolist() == [0, 3, 1, 1, 1, 0, 0, 0] and code in (0, 5)
    # no fork that needs a block: the entry is passed on and recorded
    _, _, r, _, _, code = run([[1, 0], [0, 0]], [16, 0], refs, [0], [1])
    assert r.tolist() == [0, 1, 0, 1, 0, 0, 0, 0] and code == 5


@pytest.mark.parametrize("NB", [3000, 20000])
def test_many_forks_of_rows_that_are_half_uncounted(NB):
    """200 children of 40 rows, on the plan for small pools and for large ones,
    again and again: the result of the loop below each time."""
    rng = np.random.default_rng(NB)
    rows, width, kids = 40, 6, 200
    lens = np.concatenate([rng.integers(1, width * BS + 1, rows), np.zeros(kids, int)])
    tables = np.zeros((rows + kids, width), int)
    refs = rng.integers(0, 2, NB)
    refs[0] = 0
    low = 1 + rng.permutation(400)[:rows * width]            # among the lowest free blocks
    for s in range(rows):
        for j in range(-(-lens[s] // BS)):
            tables[s, j] = low[s * width + j]
    parents, children = rng.integers(0, rows, kids), rows + rng.permutation(kids)
    # the loop: every new block first, then the entries passed on
    t, n, r = tables.copy(), lens.copy(), refs.copy()
    free = iter(np.nonzero(refs[1:] == 0)[0] + 1)
    new = {}
    for i, p in enumerate(parents):
        if lens[p] % BS and refs[tables[p, lens[p] // BS]] > 0:
            new[i] = next(free)
            r[new[i]] = 1
    for i, (p, c) in enumerate(zip(parents, children)):
        n[c] = lens[p]
        for j in range(-(-lens[p] // BS)):
            b = tables[p, j]
            if i in new and j == lens[p] // BS:
                b = new[i]
            else:
                r[b] += 1
            t[c, j] = b
    assert set(new.values()) & set(tables[:rows].ravel())    # some named blocks are handed out
    for _ in range(10):
        gt, gn, gr, before, after, code = run(tables, lens, refs, parents, children, pools=1)
        assert np.array_equal(gt, t) and np.array_equal(gn, n) and np.array_equal(gr, r) and code == 5
        want = before[0].copy()
        for i, b in new.items():
            used = lens[parents[i]] % BS
            want[b, :used] = before[0][tables[parents[i], lens[parents[i]] // BS], :used]
        assert np.array_equal(after[0], want)
