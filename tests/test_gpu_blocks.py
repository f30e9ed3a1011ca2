"""Block operations on the GPU against the plain model: every table, length,
count and pool bit by bit (nothing here is rounded), with consistent tables and
with every kind of entry the contract names."""
import numpy as np
import pytest
import torch

import blocks_ref as ref
from paged_kv_cache_255_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


class State:
    """One set of tables, counts and pools, twice: for the model and on the GPU."""

    def __init__(self, tables, lens, refs, bs, Hkv=2, pools=2, head_major=False, seed=0):
        rng = np.random.default_rng(seed + 100)
        NB = refs.shape[0]
        shape = (NB, Hkv, bs, 128) if head_major else (NB, bs, Hkv, 128)
        # every bit pattern, NaN and infinities among them
        self.pools = [rng.integers(0, 1 << 16, size=shape, dtype=np.uint16) for _ in range(pools)]
        self.tables, self.lens, self.refs, self.bs, self.hm = tables, lens, refs, bs, head_major
        self.d_tables, self.d_lens, self.d_refs = (torch.from_numpy(x.copy()).cuda()
                                                   for x in (tables, lens, refs))
        self.d_pools = [torch.from_numpy(p.view(np.int16).copy()).cuda().view(torch.bfloat16)
                        for p in self.pools]
        self.handle = pa.CachePools(self.d_pools, head_major=head_major)
        assert pa.take_device_error() >= 0      # clear what an earlier test left

    def fork(self, parents, children):
        codes = ref.fork(self.pools, self.tables, self.lens, self.refs, parents, children, self.bs, self.hm)
        pa.fork_blocks(self.handle, self.d_tables, self.d_lens, self.d_refs, ints(parents), ints(children))
        self.check(codes)

    def free(self, rows):
        codes = ref.free(self.tables, self.lens, self.refs, rows, self.bs)
        pa.free_blocks(self.d_tables, self.d_lens, self.d_refs, ints(rows), self.bs)
        self.check(codes)

    def compact(self):
        codes, remap, n = ref.compact(self.pools, self.tables, self.lens, self.refs, self.bs)
        d_remap, d_n = pa.compact_blocks(self.handle, self.d_tables, self.d_lens, self.d_refs)
        assert np.array_equal(d_remap.cpu().numpy(), remap) and d_n.item() == n
        # a block that became free holds nothing in particular
        self.check(codes, pool_ids=np.r_[0:n + 1])
        for p, d in zip(self.pools, self.d_pools):
            p[n + 1:] = bits(d)[n + 1:]

    def copy(self, pairs):
        codes = ref.copy(self.pools, pairs)
        pa.copy_blocks(self.handle, ints(pairs).view(-1, 2))
        self.check(codes)

    def check(self, codes, pool_ids=slice(None)):
        assert pa.take_device_error() == min(codes, default=0)
        assert np.array_equal(self.d_tables.cpu().numpy(), self.tables)
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        for p, d in zip(self.pools, self.d_pools):
            assert np.array_equal(bits(d)[pool_ids], p[pool_ids])


I32 = dict(dtype=torch.int32, device="cuda")


def ints(x):
    return torch.tensor(np.asarray(x, np.int32).reshape(-1), device="cuda")


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def drawn(seed, rows, width, bs, NB, shared=0, spare=0, lens=None, **kw):
    rng = np.random.default_rng(seed)
    return State(*ref.draw(rng, rows, width, bs, NB, lens=lens, shared=shared, spare=spare), bs,
                 seed=seed, **kw), rng


# -- copy ------------------------------------------------------------------------------

@pytest.mark.parametrize("bs,Hkv,pools,NB,n", [
    (16, 1, 1, 3, 1), (16, 8, 2, 40, 19), (32, 3, 4, 21, 10), (64, 5, 2, 9, 4), (256, 2, 3, 6, 2),
    (16, 1, 2, 4001, 2000),
])
def test_copy(bs, Hkv, pools, NB, n):
    s, rng = drawn(1, 1, 1, bs, NB, Hkv=Hkv, pools=pools)
    ids = rng.permutation(NB)[:2 * n].reshape(-1, 2)
    s.copy(ids)


def test_copy_skips_and_reports():
    s, _ = drawn(2, 1, 1, 16, 12)
    s.copy([[1, 2], [-1, 5], [6, -1], [7, 7], [3, 4], [-1, -1]])
    s.copy([[1, 12], [2, 3]])
    s.copy([[12, 4], [-2, 5], [6, -7], [2 ** 31 - 1, 8], [9, 10]])
    s.copy(np.zeros((0, 2)))


def test_copy_to_more_pools_than_one_launch_takes():
    s, _ = drawn(3, 1, 1, 16, 5, Hkv=1, pools=67)
    s.copy([[1, 3], [4, 2]])


def test_fork_and_compact_more_pools_than_one_launch_takes():
    s, _ = drawn(4, 3, 3, 16, 30, lens=[40, 16, 33], spare=4, Hkv=1, pools=67)
    s.fork([0, 2, 0], [4, 5, 6])
    s.free([0, 1])
    s.compact()


def test_offsets_past_32_bits():
    # 4.6 GB a pool: more elements than 32 bits count, the used blocks at its two ends
    NB, bs, Hkv = 140001, 16, 8
    pool = torch.empty(NB, bs, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    handle = pa.CachePools([pool])
    near, far = (torch.randint(-30000, 30000, (bs, Hkv, 128), dtype=torch.int16, device="cuda") for _ in range(2))
    pool[3], pool[NB - 1] = near.view(torch.bfloat16), far.view(torch.bfloat16)
    same = lambda b, x: torch.equal(pool[b].view(torch.int16), x)  # noqa: E731
    pa.copy_blocks(handle, ints([3, NB - 2, NB - 1, 5]).view(2, 2))
    assert same(NB - 2, near) and same(5, far)
    tables, lens, refs = torch.zeros(4, 3, **I32), torch.zeros(4, **I32), torch.zeros(NB, **I32)
    tables[0, 0], lens[0], refs[NB - 1] = NB - 1, 9, 1
    refs[1:NB - 1] = 1
    refs[NB - 3] = 0                                    # the only free block
    pa.fork_blocks(handle, tables, lens, refs, ints([0]), ints([2]))
    assert tables[2, 0].item() == NB - 3 and torch.equal(pool[NB - 3, :9].view(torch.int16), far[:9])
    pool[NB - 3] = near.view(torch.bfloat16)
    refs[1:NB - 3] = 0
    refs[NB - 2] = 0
    remap, live = pa.compact_blocks(handle, tables, lens, refs)
    assert live.item() == 2 and tables[0, 0].item() == 2 and tables[2, 0].item() == 1
    assert same(1, near) and same(2, far) and remap[NB - 1].item() == 2
    assert pa.take_device_error() == 0


def test_a_source_may_be_copied_twice():
    s, _ = drawn(4, 1, 1, 16, 8)
    s.copy([[1, 2], [1, 3], [1, 4]])


# -- fork ------------------------------------------------------------------------------

@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("bs,Hkv,lens", [
    (16, 8, [1, 15, 16, 17, 33]), (32, 1, [31, 32, 64, 1, 0]), (64, 3, [63, 65, 128, 5, 100]),
    (256, 2, [255, 257, 512, 300, 1]),
])
def test_fork(bs, Hkv, lens, head_major):
    s, _ = drawn(5, 5, 4, bs, 40, lens=lens, spare=9, Hkv=Hkv, head_major=head_major)
    s.fork([0, 1, 2, 3, 4, 0, 0, 3], [5, 6, 7, 8, 9, 10, 11, 12])
    s.fork([5], [13])           # a fork of a fork


def test_fork_of_shared_and_long_rows():
    s, _ = drawn(6, 3, 300, 16, 1200, lens=[4799, 4800, 37], shared=100, spare=64)
    s.fork([0, 1, 2] * 21, list(range(3, 66)))


def test_fork_takes_the_lowest_free_blocks_in_order():
    s, _ = drawn(7, 4, 3, 16, 600, lens=[17, 30, 16, 47], spare=4)
    free = [b for b in range(1, 600) if s.refs[b] == 0]
    s.fork([3, 2, 1, 0], [7, 6, 5, 4])
    # row 6 copies a full last block's row and takes none
    assert [s.tables[7, 2], s.tables[5, 1], s.tables[4, 1]] == free[:3]


def test_fork_refusals():
    s, _ = drawn(8, 4, 3, 16, 30, lens=[20, 40, 0, 9], spare=5)
    s.fork([0, 0, 0, 1], [4, 4, 1, 5])              # a child twice; a child that is not empty
    s.fork([-1, 0, -1], [6, -1, -1])                # unused places
    s.fork([-1, 3], [6, 6])                         # and one does not take the child
    s.fork([9, 0, -5, 2], [7, 9, 7, -3])            # rows out of range
    s.fork([2, 1], [7, 8])                          # an empty parent gives an empty child
    s.fork([3], [3])                                # a row onto itself


def test_fork_with_too_few_free_blocks():
    rng = np.random.default_rng(9)
    tables, lens, refs = ref.draw(rng, 3, 3, 16, 10, lens=[20, 32, 35], spare=6)
    s = State(tables, lens, refs, 16)
    assert (s.refs[1:] == 0).sum() == 2
    s.fork([0, 1, 2, 0, 1, 2], [3, 4, 5, 6, 7, 8])  # 0 and 2 get one, the later ones none; 1 needs none
    assert list(s.lens[3:]) == [20, 32, 35, 0, 32, 0]


def test_fork_passes_on_null_and_bad_entries():
    tables = np.array([[1, 0, 2], [3, 99, 4], [-1, 5, 0], [6, 15, 50], [0, 0, 0], [0, 0, 0], [0, 0, 0],
                       [0, 0, 0]], np.int32)
    lens = np.array([48, 40, 33, 41, 0, 0, 0, -4], np.int32)
    refs = np.zeros(20, np.int32)
    refs[[1, 2, 3, 4, 5, 6]] = 1                    # 15 is owned by row 3 but not counted
    s = State(tables, lens, refs, 16)
    s.fork([0], [4])
    s.fork([1, 2], [5, 6])
    s.fork([3], [7])


def test_lengths_past_the_table_are_clamped():
    s, _ = drawn(10, 2, 2, 16, 20, lens=[32, 20], spare=3)
    s.lens[0] = 1000
    s.d_lens[0] = 1000
    s.fork([0], [2])
    assert s.lens[2] == 32
    s.free([0])


# -- free -------------------------------------------------------------------------------

@pytest.mark.parametrize("bs,width,NB", [(16, 1, 10), (16, 700, 3000), (256, 5, 60)])
def test_free(bs, width, NB):
    s, rng = drawn(11, 4, width, bs, NB, shared=width // 2, spare=1)
    s.free([2, 0])
    s.free([4, -1, 1, 0])        # an empty row, an unused place, a freed row
    s.free([3])
    assert not s.refs.any()


def test_free_reports_and_keeps_counts_from_going_below_zero():
    tables = np.array([[1, 1, 2], [2, 30, 0], [-4, 3, 3], [3, 3, 3]], np.int32)
    lens = np.array([48, 48, 48, 48], np.int32)
    refs = np.zeros(20, np.int32)
    refs[[1, 2, 3]] = [2, 1, 4]
    s = State(tables, lens, refs, 16)
    s.free([0])
    s.free([1])                  # 2 has no reference left, 30 is no block, 0 is the null block
    s.free([2, 3, 7, -2])        # five entries, four references; rows out of range


def test_a_row_listed_twice_is_freed_once():
    s, _ = drawn(12, 3, 40, 16, 200, shared=10)
    s.free([1, 1, 1, 0, 1])


# -- compact ------------------------------------------------------------------------------

@pytest.mark.parametrize("bs,Hkv,rows,width,NB,shared", [
    (16, 8, 4, 5, 64, 2), (32, 1, 1, 1, 3, 0), (16, 2, 6, 60, 3000, 10), (256, 3, 2, 3, 30, 0),
    (16, 1, 40, 30, 1300, 0),
])
def test_compact(bs, Hkv, rows, width, NB, shared):
    s, rng = drawn(13, rows, width, bs, NB, shared=shared, Hkv=Hkv, pools=3)
    s.free(list(range(0, rows, 2))[:max(1, rows // 2)] if rows > 1 else [])
    s.compact()
    s.compact()                  # now nothing moves
    s.free(list(range(rows)))
    s.compact()                  # nothing is left


def test_compact_edges():
    s = State(np.zeros((0, 4), np.int32), np.zeros(0, np.int32), np.array([5, 0, 3, 0, 1], np.int32), 16)
    s.compact()                  # blocks counted outside any table; the null block's count is not looked at
    s = State(np.zeros((2, 4), np.int32), np.zeros(2, np.int32), np.zeros(1, np.int32), 16)
    s.compact()                  # a pool of the null block alone
    full = np.arange(1, 9, dtype=np.int32).reshape(2, 4)
    s = State(full[:, ::-1].copy(), np.array([64, 64], np.int32), np.r_[0, np.ones(8, np.int32)].astype(np.int32), 16)
    s.compact()                  # no free block at all


def test_compact_leaves_and_reports_bad_entries():
    tables = np.array([[9, 0, 40], [-3, 8, 6]], np.int32)
    refs = np.zeros(12, np.int32)
    refs[[8, 9, 11]] = 1         # 6 is not counted, 11 stands in no table
    s = State(tables, np.array([48, 48], np.int32), refs, 16)
    s.compact()
    assert s.tables[0, 0] == 2 and s.tables[1, 1] == 1


# -- together, on streams and in graphs ----------------------------------------------------

@pytest.mark.parametrize("seed", range(6))
def test_a_run_of_operations(seed):
    rng = np.random.default_rng(seed + 50)
    bs = int(rng.choice([16, 32, 64]))
    s, _ = drawn(seed + 50, 6, 5, bs, 70, shared=int(rng.integers(0, 3)), spare=14,
                 Hkv=int(rng.integers(1, 4)), head_major=bool(seed % 2))
    for _ in range(12):
        op = rng.integers(0, 3)
        live, empty = np.nonzero(s.lens > 0)[0], np.nonzero(s.lens <= 0)[0]
        if op == 0 and len(live) and len(empty):
            n = int(rng.integers(1, len(empty) + 1))
            s.fork(rng.choice(live, n), rng.permutation(empty)[:n])
        elif op == 1 and len(live):
            s.free(rng.permutation(live)[:int(rng.integers(1, len(live) + 1))])
        else:
            s.compact()
        assert np.array_equal(s.refs, ref.counts(s.tables, s.lens, 70, bs))


def test_fork_and_free_in_a_graph():
    s, _ = drawn(60, 3, 6, 16, 80, lens=[90, 33, 64], spare=6)
    parents, children, gone = ints([0, 1, 2, 0]), ints([3, 4, 5, 6]), ints([0, 4])
    pa.free_blocks(s.d_tables, s.d_lens, s.d_refs, ints([-1]), 16)      # loaded before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.fork_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, parents, children)
        pa.free_blocks(s.d_tables, s.d_lens, s.d_refs, gone, 16)
        pa.compact_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs)
    s.check(set())               # a capture runs nothing
    g.replay()
    ref.fork(s.pools, s.tables, s.lens, s.refs, [0, 1, 2, 0], [3, 4, 5, 6], 16)
    ref.free(s.tables, s.lens, s.refs, [0, 4], 16)
    _, _, n = ref.compact(s.pools, s.tables, s.lens, s.refs, 16)
    s.check(set(), pool_ids=np.r_[0:n + 1])
    # other rows on the second replay
    parents.copy_(ints([1, -1, 2, -1]))
    children.copy_(ints([0, 1, 4, 2]))
    gone.copy_(ints([6, -1]))
    g.replay()
    ref.fork(s.pools, s.tables, s.lens, s.refs, [1, -1, 2, -1], [0, 1, 4, 2], 16)
    ref.free(s.tables, s.lens, s.refs, [6, -1], 16)
    codes, _, n = ref.compact(s.pools, s.tables, s.lens, s.refs, 16)
    torch.cuda.synchronize()
    assert pa.take_device_error() == min(codes, default=0)
    assert np.array_equal(s.d_tables.cpu().numpy(), s.tables)
    assert np.array_equal(s.d_refs.cpu().numpy(), s.refs)


def test_another_stream():
    s, _ = drawn(61, 3, 6, 16, 80, lens=[90, 33, 64], spare=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.fork([0, 1], [3, 4])
    pa.fork_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, ints([2]), ints([5]), stream=side)
    side.synchronize()
    s.check(ref.fork(s.pools, s.tables, s.lens, s.refs, [2], [5], 16))


def test_outputs_for_another_stream_come_from_its_memory():
    # a buffer that the current stream has freed may still be in use there
    s, _ = drawn(63, 3, 6, 16, 80, lens=[90, 33, 64], spare=6)
    side = torch.cuda.Stream()
    n = s.d_refs.shape[0]
    freed = [torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")]
    old = {f.data_ptr() for f in freed}
    side.wait_stream(torch.cuda.current_stream())
    del freed
    remap, live = pa.compact_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, stream=side)
    assert not {remap.data_ptr(), live.data_ptr()} & old
    side.synchronize()
    codes, want, k = ref.compact(s.pools, s.tables, s.lens, s.refs, s.bs)
    assert np.array_equal(remap.cpu().numpy(), want) and live.item() == k
    s.check(codes, pool_ids=np.r_[0:k + 1])


@pytest.mark.parametrize("remap,num_live", [((79,), (1,)), ((80, 1), (1,)), ((80,), ()), ((80,), (2,))])
def test_compact_refuses_outputs_of_another_shape(remap, num_live):
    s, _ = drawn(64, 3, 6, 16, 80, lens=[90, 33, 64], spare=6)
    with pytest.raises(ValueError):
        pa.compact_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs,
                          remap=torch.empty(remap, dtype=torch.int32, device="cuda"),
                          num_live=torch.empty(num_live, dtype=torch.int32, device="cuda"))
    s.check(set())


def test_binding_refusals():
    s, _ = drawn(62, 2, 3, 16, 20, spare=1)
    i = ints([0])
    with pytest.raises(ValueError):
        pa.CachePools([s.d_pools[0], s.d_pools[0]])                     # a pool twice
    with pytest.raises(ValueError):
        pa.CachePools([s.d_pools[0], s.d_pools[1][:5]])                 # two shapes
    with pytest.raises(ValueError):
        pa.copy_blocks(s.handle, i)
    with pytest.raises(ValueError):
        pa.fork_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, i[0], i[0])
    with pytest.raises(ValueError):
        pa.fork_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, i, ints([0, 1]))
    with pytest.raises(ValueError):
        pa.fork_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, ints([0] * 4), ints([1] * 4))
    with pytest.raises(ValueError):
        pa.fork_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs[1:], i, i)
    with pytest.raises(ValueError):
        pa.free_blocks(s.d_tables, s.d_lens[:1], s.d_refs, i, 16)
    with pytest.raises(ValueError):
        pa.free_blocks(s.d_tables.t(), s.d_lens, s.d_refs, i, 16)
    with pytest.raises(pa.PagedAttnError):
        pa.free_blocks(s.d_tables, s.d_lens, s.d_refs, i, 24)
    with pytest.raises(ValueError):
        pa.compact_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs, remap=i)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.compact_blocks(s.handle, s.d_tables, s.d_lens, s.d_refs,
                          workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pa.PA_ERR_WORKSPACE
    s.check(set())


def test_a_pool_past_the_small_plan():
    # 20000 blocks: more counts than the plan with few warps takes
    s, _ = drawn(70, 4, 300, 16, 20000, lens=[4000, 4799, 33, 4800], shared=3, spare=5, Hkv=1, pools=1)
    s.fork([0, 1, 2, 3, 0], [4, 5, 6, 7, 8])
    s.free([1, 3, 4])
    s.compact()
