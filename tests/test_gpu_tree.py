"""Decode over trees of drafted tokens against attention in 64 bits (tree_ref), by the
bounds of tile_codes: weights and outputs rounded to bf16."""
import time

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


def random_tree(rng, n):
    return [int(rng.integers(max(0, j // 3), j)) if j else -1 for j in range(n)]


class Batch:
    """Sequences of base[i] tokens and a tree of nodes[i] over a pool in which everything
    that no row sees is NaN, and table entries past a sequence's blocks are no block ids.

    masks: "tree", "random" (any bits), or a function (rng, n) -> whole numbers."""

    def __init__(self, base, nodes, Hq=16, Hkv=8, bs=16, hm=False, seed=0, masks="tree", pad=(0, 0), mask_words=None,
                 scale=D ** -0.5):
        rng = np.random.default_rng(seed)
        base, nodes = np.array(base), np.array(nodes)
        S, L = len(base), np.array(base) + np.array(nodes)
        bits = []
        for n in nodes:
            if masks == "tree":
                bits += ref.ancestors(random_tree(rng, n))
            elif masks == "random":
                bits += [sum(int(x) << i for i, x in enumerate(rng.integers(0, 2, n))) for _ in range(n)]
            else:
                bits += masks(rng, int(n))
        self.words = mask_words or max(1, -(-int(nodes.max()) // 64))
        real = ref.words(bits, self.words)
        T = pad[0] + len(bits) + pad[1]
        mask = np.full((T, self.words), -1, np.int64)
        mask[pad[0]:pad[0] + len(bits)] = real
        starts = pad[0] + np.concatenate([[0], np.cumsum(nodes)])
        nb = -(-L // bs)
        width, total = max(1, int(nb.max())), int(nb.sum())
        NB = total + 3
        ids = list(1 + rng.permutation(NB - 1))
        tables = np.full((S, width), NB + 5, np.int32)
        seen = np.zeros((NB, bs), bool)
        for s in range(S):
            union = 0
            for i in range(nodes[s]):
                union |= bits[int(starts[s]) - pad[0] + i]
            for j in range(nb[s]):
                tables[s, j] = ids.pop()
                for r in range(min(bs, L[s] - j * bs)):
                    t = int(j * bs + r - base[s])
                    seen[tables[s, j], r] = nodes[s] > 0 and (t < 0 or (union >> t & 1 and t < 64 * self.words))
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        kv = torch.randn(2, NB, bs, Hkv, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        kv[:, ~torch.from_numpy(seen).cuda()] = float("nan")
        if hm:
            kv = kv.transpose(2, 3).contiguous()
        self.k, self.v = kv[0], kv[1]
        self.q = torch.randn(T, Hq, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        self.q[:pad[0]] = float("nan")
        self.q[T - pad[1]:] = float("nan")
        i32 = dict(device="cuda", dtype=torch.int32)
        self.tables, self.lens, self.starts = (torch.tensor(x, **i32) for x in (tables, L, starts))
        self.mask, self.bs, self.hm, self.scale, self.pad = torch.from_numpy(mask).cuda(), bs, hm, scale, pad

    def run(self, **kw):
        return pa.decode_tree(self.q, self.k, self.v, self.tables, self.lens, self.starts, self.mask, self.scale,
                              head_major=self.hm, **kw)

    def reference(self):
        return ref.attention(self.q, self.k, self.v, self.tables, self.lens, self.starts, self.mask, self.scale,
                             self.bs, self.hm)

    def inside(self):
        T = self.q.shape[0]
        lo, hi = (min(max(int(x), 0), T) for x in (self.starts[0], self.starts[-1]))
        i = torch.arange(T, device="cuda")
        return (i >= lo) & (i < hi)

    def check(self, out=None, code=0):
        if out is None:
            out = torch.full_like(self.q, 77.0)
            assert self.run(out=out) is out
        assert pa.take_device_error() == code
        inside = self.inside()
        assert (out[~inside] == 77.0).all()
        o, A = self.reference()
        err, bound = (out.double() - o).abs()[inside], tc.element_bound(o, A)[inside]
        assert torch.isfinite(out[inside]).all()
        assert (err <= bound).all(), (err - bound).max()
        empty = inside & ~A.bool().flatten(1).any(1)
        assert (out[empty] == 0).all()
        return out


HEADS = [(1, 1), (8, 8), (16, 8), (12, 4), (10, 2), (14, 2), (32, 4), (16, 1), (33, 3), (3, 1), (64, 8)]


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_heads(Hq, Hkv, hm):
    Batch([300, 0, 16, 129, 40], [7, 12, 1, 5, 0], Hq, Hkv, hm=hm).check()


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_block_sizes(bs, hm):
    Batch([0, 1, bs - 1, bs, bs + 1, 3 * bs + 7, 300], [5, 9, 1, 17, 16, 3, 33], bs=bs, hm=hm).check()


# the tree's place in the key tiles of 128: behind them, at their borders, over one
@pytest.mark.parametrize("base", [0, 1, 90, 111, 112, 120, 127, 128, 129, 255, 256, 1000])
def test_context_lengths(base):
    Batch([base, base + 3], [8, 40], 8, 2).check()


# rows: one, a tile of 128 less one, full, one more, a pair, more than a pair
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 1, 1), (63, 4, 2), (64, 4, 2), (65, 4, 2), (127, 4, 2), (128, 4, 2), (129, 4, 2),
                                      (300, 4, 2), (17, 8, 1), (40, 16, 1), (257, 1, 1), (1000, 2, 1), (1024, 1, 1)])
def test_node_counts(n, Hq, Hkv):
    Batch([200, 33], [n, 3], Hq, Hkv).check()


@pytest.mark.parametrize("masks", ["random", "chain", "self", "none", "all"])
@pytest.mark.parametrize("base", [0, 77, 700])
def test_masks(masks, base):
    f = dict(random="random", chain=lambda r, n: [(2 << i) - 1 for i in range(n)], self=lambda r, n: [1 << i for i in range(n)],
             none=lambda r, n: [0] * n, all=lambda r, n: [(1 << n) - 1] * n)[masks]
    Batch([base, base, base + 1], [33, 1, 70], 8, 4, masks=f).check()


def test_bits_past_the_tree_are_not_read():
    b = Batch([50, 9, 300], [10, 64, 33], 8, 2, mask_words=3)
    want = b.check().clone()
    for s, n in enumerate((10, 64, 33)):
        rows = slice(int(b.starts[s]), int(b.starts[s + 1]))
        for w in range(3):
            keep = max(0, min(64, n - 64 * w))
            b.mask[rows, w] |= -1 << keep if keep < 64 else 0
    assert torch.equal(b.run(), want)


def test_nodes_past_the_mask_are_not_seen():
    # 150 nodes, 64 bits: a row sees of the nodes only the first 64 at most
    Batch([30, 300], [150, 9], 8, 2, mask_words=1).check()
    Batch([30], [1024], 2, 1, mask_words=16, masks="random").check()


def test_a_chain_is_decode_multi():
    b = Batch([300, 1, 64], [4, 4, 4], 16, 8, masks=lambda r, n: [(2 << i) - 1 for i in range(n)])
    out = b.check()
    multi = pa.decode_multi(b.q.view(3, 4, 16, D), b.k, b.v, b.tables, b.lens, b.scale)
    b.check(multi.view(12, 16, D).contiguous())
    assert pa.prefill(b.q, b.k, b.v, b.tables, b.lens, b.starts, b.scale).shape == out.shape


def test_one_node_is_decode():
    b = Batch([300, 0, 64, 1023], [1, 1, 1, 1], 32, 8)
    b.check()
    b.check(pa.decode(b.q, b.k, b.v, b.tables, b.lens, b.scale))


def test_padding_rows_are_left():
    Batch([30, 300], [5, 9], pad=(3, 7)).check()
    b = Batch([30, 300], [5, 9], pad=(0, 4))
    b.starts.fill_(6)           # no sequence has nodes
    out = torch.full_like(b.q, 77.0)
    b.run(out=out)
    assert pa.take_device_error() == 0 and (out == 77.0).all()


@pytest.mark.parametrize("S", [1, 2, 100, 400, 1500])
def test_many_sequences(S):
    rng = np.random.default_rng(S)
    base, nodes = rng.integers(0, 400, S), rng.integers(0, 20, S)
    nodes[0] = 20
    Batch(base, nodes, 8, 2, seed=S).check()


def test_runs_of_sequences_without_nodes():
    base, nodes = np.full(900, 40), np.zeros(900, int)
    nodes[[3, 500, 501, 899]] = [5, 9, 1, 30]
    Batch(base, nodes, 4, 2).check()


# every tree of the same number of units: they are shared side by side, in few and many
# sequences, some without nodes or context; and more of them than SMs
@pytest.mark.parametrize("S,lo,hi,Hq,Hkv", [(1, 97, 128, 8, 1), (7, 65, 128, 8, 2), (5, 129, 192, 12, 3), (400, 65, 128, 8, 2),
                                            (800, 33, 64, 16, 2), (1, 5000, 5000, 8, 1)])
def test_units_side_by_side(S, lo, hi, Hq, Hkv):
    rng = np.random.default_rng(S + lo)
    base, nodes = rng.integers(0, 500, S), rng.integers(lo, hi + 1, S)
    if S > 1:
        nodes[rng.permutation(S)[:S // 5]] = 0
    same = int(rng.integers(1, 1 << 40)) | 1
    Batch(base, nodes, Hq, Hkv, masks=lambda r, n: [same & (1 << n) - 1] * n, mask_words=3).check()


# one unit over all SMs, units cut into two or three, more units than SMs
@pytest.mark.parametrize("base,nodes,Hq,Hkv", [
    ([40000], [5], 4, 1), ([20000], [60], 8, 1), ([9000, 5], [100, 3], 4, 1), ([3000] * 5, [33] * 5, 16, 8),
    ([1000] * 40, [12, 70] * 20, 8, 8), ([5000, 100, 2500], [64, 8, 129], 16, 2), ([2000] * 3, [300, 1, 64], 8, 4)])
def test_cuts(base, nodes, Hq, Hkv):
    b = Batch(base, nodes, Hq, Hkv)
    out = b.check()
    o, _ = b.reference()
    err = tc.row_error(out, o)
    assert (err <= tc.ROW_REL).all(), err.max()
    assert torch.equal(b.run(), out)


@pytest.mark.parametrize("base,nodes,Hq,Hkv,bs,hm", [
    (48000, 20, 16, 1, 16, False), (47990, 40, 4, 1, 64, True), (9000, 64, 16, 4, 256, False), (4000, 130, 8, 2, 16, True)])
def test_coded_keys(base, nodes, Hq, Hkv, bs, hm):
    """A lost, doubled or stale group of 16 keys shows on every row."""
    rng = np.random.default_rng(base)
    S = 3
    b = Batch([base, base - 77, 5], [nodes, nodes // 2, nodes], Hq, Hkv, bs, hm)
    code = torch.stack(tc.coded_rows(int(b.lens.max()) + 112 * Hkv, "cuda"))
    shift = 112 * torch.arange(Hkv, device="cuda")
    for x, c in ((b.k, code[0]), (b.v, code[1])):
        x.fill_(float("nan"))
        y = x.transpose(1, 2) if hm else x
        for s in range(S):
            t = torch.arange(int(b.lens[s]), device="cuda")
            y[b.tables[s].long()[t // bs], t % bs] = c[t[:, None] + shift]
    dim = torch.from_numpy(rng.integers(0, D, b.q.shape[:2])).cuda()
    b.q.zero_()
    b.q.scatter_(2, dim[..., None], 400.0)
    b.check()


def test_what_a_row_does_not_see_does_not_reach_it():
    # two branches under a root: nodes 1, 2 and 3, 4
    tree = lambda r, n: ref.ancestors([-1, 0, 1, 0, 3])     # noqa: E731
    for base in (0, 60, 126, 500):
        b = Batch([base, base], [5, 5], 8, 2, masks=tree)
        want = b.check().clone()
        at = lambda s, i: (int(b.tables[s, (base + i) // 16]), (base + i) % 16)     # noqa: E731
        blk, row = at(0, 3)
        b.v[blk, row, 0, 5] = float("inf")
        b.v[blk, row, 1, 7] = float("nan")
        b.v[blk, row, 1, 8] = float("-inf")
        b.k[at(0, 4)] = float("nan")
        out = b.run()
        assert torch.equal(out[[0, 1, 2, 5, 6, 7, 8, 9]], want[[0, 1, 2, 5, 6, 7, 8, 9]])
        # those that see node 3: its infinities and NaN and nothing else of it
        for i, other in ((3, False), (4, True)):
            assert (out[i, :4, 5] == float("inf")).all() or other
            assert out[i, 4:, 7].isnan().all()
            if other:
                assert out[i].isnan().all()         # node 4's keys
            else:
                assert (out[i, 4:, 8] == float("-inf")).all()
                rest = torch.ones(8, D, dtype=torch.bool, device="cuda")
                rest[:4, 5] = rest[4:, 7] = rest[4:, 8] = False
                assert torch.equal(out[i][rest], want[i][rest])


def test_infinities_in_a_cut_unit():
    # one long sequence over many shares: the nodes' share alone holds the infinity
    tree = lambda r, n: [1 << i for i in range(n)]      # noqa: E731
    for hm in (False, True):
        b = Batch([30000], [40], 4, 1, masks=tree, hm=hm)
        want = b.check().clone()
        t = 30000 + 33
        at = (int(b.tables[0, t // 16]), 0, t % 16) if hm else (int(b.tables[0, t // 16]), t % 16, 0)
        b.v[at][100] = float("inf")
        out = b.run()
        assert (out[33, :, 100] == float("inf")).all()
        out[33, :, 100] = want[33, :, 100]
        assert torch.equal(out, want)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-3, 3.0])
def test_scales(scale):
    Batch([100, 0, 300], [12, 7, 40], 16, 4, scale=scale, masks="random").check()


def test_large_scores_and_equal_ones():
    b = Batch([400, 3], [30, 9], 8, 2)
    b.q *= 30
    b.check()
    b.q.zero_()
    b.check()


# Scores of powers of two from key tile to key tile, up to about 400 (of 2): rows whose maximum
# grows by more than the exponent's range, by a little, or falls. 400 units of 2^-24, and what
# 128 products add, are a few 1e-5 of a weight: inside element_bound's tenth.
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("nodes,Hq,Hkv", [(40, 16, 2), (20, 16, 2), (6, 16, 2), (3, 16, 2)])
def test_maxima_that_rise_and_fall(nodes, Hq, Hkv, down):
    b = Batch([1000, 130, 700], [nodes, nodes, 1], Hq, Hkv)
    for s in range(3):
        for j in range(-(-int(b.lens[s]) // b.bs)):
            e = j * b.bs // 128 - 3
            b.k[b.tables[s, j].long()] *= 2.0 ** (1 - e if down else e)
    b.q *= 2.0 ** torch.randint(-4, 3, b.q.shape[:2], device="cuda", generator=torch.Generator("cuda").manual_seed(9))[..., None]
    b.check()


def test_bad_blocks_read_as_zeros():
    b = Batch([200, 50], [9, 40], 8, 2)
    b.tables[0, 3] = b.k.shape[0]
    b.check(code=4)
    b = Batch([200, 50], [9, 40], 8, 2, hm=True)
    b.tables[1, 4] = -1             # nodes among them
    b.tables[0, 12] = 1 << 30
    b.check(code=4)


def test_lengths_outside_the_table_and_short_of_the_nodes():
    b = Batch([120, 30], [9, 5], 8, 2)
    b.lens[1] = -5
    b.check()
    b = Batch([112, 30], [16, 5], 8, 2)
    b.lens[0] = 1000                # clamped to the table's 128
    b.check()
    # more nodes than tokens: those before the first token do not exist
    b = Batch([0, 20], [9, 30], 8, 2, masks=lambda r, n: [(1 << n) - 1] * n)
    b.lens.copy_(torch.tensor([4, 17]))
    b.check()


def test_starts_out_of_order_stay_within_the_buffers():
    b = Batch([30, 300, 20], [5, 9, 4], 8, 2)
    for starts in ([0, 7, 3, 18], [18, 3, 0, -4], [-5, 3, 7, 900], [5, 5, 5, 5], [0, 18, 0, 18]):
        b.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        b.run()
        assert pa.take_device_error() in (0, 4)


def test_offsets_past_32_bits():
    # 4.6 GB a pool: more elements than 32 bits count, the used blocks at its two ends
    b = Batch([600, 31], [33, 9], 16, 8)
    n, NB = b.k.shape[0], 140001
    far = torch.arange(n, device="cuda") % 2 == 1
    place = torch.arange(n, device="cuda") + torch.where(far, NB - n, 0)
    for hm in (False, True):
        big = []
        for x in (b.k, b.v):
            y = torch.empty(NB, *(x.transpose(1, 2) if hm else x).shape[1:], dtype=x.dtype, device="cuda")
            y[place] = x.transpose(1, 2) if hm else x
            big.append(y)
        used = b.tables < n
        tables = torch.where(used, place[b.tables.clamp(max=n - 1).long()], b.tables.long()).int()
        out = torch.full_like(b.q, 77.0)
        pa.decode_tree(b.q, *big, tables, b.lens, b.starts, b.mask, b.scale, out=out, head_major=hm)
        b.check(out)


def test_streams_threads_and_graphs():
    import threading
    b, c = Batch([3000, 90, 0], [33, 8, 4], 32, 8), Batch([40, 700], [70, 12], 16, 4, hm=True)
    want = [x.check().clone() for x in (b, c)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [b.run(stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) for o in outs)
    bad = []

    def work(i, stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                for x, w in zip((b, c), want):
                    if not torch.equal(x.run(), w):
                        bad.append(i)
    main = torch.cuda.current_stream()
    threads = [threading.Thread(target=work, args=(i, st)) for i, st in enumerate([main, main] + streams)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad
    graphs, outs = [], []
    for x in (b, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.run())
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    # other lengths, trees and starts in the captured arrays
    b.lens[0] -= 20
    b.lens[2] = 0
    b.starts.copy_(torch.tensor([0, 10, 45, 45], dtype=torch.int32))
    b.mask.fill_(-1)
    b.lens[1] = 60
    k, v = b.k, b.v
    for x in (k, v):            # nodes that nobody saw before hold NaN
        x.nan_to_num_(0.25)
    outs[0].fill_(77.0)
    graphs[0].replay()
    torch.cuda.synchronize()
    b.check(outs[0])


def test_own_workspace_and_refusals():
    b = Batch([3000, 2], [40, 2], 8, 2)
    n = pa.decode_tree_workspace_size(8, 2)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(b.q, 77.0)
    b.check(b.run(out=out, workspace=ws))
    with pytest.raises(pa.PagedAttnError) as e:
        b.run(workspace=ws[:-256])
    assert e.value.status == pa.PA_ERR_WORKSPACE
    for bad in (dict(starts=b.starts[:-1]), dict(mask=b.mask[:-1]), dict(mask=b.mask[:, 0]), dict(mask=b.mask.int()),
                dict(q=b.q.float()), dict(lens=b.lens[:-1])):
        a = dict(q=b.q, k=b.k, v=b.v, tables=b.tables, lens=b.lens, starts=b.starts, mask=b.mask)
        a.update(bad)
        with pytest.raises(ValueError):
            pa.decode_tree(*a.values(), 0.1)
    with pytest.raises(pa.PagedAttnError):
        pa.decode_tree(b.q, b.k, b.v, b.tables, b.lens, b.starts, b.mask.expand(-1, 17).contiguous(), 0.1)
    assert (pa.decode_tree(b.q, b.k, b.v, b.tables[:0], b.lens[:0], b.starts[:1], b.mask, 0.1, out=out.fill_(77.0)) == 77).all()


@pytest.mark.parametrize("base,nodes,Hq,Hkv,hm", [([20], [5], 16, 1, False), ([3000] * 4, [60] * 4, 64, 8, False),
                                                 ([900, 40, 10], [300, 8, 0], 32, 4, True)])
def test_a_held_arrival_is_reported_and_the_next_calls_are_right(base, nodes, Hq, Hkv, hm):
    b = Batch(base, nodes, Hq, Hkv, hm=hm)
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
