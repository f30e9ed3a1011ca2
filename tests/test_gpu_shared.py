"""Decode over shared prefixes against attention in 64 bits.

Tolerance, element by element. With p the exact softmax weights, o = sum p v and
A = sum p |v|: the weights are rounded to bf16 before the second product (at
most 2^-8 of each), which moves the numerator by at most 2^-8 A; the sum of the
weights is taken of the rounded or of the exact ones, which moves the quotient
by at most 2^-8 |o|; the result is rounded to bf16, 2^-8 |o| at most. What is
computed in fp32 (scores of 128 terms, sums over at most 10^5 tokens in tiles,
2^x to 2^-22) is far below a tenth of that. So |got - o| <= 1.1 * 2^-8 (A + 2 |o|).
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_255_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib(pa_lib):
    return pa_lib


def reference(q, k, v, tables, lens, scale, bs, hm):
    """(o, A) in 64 bits from each sequence's own table."""
    S, Hq, _ = q.shape
    Hkv = k.shape[1] if hm else k.shape[2]
    o = torch.zeros(S, Hq, D, dtype=torch.float64, device=q.device)
    A = torch.zeros_like(o)
    for s, n in enumerate(lens.tolist()):
        n = min(max(n, 0), tables.shape[1] * bs)
        if n == 0:
            continue
        blocks = tables[s, :-(-n // bs)].long()
        bad = (blocks < 0) | (blocks >= k.shape[0])
        K, V = (x[blocks.clamp(0, k.shape[0] - 1)] for x in (k, v))
        K, V = (torch.where(bad[:, None, None, None], 0, x) for x in (K, V))
        if hm:
            K, V = K.transpose(1, 2), V.transpose(1, 2)
        K, V = (x.reshape(-1, Hkv, D)[:n].transpose(0, 1).double() for x in (K, V))
        p = torch.softmax(q[s].double().view(Hkv, -1, D) @ K.transpose(1, 2) * scale, -1)
        o[s], A[s] = (p @ V).reshape(Hq, D), (p @ V.abs()).reshape(Hq, D)
    return o, A


class Batch:
    """Groups of sequences over a pool in which everything that no sequence sees
    is NaN, and table entries past a sequence's blocks are no block ids."""

    def __init__(self, sizes, prefix, own, Hq=16, Hkv=8, bs=16, hm=False, seed=0, lens=None, pad=(0, 0)):
        """`own`: tokens of every sequence after its prefix; `lens` overrides
        lengths ({sequence: tokens}); `pad`: sequences before and after the groups."""
        rng = np.random.default_rng(seed)
        S = pad[0] + sum(sizes) + pad[1]
        starts = pad[0] + np.concatenate([[0], np.cumsum(sizes)])
        group = np.full(S, -1)
        for g in range(len(sizes)):
            group[starts[g]:starts[g + 1]] = g
        L = np.array([own[i % len(own)] + (prefix[g] * bs if g >= 0 else 0) for i, g in enumerate(group)])
        for i, n in (lens or {}).items():
            L[i] = n
        nb = -(-L // bs)
        width = max(1, int(nb.max()))
        total = int(sum(prefix)) + int(nb.sum())
        NB = total + 3
        ids = list(1 + rng.permutation(NB - 1))
        pre = [[ids.pop() for _ in range(p)] for p in prefix]
        tables = np.full((S, width), NB + 5, np.int32)
        for s in range(S):
            for j in range(nb[s]):
                shared = group[s] >= 0 and j < prefix[group[s]]
                tables[s, j] = pre[group[s]][j] if shared else ids.pop()
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        kv = torch.randn(2, NB, bs, Hkv, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        seen = np.zeros((NB, bs), bool)
        for s in range(S):
            for j in range(nb[s]):
                seen[tables[s, j], :min(bs, L[s] - j * bs)] = True
        kv[:, ~torch.from_numpy(seen).cuda()] = float("nan")
        if hm:
            kv = kv.transpose(2, 3).contiguous()
        self.k, self.v = kv[0], kv[1]
        self.q = torch.randn(S, Hq, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        i32 = dict(device="cuda", dtype=torch.int32)
        self.tables, self.lens = torch.tensor(tables, **i32), torch.tensor(L, **i32)
        self.starts, self.prefix = torch.tensor(starts, **i32), torch.tensor(prefix, **i32)
        self.bs, self.hm, self.scale, self.group = bs, hm, D ** -0.5, group

    def run(self, **kw):
        return pa.decode_shared(self.q, self.k, self.v, self.tables, self.lens, self.starts, self.prefix,
                                self.scale, head_major=self.hm, **kw)

    def check(self, out=None, code=0):
        inside = torch.from_numpy(self.group >= 0).cuda()
        if out is None:
            out = torch.full_like(self.q, 77.0)
            assert self.run(out=out) is out
        assert pa.take_device_error() == code
        assert (out[~inside] == 77.0).all()
        o, A = reference(self.q, self.k, self.v, self.tables, self.lens, self.scale, self.bs, self.hm)
        err = (out.double() - o).abs()[inside]
        bound = (1.1 * 2 ** -8 * (A + 2 * o.abs()))[inside]
        assert torch.isfinite(out[inside]).all()
        assert (err <= bound).all(), (err - bound).max()
        return out


@pytest.fixture(autouse=True)
def _no_error_left():
    yield
    pa.take_device_error()


HEADS = [(1, 1), (8, 8), (16, 8), (12, 4), (10, 2), (14, 2), (32, 4), (16, 1), (33, 3)]


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_heads(Hq, Hkv, hm):
    Batch([7, 3], [9, 4], [1, 16, 17, 40, 5], Hq, Hkv, hm=hm).check()


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_block_sizes(bs, hm):
    Batch([4, 1, 6], [3, 2, 1], [0, 1, bs - 1, bs, bs + 1, 3 * bs + 7], bs=bs, hm=hm).check()


@pytest.mark.parametrize("tokens", [16, 112, 128, 144, 256, 1040])
def test_prefix_lengths(tokens):
    Batch([5], [tokens // 16], [0, 1, 3, 60], 8, 2).check()


# one tile of queries, a little over one, over two, over a pair of tiles
@pytest.mark.parametrize("n,Hq,Hkv", [(2, 2, 1), (64, 4, 2), (65, 4, 2), (128, 4, 2), (129, 4, 2), (300, 4, 2),
                                      (17, 8, 1), (40, 16, 1), (257, 1, 1), (300, 2, 2)])
def test_group_sizes(n, Hq, Hkv):
    Batch([n, 3], [6, 11], [1, 2, 30], Hq, Hkv).check()


def test_one_token_and_empty_sequences():
    Batch([4, 3, 2, 2], [2, 0, 1, 5], [0, 1], lens={0: 0, 2: 0, 4: 0, 5: 1, 7: 0, 8: 0}).check()
    Batch([3], [4], [0], lens={0: 0, 1: 0, 2: 0}).check()


def test_sequences_shorter_than_their_prefix():
    # the prefix computed together ends at the shortest length, on a multiple of 16
    Batch([6], [8], [10, 0, 33], lens={1: 77, 3: 100}).check()
    Batch([6], [8], [10, 0, 33], lens={1: 3}).check()
    Batch([4], [8], [0], lens={0: 120, 1: 127, 2: 0, 3: 113}).check()


def test_groups_of_one_and_no_prefix_are_plain_decode():
    # decode's sums over other shares of the tokens: each result is within the
    # bound above, which does not depend on how the sums are split
    b = Batch([1] * 9, [4] * 9, [5, 100, 33])
    b.check()
    b.check(pa.decode(b.q, b.k, b.v, b.tables, b.lens, b.scale))
    Batch([5, 4], [0, 0], [5, 100, 33]).check()


@pytest.mark.parametrize("G", [33, 70, 200])
def test_many_groups(G):
    rng = np.random.default_rng(G)
    Batch(list(rng.integers(1, 5, G)), list(rng.integers(0, 9, G)), list(rng.integers(0, 50, 37)), 8, 2).check()


def test_more_groups_than_plan_threads():
    Batch([2, 1] * 600, [1, 2] * 600, [1, 7, 20], 2, 1).check()


def test_as_many_groups_as_allowed():
    Batch([2] * 4095 + [1], [1] * 4096, [1, 7, 0, 20], 2, 1).check()


def test_as_many_sequences_as_allowed():
    # 65535 sequences with one table row and two queries: two results
    S = 65535
    b = Batch([2], [2], [5], 2, 1)
    _, width = b.tables.shape
    o, A = reference(b.q, b.k, b.v, b.tables[:1].expand(2, -1), b.lens, b.scale, 16, False)
    odd = torch.arange(S, device="cuda") % 2
    i32 = dict(device="cuda", dtype=torch.int32)
    for starts in ([0, S], [0, 40000, S], [7, S - 9]):
        prefix = torch.full((len(starts) - 1,), 2, **i32)
        out = pa.decode_shared(b.q[odd], b.k, b.v, b.tables[:1].expand(S, width).contiguous(),
                               b.lens[:1].expand(S).contiguous(), torch.tensor(starts, **i32), prefix, b.scale)
        got = out[starts[0]:starts[-1]].double()
        want, bound = (x[odd][starts[0]:starts[-1]] for x in (o, 1.1 * 2 ** -8 * (A + 2 * o.abs())))
        assert ((got - want).abs() <= bound).all()
    assert pa.take_device_error() == 0


def test_offsets_past_32_bits():
    # 4.6 GB a pool: more elements than 32 bits count, the used blocks at its two ends
    b = Batch([30, 3], [40, 9], [30, 1, 70], 16, 8)
    n, NB = b.k.shape[0], 140001
    far = torch.arange(n, device="cuda") % 2 == 1
    place = torch.arange(n, device="cuda") + torch.where(far, NB - n, 0)
    for hm in (False, True):
        big = []
        for x in (b.k, b.v):
            y = torch.empty(NB, *(x.transpose(1, 2) if hm else x).shape[1:], dtype=x.dtype, device="cuda")
            y[place] = x.transpose(1, 2) if hm else x
            big.append(y)
        inside = b.tables < n
        tables = torch.where(inside, place[b.tables.clamp(max=n - 1).long()], b.tables.long()).int()
        out = pa.decode_shared(b.q, *big, tables, b.lens, b.starts, b.prefix, b.scale, head_major=hm)
        b.check(out)


def test_rows_outside_the_groups_are_left():
    Batch([5, 3], [3, 7], [4, 18], pad=(2, 6)).check()
    b = Batch([5, 3], [3, 7], [4, 18], pad=(0, 3))
    b.starts.fill_(4)           # all groups empty
    b.group[:] = -1
    out = torch.full_like(b.q, 77.0)
    b.run(out=out)
    assert pa.take_device_error() == 0 and (out == 77.0).all()


def test_long_prefix_for_few_and_many():
    Batch([3], [1300], [9, 400], 16, 8).check()
    Batch([50, 2], [400, 900], [9, 130], 32, 4).check()


@pytest.mark.parametrize("n,blocks", [(128, 1000), (20, 700), (20, 701), (20, 3000), (9, 2999)])
def test_many_key_tiles_per_share(n, blocks):
    # every ring and barrier of the prefix kernel goes round many times
    for _ in range(3):
        Batch([n], [blocks], [3, 40], 16, 1).check()


# pairs of 128-row query tiles: 3 with the last half empty, 4 and 38 of one group; 2 of
# every group on the prefix kernel, with others between; 2 and 1
@pytest.mark.parametrize("sizes,blocks,Hq,Hkv,own", [
    ([80], [600], 24, 3, [60, 5]), ([256], [300], 32, 8, [400, 16]), ([256], [1100], 32, 8, [16, 700, 0]),
    ([1200], [40], 8, 1, [3, 20]), ([64, 60], [200, 333], 16, 2, [300, 1]),
    ([64, 1, 3, 60], [200, 9, 4, 333], 16, 2, [300, 1]), ([64, 20], [200, 333], 16, 2, [90, 1]),
])
def test_pairs_of_query_tiles(sizes, blocks, Hq, Hkv, own):
    Batch(sizes, blocks, own, Hq, Hkv).check()


# parts of a row spread over groups of threads and over CTAs: few rows with many
# parts, some, and many rows; prefixes packed into one unit and on the prefix kernel
@pytest.mark.parametrize("sizes,blocks,Hq,Hkv,own", [
    ([4], 1000, 16, 8, [3, 90]), ([2], 2500, 2, 1, [1, 700]), ([3, 2], 700, 8, 2, [3000, 20]),
    ([16, 16], 60, 64, 8, [200, 17]), ([20, 12], 60, 16, 8, [200, 17]), ([300], 30, 16, 2, [64, 3, 0]),
])
def test_parts_of_rows(sizes, blocks, Hq, Hkv, own):
    Batch(sizes, [blocks] * len(sizes), own, Hq, Hkv).check()


def test_a_group_larger_than_the_plan():
    Batch([1500, 700], [3, 2], [5, 20, 0, 33], 1, 1).check()


def test_long_own_part():
    Batch([4], [2], [5000, 20], 8, 4).check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-3, 3.0])
def test_scales(scale):
    b = Batch([6, 2], [9, 3], [1, 40], 16, 4)
    b.scale = scale
    b.check()


def test_values_hidden_from_some_do_not_reach_them():
    # position 100 on is seen by sequences 0 and 2, not by 1 (100 tokens)
    b = Batch([3], [8], [20], 8, 2, lens={1: 100})
    blk = b.tables[0, 100 // 16].item()
    b.v[blk, 100 % 16:] = float("inf")
    b.k[blk, 100 % 16:, 0] = float("nan")
    out = b.run()
    o, A = reference(b.q[1:2], b.k, b.v, b.tables[1:2], b.lens[1:2], b.scale, 16, False)
    assert ((out[1].double() - o[0]).abs() <= 1.1 * 2 ** -8 * (A[0] + 2 * o[0].abs())).all()
    assert not torch.isfinite(out[0]).any() and not torch.isfinite(out[2]).any()


def test_large_scores_and_equal_ones():
    b = Batch([5], [20], [30], 8, 2)
    b.q *= 30                   # one key takes nearly all the weight
    b.check()
    b.q.zero_()
    b.check()


def test_bad_blocks_read_as_zeros():
    b = Batch([4], [9], [40], 8, 2)
    b.tables[:, 3] = b.k.shape[0]
    b.check(code=4)
    b = Batch([4], [9], [40], 8, 2, hm=True)
    b.tables[:, 8] = -1
    b.tables[2, 10] = 1 << 30
    b.check(code=4)


def test_lengths_and_prefixes_past_the_table_are_clamped():
    b = Batch([3], [4], [16], 8, 2)
    b.lens[1] = 1000
    b.prefix[0] = 4
    b.check()
    b.lens[2] = -5
    b.check()
    b = Batch([3], [4], [0], 8, 2)
    b.prefix[0] = 1 << 30       # the tables agree over their whole width
    b.check()
    b.prefix[0] = -3
    b.check()


def test_starts_out_of_order_stay_within_the_buffers():
    b = Batch([3, 4, 2], [4, 2, 5], [7], 8, 2)
    for starts in ([0, 7, 3, 9], [9, 3, 0, -4], [-5, 3, 7, 900], [5, 5, 5, 5], [4, 0, 0, 9]):
        b.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        b.run()
        assert pa.take_device_error() in (0, 4)     # a table entry past a row's blocks is no block id


def test_same_bits_again_and_on_other_streams():
    b = Batch([9, 30], [40, 21], [3, 90, 250], 32, 8)
    want = b.check()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [b.run(stream=streams[i % 2]) for i in range(8)]      # two calls at once
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_buffers_for_another_stream_come_from_its_memory():
    # a buffer that the current stream has freed may still be in use there
    b = Batch([9, 30], [40, 21], [3, 90, 250], 32, 8)
    want = b.check()
    side = torch.cuda.Stream()
    ws_bytes = 3 << 20
    freed = [torch.empty_like(want), torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")]
    old = {f.data_ptr() for f in freed}
    side.wait_stream(torch.cuda.current_stream())
    del freed
    out, ws = b.run(stream=side), pa._scratch("shared", ws_bytes, want.device, side)
    assert not {out.data_ptr(), ws.data_ptr()} & old
    side.synchronize()
    assert torch.equal(out, want)


def test_several_threads_and_current_streams():
    import threading
    batches = [Batch([9, 30], [40, 21], [3, 90, 250], 32, 8), Batch([4, 20], [12, 33], [60, 5], 16, 4, hm=True)]
    want = [b.check().clone() for b in batches]
    bad = []

    def work(i, stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                for b, w in zip(batches, want):
                    if not torch.equal(b.run(), w):
                        bad.append(i)

    main = torch.cuda.current_stream()
    streams = [main, main, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i, s)) for i, s in enumerate(streams)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


def test_two_graphs_and_changed_groups():
    b, c = Batch([9, 6], [12, 5], [3, 90]), Batch([4, 4, 4], [30, 1, 8], [64, 2], 32, 4, hm=True)
    b.check(), c.check()
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
    b.check(outs[0]), c.check(outs[1])
    # other lengths, other groups of the same tables
    b.lens[:9] -= 7
    b.starts.copy_(torch.tensor([0, 4, 9], dtype=torch.int32))
    b.prefix.copy_(torch.tensor([10, 12], dtype=torch.int32))
    b.group[9:] = -1
    outs[0].fill_(77.0)
    graphs[0].replay()
    torch.cuda.synchronize()
    b.check(outs[0])


def test_own_workspace_and_refusals():
    b = Batch([3, 2], [4, 2], [9], 8, 2)
    n = pa.decode_shared_workspace_size(5, 2, 8, 2)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(b.q, 77.0)
    b.check(b.run(out=out, workspace=ws))
    with pytest.raises(pa.PagedAttnError) as e:
        b.run(workspace=ws[:-1024])
    assert e.value.status == pa.PA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        pa.decode_shared(b.q, b.k, b.v, b.tables, b.lens, b.starts[:-1], b.prefix, 0.1)
    with pytest.raises(ValueError):
        pa.decode_shared(b.q.float(), b.k, b.v, b.tables, b.lens, b.starts, b.prefix, 0.1)
    with pytest.raises(ValueError):
        pa.decode_shared_workspace_size(5, 4097, 8, 2)
    with pytest.raises(ValueError):
        pa.decode_shared_workspace_size(5, 1, 34, 2)
    empty = pa.decode_shared(b.q, b.k, b.v, b.tables, b.lens, b.starts[:1], b.prefix[:0], 0.1, out=out.fill_(77.0))
    assert (empty == 77.0).all()


def test_prompt_to_samples_and_back():
    """Prefill a prompt, fork it, let the samples grow, decode them over the
    shared prompt, free some, compact, and decode again."""
    bs, Hq, Hkv, NB, rows, n = 16, 16, 8, 120, 6, 5
    L = 300
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    i32 = dict(device="cuda", dtype=torch.int32)
    nan = lambda: torch.full((NB, bs, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16)  # noqa: E731
    k, v = nan(), nan()
    pools = pa.CachePools([k, v])
    width = 24
    tables = torch.zeros(rows, width, **i32)
    lens, refs = torch.zeros(rows, **i32), torch.zeros(NB, **i32)
    nb = -(-L // bs)
    ids = 1 + torch.randperm(NB - 1, generator=gen, device="cuda")[:nb]
    tables[0, :nb], lens[0], refs[ids] = ids.int(), L, 1
    pos = torch.arange(L, device="cuda")
    pa.store_kvcache(rnd(L, Hkv, D), rnd(L, Hkv, D), k, v, tables[0].long()[pos // bs] * bs + pos % bs)
    pa.prefill(rnd(L, Hq, D), k, v, tables[:1], lens[:1], torch.tensor([0, L], **i32), D ** -0.5)
    pa.fork_blocks(pools, tables, lens, refs, torch.zeros(n, **i32), torch.arange(1, rows, **i32))
    starts, prefix = torch.tensor([0, rows], **i32), torch.tensor([L // bs], **i32)
    for step in range(20):
        # every sequence takes a token; at a block's end it takes a block
        for r in range(rows):
            at = int(lens[r])
            if at % bs == 0:
                b = int((refs[1:] == 0).nonzero()[0]) + 1
                tables[r, at // bs], refs[b] = b, 1
        slot = tables.gather(1, (lens // bs).long()[:, None])[:, 0].long() * bs + lens.long() % bs
        lens += 1
        pa.store_kvcache(rnd(rows, Hkv, D), rnd(rows, Hkv, D), k, v, slot)
        q = rnd(rows, Hq, D)
        out = pa.decode_shared(q, k, v, tables, lens, starts, prefix, D ** -0.5)
        o, A = reference(q, k, v, tables, lens, D ** -0.5, bs, False)
        assert ((out.double() - o).abs() <= 1.1 * 2 ** -8 * (A + 2 * o.abs())).all()
    pa.free_blocks(tables, lens, refs, torch.tensor([0, 3], **i32), bs)
    _, live = pa.compact_blocks(pools, tables, lens, refs)
    assert sorted(refs.nonzero()[:, 0].tolist()) == list(range(1, int(live) + 1))
    k[int(live) + 1:] = float("nan")
    v[int(live) + 1:] = float("nan")
    want, _ = reference(q, k, v, tables, lens, D ** -0.5, bs, False)
    out2 = pa.decode_shared(q, k, v, tables, lens, starts, prefix, D ** -0.5)
    plain = pa.decode(q, k, v, tables, lens, D ** -0.5)
    for r in (1, 2, 4, 5):
        assert torch.equal(want[r], o[r])               # the same tokens as before
        bound = 1.1 * 2 ** -8 * (A[r] + 2 * o[r].abs())
        assert ((out2[r].double() - o[r]).abs() <= bound).all()
        assert ((plain[r].double() - o[r]).abs() <= bound).all()
    assert not out2[0].any() and not out2[3].any()
    assert pa.take_device_error() == 0
