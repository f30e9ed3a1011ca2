"""Keeping the accepted tokens of drafts against the plain model (tree_ref.keep), bit by
bit, and a speculative step from projections to kept tokens."""
import numpy as np
import pytest
import torch

import blocks_ref
import rotary_ref
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


class State:
    def __init__(self, base, nodes, bs=16, Hkv=2, pools=2, hm=False, seed=0, spare=2):
        self.rng = rng = np.random.default_rng(seed)
        L = np.array(base) + np.array(nodes)
        nb = -(-L // bs)
        NB = 2 + int(nb.sum()) + spare
        ids = list(1 + rng.permutation(NB - 1))
        self.tables = np.zeros((len(L), max(1, int(nb.max()) + 1)), np.int32)
        for s, n in enumerate(nb):
            self.tables[s, :n] = [ids.pop() for _ in range(n)]
        self.lens, self.starts = L.astype(np.int32), np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.refs = blocks_ref.counts(self.tables, self.lens, NB, bs)
        shape = (NB, Hkv, bs, D) if hm else (NB, bs, Hkv, D)
        self.pools = [rng.integers(0, 1 << 16, size=shape, dtype=np.uint16) for _ in range(pools)]
        self.bs, self.hm, self.nodes = bs, hm, np.array(nodes)

    def paths(self, m):
        kept = np.full((len(self.lens), m), -1, np.int32)
        for s, n in enumerate(self.nodes):
            a = int(self.rng.integers(0, min(n, m) + 1))
            kept[s, :a] = np.sort(self.rng.choice(n, a, False)) if a else []
        return kept

    def keep(self, kept, counted=True, **kw):
        d = {k: torch.from_numpy(getattr(self, k).copy()).cuda() for k in ("tables", "lens", "starts", "refs")}
        d_pools = [torch.from_numpy(p.view(np.int16).copy()).cuda().view(torch.bfloat16) for p in self.pools]
        handle = pa.CachePools(d_pools, head_major=self.hm)
        pa.keep_tokens(handle, d["tables"], d["lens"], d["starts"], torch.from_numpy(kept).cuda(),
                       ref_counts=d["refs"] if counted else None, **kw)
        codes = ref.keep(self.pools, self.tables, self.lens, self.starts, kept, self.refs if counted else None, self.bs,
                         self.hm)
        torch.cuda.synchronize()
        assert pa.take_device_error() == min(codes, default=0)
        for k in ("tables", "lens", "refs"):
            assert np.array_equal(d[k].cpu().numpy(), getattr(self, k)), k
        for p, x in zip(self.pools, d_pools):
            assert np.array_equal(x.view(torch.int16).cpu().numpy().view(np.uint16), p)


@pytest.mark.parametrize("hm", [False, True])
@pytest.mark.parametrize("bs,Hkv,pools", [(16, 8, 2), (16, 1, 5), (256, 3, 4), (64, 2, 70), (32, 5, 1), (128, 8, 130)])
def test_random_paths(bs, Hkv, pools, hm):
    for seed in range(3):
        st = State([0, 5, 16, 300, 31, 40], [8, 1, 33, 60, 0, 17], bs, Hkv, pools, hm, seed)
        st.keep(st.paths(12), counted=seed != 1)


@pytest.mark.parametrize("m", [1, 7, 8, 9, 255, 256, 257, 1024])
def test_long_lists(m):
    st = State([3, 100], [1024, 700], pools=2, seed=m)
    st.keep(st.paths(m))


def test_every_path_kind():
    st = State([10] * 6, [9] * 6)
    st.keep(np.array([[-1] * 9, [0] + [-1] * 8, list(range(9)), [8] + [-1] * 8, [0, 1, 2, 7, 8, -1, -1, -1, -1],
                      [1, 3, 5, 7, -1, 2, 4, 6, 8]], np.int32))
    assert st.lens.tolist() == [10, 11, 19, 11, 15, 14]


def test_lists_that_do_not_ascend_end_there():
    for row in ([0, 0, 1], [2, 1, 3], [0, 9, 1], [0, -2, 1], [1 << 30, 0, 1], [5, 6, 6]):
        st = State([10, 20], [9, 4])
        st.keep(np.array([row, [0, 2, -1]], np.int32))


def test_drafts_that_are_none():
    st = State([10, 0, 20, 30], [9, 0, 4, 2])
    st.lens[0] = 5                  # fewer tokens than nodes: left as it is
    st.lens[2] = -3
    st.keep(st.paths(4), counted=False)
    st = State([10, 20], [9, 4])
    st.starts[:] = [-4, 9, 13]
    st.keep(np.array([[1, 2], [1, 3]], np.int32))
    st = State([10, 20], [9, 4])
    st.starts[:] = [9, 2, 6]        # decreasing
    st.keep(np.array([[1, 2], [1, 3]], np.int32))


def test_bad_entries_are_skipped_and_recorded():
    for at, bad in ((1, 0), (1, 999), (2, -7), (3, 1 << 30)):
        st = State([20, 40], [44, 9], bs=16)
        st.tables[0, at] = bad
        st.keep(np.array([[0, 5, 20, 40, 43], [0, 1, 2, 7, -1]], np.int32))
    st = State([20, 40], [44, 9], bs=16)
    st.refs[st.tables[0, 3]] = 0            # nobody counts the block that is given back
    st.keep(np.array([[0, 5], [0, -1]], np.int32))
    assert st.refs.min() == 0


def test_shared_blocks_lose_one_count():
    st = State([20, 40], [44, 9], bs=16)
    st.refs[st.tables[0, 3]] = 3
    st.keep(np.array([[0, 5], [0, -1]], np.int32))


def test_tables_alone_streams_and_graphs():
    st = State([20, 40], [44, 9])
    i32 = lambda x: torch.from_numpy(x.copy()).cuda()        # noqa: E731
    x = torch.from_numpy(st.pools[0].view(np.int16).copy()).cuda().view(torch.bfloat16)
    handle = pa.CachePools([x])
    t, ln, rf, ks, saved = i32(st.tables), i32(st.lens), i32(st.refs), i32(np.array([[0, 5], [0, 7]], np.int32)), x.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.keep_tokens(handle, t, ln, i32(st.starts), ks, ref_counts=rf, stream=side)
    side.synchronize()
    want = x.clone(), t.clone(), ln.clone(), rf.clone()
    assert pa.take_device_error() == 0
    starts = i32(st.starts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.keep_tokens(handle, t, ln, starts, ks, ref_counts=rf)
    for _ in range(2):
        x.copy_(saved), t.copy_(i32(st.tables)), ln.copy_(i32(st.lens)), rf.copy_(i32(st.refs))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((x, t, ln, rf), want))


def test_pools_past_32_bits():
    NB, bs, Hkv = 140001, 16, 8
    for hm in (False, True):
        x = torch.zeros((NB, Hkv, bs, D) if hm else (NB, bs, Hkv, D), device="cuda", dtype=torch.bfloat16)
        rows = torch.randn(6, Hkv, D, device="cuda").bfloat16()
        i32 = dict(device="cuda", dtype=torch.int32)
        table = torch.tensor([[5, NB - 1]], **i32)
        at = lambda t: ((int(table[0, t // 16]), slice(None), t % 16) if hm else (int(table[0, t // 16]), t % 16))   # noqa: E731
        for i in range(6):
            x[at(13 + i)] = rows[i]
        lens = torch.tensor([19], **i32)
        pa.keep_tokens(pa.CachePools([x], head_major=hm), table, lens, torch.tensor([0, 6], **i32),
                       torch.tensor([[1, 4, 5]], **i32))
        assert lens.item() == 16 and pa.take_device_error() == 0
        for i, k in enumerate((1, 4, 5)):
            assert torch.equal(x[at(13 + i)], rows[k])
        assert torch.equal(x[at(16)], rows[3]) and torch.equal(x[at(18)], rows[5])
        del x


@pytest.mark.parametrize("hm", [False, True])
def test_speculative_steps(hm):
    """Prompt appended with its rotation and attended; then steps of: draft a tree, append
    its nodes at the positions of their depths, attend over the tree, keep a path. After
    every step the cache holds, bit by bit, what appending the kept tokens alone would
    have left, and attention agrees with a cache that never saw a draft."""
    bs, Hq, Hkv, NB, S, n = 16, 16, 8, 100, 3, 21
    rng = np.random.default_rng(7)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()      # noqa: E731
    i32 = dict(device="cuda", dtype=torch.int32)
    shape = (NB, Hkv, bs, D) if hm else (NB, bs, Hkv, D)
    k, v, k2, v2 = (torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(4))
    R, qw, kw = pa.Rotary(128, scaling="yarn", factor=4.0, original_context=64), rnd(D), rnd(D)
    tables, refs = torch.zeros(S, 24, **i32), torch.zeros(NB, **i32)
    free = list(1 + rng.permutation(NB - 1))

    def grow(s, tokens):
        """The caller hands out blocks and counts them."""
        for e in range(-(-tokens // bs)):
            if tables[s, e] == 0:
                b = free.pop()
                tables[s, e], refs[b] = b, 1

    def slots(s, t):
        return tables[s].long()[t // bs] * bs + t % bs

    lens = torch.tensor([40, 16, 5], **i32)
    for s in range(S):
        grow(s, int(lens[s]))
    owner = torch.repeat_interleave(torch.arange(S, device="cuda"), lens.long())
    pos = torch.cat([torch.arange(int(x), device="cuda") for x in lens])
    at = torch.cat([slots(s, torch.arange(int(lens[s]), device="cuda")) for s in range(S)])
    T = len(pos)
    qkv = rnd(T, Hq + 2 * Hkv, D)
    for kc, vc in ((k, v), (k2, v2)):
        q = pa.append_kvcache(*qkv.split([Hq, Hkv, Hkv], 1), kc, vc, at, pos.int(), R, q_weight=qw, k_weight=kw, head_major=hm)
    assert owner.shape == pos.shape
    pools = pa.CachePools([k, v], head_major=hm)
    starts = torch.arange(S + 1, **i32) * n
    for step in range(6):
        parents = [[-1] + [int(rng.integers(0, j)) for j in range(1, n)] for _ in range(S)]
        depth = [[0] * n for _ in range(S)]
        for s in range(S):
            for j in range(1, n):
                depth[s][j] = depth[s][parents[s][j]] + 1
        mask = torch.from_numpy(ref.words(sum((ref.ancestors(p) for p in parents), []), 1)).cuda()
        base = lens.clone()
        lens += n
        for s in range(S):
            grow(s, int(lens[s]))
        pos = torch.cat([int(base[s]) + torch.tensor(depth[s], device="cuda") for s in range(S)]).int()
        at = torch.cat([slots(s, int(base[s]) + torch.arange(n, device="cuda")) for s in range(S)])
        qkv = rnd(S * n, Hq + 2 * Hkv, D)
        parts = qkv.split([Hq, Hkv, Hkv], 1)
        q = pa.append_kvcache(*parts, k, v, at, pos, R, q_weight=qw, k_weight=kw, head_major=hm)
        out = pa.decode_tree(q, k, v, tables, lens, starts, mask, D ** -0.5, head_major=hm)
        o, A = ref.attention(q, k, v, tables, lens, starts, mask, D ** -0.5, bs, hm)
        assert ((out.double() - o).abs() <= tc.element_bound(o, A)).all()
        # a path from the root
        kept = np.full((S, n), -1, np.int32)
        for s in range(S):
            path, node = [0], 0
            while True:
                children = [j for j in range(n) if parents[s][j] == node]
                if not children or len(path) > 4:
                    break
                node = children[int(rng.integers(0, len(children)))]
                path.append(node)
            kept[s, :len(path)] = path
        before = refs.sum().item()
        pa.keep_tokens(pools, tables, lens, starts, torch.from_numpy(kept).cuda(), ref_counts=refs)
        count = (kept >= 0).sum(1)
        assert torch.equal(lens, base + torch.from_numpy(count).cuda())
        assert before - refs.sum().item() == sum(-(-int(base[s] + n) // bs) - -(-int(lens[s]) // bs) for s in range(S))
        free += [b for b in range(1, NB) if refs[b] == 0 and b not in free]
        # the cache without drafts, and the kept rows' attention through plain decode
        for s in range(S):
            rows = s * n + torch.from_numpy(kept[s, :count[s]]).cuda().long()
            t = int(base[s]) + torch.arange(count[s], device="cuda")
            if step == 0 and s == 0:
                want_q, _ = rotary_ref.rotated(parts[0][rows], t, rotary_ref.frequencies(128, 1e4, "yarn", 4.0, 64.0), False,
                                               R.amplitude, qw)
                assert (q[rows].double() - want_q).abs().max() < 0.05 * want_q.abs().max()
            pa.append_kvcache(None, parts[1][rows], parts[2][rows], k2, v2, slots(s, t), t.int(), R, k_weight=kw, head_major=hm)
            both = [(x.transpose(1, 2) if hm else x)[tables[s].long()[torch.arange(int(lens[s]), device="cuda") // bs],
                                                     torch.arange(int(lens[s]), device="cuda") % bs] for x in (k, v, k2, v2)]
            assert torch.equal(both[0], both[2]) and torch.equal(both[1], both[3])
            last = pa.decode(q[rows[-1:]], k2, v2, tables[s:s + 1], lens[s:s + 1], D ** -0.5, head_major=hm)
            assert ((last.double() - o[rows[-1:]]).abs() <= tc.element_bound(o, A)[rows[-1:]]).all()
    assert pa.take_device_error() == 0
