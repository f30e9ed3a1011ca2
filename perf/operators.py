"""Cases for the operators on the pages of a KV cache and for decode attention
over a shared prefix, each with its plain form in torch.

A pool is [num_blocks, block_size, num_kv_heads, 128] bf16, or [num_blocks,
num_kv_heads, block_size, 128] (head_major); a model keeps one for K and one
for V in every layer, all indexed by the same block ids. A sequence is a row of
`block_tables` that owns its first ceil(context_len / block_size) entries;
`ref_counts[b]` is the number of owned entries that name block b, and 0 marks a
free block. Block 0 is the null block, which no row owns.

  copy     block dst becomes a copy of block src, for a list of (src, dst)
  fork     a child row shares its parent's full blocks and gets a copy of the
           used rows of the partly filled last one, in the lowest free block
  free     rows give up their blocks
  compact  the live blocks move to ids 1 .. n, and every table follows
  shared   one query token per sequence; the sequences of a group have their
           first prefix_blocks table entries in common
"""
import random

import numpy as np
import torch

own = False

HEAD_DIM = 128


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # two blocks copied in one layer's K and V: a copy-on-write in a decode step
        dict(name="copy_two_blocks", kind="copy", pools=2, blocks=128, block_size=16, kv_heads=8, pairs=2),
        # half of a pool of four layers copied: blocks duplicated for a batch of new sequences
        dict(name="copy_half_pool", kind="copy", pools=8, blocks=4096, block_size=16, kv_heads=8, pairs=2047),
        # one prompt answered three more times, one layer
        dict(name="fork_prompt", kind="fork", pools=2, blocks=128, block_size=16, kv_heads=8, parents=1,
             children=3, lo=301, hi=301, head_major=False),
        # 16 prompts, 16 samples of each, large blocks, four layers
        dict(name="fork_samples", kind="fork", pools=8, blocks=512, block_size=256, kv_heads=8, parents=16,
             children=256, lo=500, hi=3900, head_major=True),
        # the sequences that ended in one decode step
        dict(name="free_step", kind="free", blocks=2049, block_size=16, rows=64, freed=4, lo=64, hi=1024, shared=8),
        # a whole batch of long sequences given up at once
        dict(name="free_batch", kind="free", blocks=131072, block_size=16, rows=256, freed=255, lo=512, hi=16384,
             shared=128),
        # a small pool, half live, one layer
        dict(name="compact_small", kind="compact", pools=2, blocks=128, block_size=16, kv_heads=8, rows=4, lo=1,
             hi=300),
        # a fragmented pool of four layers, about half live
        dict(name="compact_fragmented", kind="compact", pools=8, blocks=4096, block_size=16, kv_heads=8, rows=16,
             lo=512, hi=3800),
        # the smallest shared batch: four samples of one short prompt
        dict(name="shared_tiny", kind="shared", q_heads=16, kv_heads=8, block_size=16, groups=1, seqs=4,
             prefix_lo=8, prefix_hi=8, lo=1, hi=64, head_major=False),
        # 60 sequences: 12 prompts, 5 samples of each, ragged
        dict(name="shared_samples", kind="shared", q_heads=16, kv_heads=8, block_size=16, groups=12, seqs=60,
             prefix_lo=4, prefix_hi=48, lo=1, hi=500, head_major=False),
        # 128 sequences behind one 2048-token system prompt, 256 tokens of their own
        dict(name="shared_system_prompt", kind="shared", q_heads=64, kv_heads=8, block_size=16, groups=1, seqs=128,
             prefix_lo=128, prefix_hi=128, lo=256, hi=256, head_major=False),
        # 256 sequences over one 32768-token document
        dict(name="shared_document", kind="shared", q_heads=32, kv_heads=8, block_size=64, groups=1, seqs=256,
             prefix_lo=512, prefix_hi=512, lo=16, hi=1000, head_major=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng: random.Random):
    kind = rng.choice(["copy", "fork", "free", "compact", "shared", "shared"])
    bs = 1 << rng.randint(4, 8)
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    pools = 2 * rng.randint(1, 4)
    block_bytes = bs * hkv * HEAD_DIM * 2
    most = max(8, min(4096, (1 << 30) // (pools * block_bytes)))     # a pool set of 1 GB at most
    if kind == "copy":
        blocks = _log(rng, 8, most)
        return dict(kind=kind, pools=pools, blocks=blocks, block_size=bs, kv_heads=hkv,
                    pairs=_log(rng, 1, (blocks - 1) // 2))
    if kind == "fork":
        parents = _log(rng, 1, 16)
        children = _log(rng, parents, 200)
        hi = _log(rng, 2, 3900)
        blocks = 1 + parents * -(-hi // bs) + children + rng.randint(0, 40)
        while pools > 2 and pools * blocks * block_bytes > 2 << 30:
            pools -= 2
        return dict(kind=kind, pools=pools, blocks=blocks, block_size=bs, kv_heads=hkv, parents=parents,
                    children=children, lo=rng.randint(1, hi), hi=hi, head_major=rng.random() < 0.5)
    if kind == "free":
        rows = _log(rng, 2, 250)
        hi = _log(rng, 1, 16000)
        shared = rng.randint(0, -(-hi // bs) // 2)
        blocks = 2 + shared + rows * -(-hi // bs) + rng.randint(50, 150)
        return dict(kind=kind, blocks=blocks, block_size=bs, rows=rows, freed=_log(rng, 1, rows - 1),
                    lo=rng.randint(1, hi), hi=hi, shared=shared)
    if kind == "compact":
        rows = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, (most - 2) // rows * bs))
        live = rows * -(-hi // bs)
        return dict(kind=kind, pools=pools, blocks=min(most, 2 + live + _log(rng, 1, live)), block_size=bs,
                    kv_heads=hkv, rows=rows, lo=rng.randint(1, hi), hi=hi)
    seqs = _log(rng, 1, 200)
    groups = _log(rng, 1, seqs)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    # tokens of prefix over all groups and of the sequences' own, at most
    prefix_hi = _log(rng, 16, max(16, min(20000, 60000 // groups)))
    hi = _log(rng, 1, max(1, min(2000, 200000 // seqs)))
    prefix_hi = max(1, min(prefix_hi, 30000 * 256 * 32 // (seqs * group * hkv)) // bs)
    return dict(kind="shared", q_heads=group * hkv, kv_heads=hkv, block_size=bs, groups=groups, seqs=seqs,
                prefix_lo=rng.randint(0, prefix_hi), prefix_hi=prefix_hi, lo=rng.randint(0, hi), hi=hi,
                head_major=rng.random() < 0.5)


# -- structure that follows from the case alone --------------------------------

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], in a fixed shuffled order."""
    v = lo + (np.arange(n) * (hi - lo)) // max(1, n - 1)
    return np.random.RandomState(n).permutation(v).astype(np.int64)


def _groups(case):
    """First sequence of each group (and the end), and each group's prefix blocks."""
    S, G = case["seqs"], case["groups"]
    starts = (np.arange(G + 1) * S) // G
    return starts, _spread(G, case["prefix_lo"], case["prefix_hi"])


def _shared_lengths(case):
    starts, prefix = _groups(case)
    own_len = _spread(case["seqs"], case["lo"], case["hi"])
    return np.repeat(prefix, np.diff(starts)) * case["block_size"] + own_len, own_len


def _row_lengths(case):
    n = case["parents"] if case["kind"] == "fork" else case["rows"]
    return _spread(n, case["lo"], case["hi"])


def work(case):
    kind, row = case["kind"], HEAD_DIM * 2
    if kind == "copy":
        n = case["pairs"] * case["pools"] * case["block_size"] * case["kv_heads"] * row
        return {"bytes": 2 * n + 8 * case["pairs"], "flops": 0}
    if kind == "fork":
        bs = case["block_size"]
        L = _row_lengths(case)[np.arange(case["children"]) % case["parents"]]
        tail = int((L % bs).sum()) * case["pools"] * case["kv_heads"] * row
        # a parent's entries are read once, a child's written; counts of shared blocks are
        # read and written, and the counts are searched for free blocks
        ents = int((-(-L // bs)).sum())
        full = int((_row_lengths(case) // bs).sum())
        return {"bytes": 2 * tail + 4 * ents + 12 * full + 4 * case["blocks"], "flops": 0}
    if kind == "free":
        L = _row_lengths(case)[:case["freed"]]
        ents = int((-(-L // case["block_size"])).sum())
        return {"bytes": 16 * ents + 12 * case["freed"], "flops": 0}    # entry and count, read and written
    if kind == "compact":
        L = _row_lengths(case)
        live = int((-(-L // case["block_size"])).sum())
        moved = live - live * live // (case["blocks"] - 1)     # live ids above `live`, on average
        n = moved * case["pools"] * case["block_size"] * case["kv_heads"] * row
        return {"bytes": 2 * n + 8 * live + 12 * case["blocks"], "flops": 0}
    starts, prefix = _groups(case)
    L, own_len = _shared_lengths(case)
    tokens = int(prefix.sum()) * case["block_size"] + int(own_len.sum())
    S, hq = case["seqs"], case["q_heads"]
    return {"bytes": tokens * case["kv_heads"] * 2 * row + 2 * S * hq * row + 4 * tokens // case["block_size"],
            "flops": 4 * int(L.sum()) * hq * HEAD_DIM}


# -- inputs ----------------------------------------------------------------------

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _pool_shape(case):
    bs, hkv = case["block_size"], case["kv_heads"]
    return (case["blocks"], hkv, bs, HEAD_DIM) if case.get("head_major") else (case["blocks"], bs, hkv, HEAD_DIM)


def _int_views(flat, blocks, rows, width):
    """ref_counts [blocks], block_tables [rows, width], context_lens [rows] in one buffer."""
    refs, tables, lens = torch.split(flat, [blocks, rows * width, rows])
    return refs, tables.view(rows, width), lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    kind = case["kind"]
    if kind == "shared":
        return _prepare_shared(s, case, gen)
    NB = case["blocks"]
    if kind != "free":
        # the K and V pools of every layer: slices of one allocation
        s["all"] = _normal((case["pools"],) + _pool_shape(case), gen)
        s["caches"] = list(s["all"].unbind(0))
    ids = 1 + torch.randperm(NB - 1, generator=gen, device="cuda")      # block ids in random order
    if kind == "copy":
        n = case["pairs"]
        pairs = torch.stack([ids[:n], ids[n:2 * n]], 1).to(torch.int32)
        if n > 8:
            pairs[::9] = -1                      # unused places of a list of fixed length
        s["pairs"] = pairs.contiguous()
    else:
        _prepare_tables(s, case, ids, gen)
    if own:
        from paged_kv_cache_255_gb300 import pagedattn as pa
        s["pa"] = pa
        if kind != "free":
            s["pools"] = pa.CachePools(s["caches"], head_major=bool(case.get("head_major")))
    return s


def _prepare_tables(s, case, ids, gen):
    kind, bs, NB = case["kind"], case["block_size"], case["blocks"]
    L = _row_lengths(case)
    n = len(L)
    rows = n + (case["children"] if kind == "fork" else 0)
    width = max(1, int(-(-L.max() // bs)))
    nb = torch.from_numpy(-(-L // bs)).cuda()
    flat = torch.zeros(NB + rows * width + rows, dtype=torch.int32, device="cuda")
    refs, tables, lens = _int_views(flat, NB, rows, width)
    lens[:n] = torch.from_numpy(L).to("cuda", torch.int32)
    col = torch.arange(width, device="cuda")
    owned = col < nb[:, None]
    # the first `shared` entries of every row name the same blocks, the rest are its own
    shared = min(case.get("shared", 0), width)
    mine = owned & (col >= shared)
    at = mine.flatten().cumsum(0).view(n, width) - 1 + shared
    entry = torch.where(mine, ids[at.clamp(0, NB - 2)], ids[col.clamp(max=NB - 2)])
    tables[:n] = torch.where(owned, entry, 0).to(torch.int32)
    refs.index_add_(0, tables[:n].flatten().long(), owned.flatten().to(torch.int32))
    s["refs"], s["tables"], s["lens"] = refs, tables, lens
    # a pass changes these in place: it starts from this copy each time
    s["ints"], s["saved"] = flat, flat.clone()
    if kind == "fork":
        c = torch.arange(case["children"], device="cuda")
        s["children"] = (n + torch.randperm(case["children"], generator=gen, device="cuda")).to(torch.int32)
        s["parents"] = (c % n).to(torch.int32)
    elif kind == "free":
        s["rows"] = torch.arange(case["freed"], device="cuda", dtype=torch.int32)


def _prepare_shared(s, case, gen):
    bs, hkv, S, G = case["block_size"], case["kv_heads"], case["seqs"], case["groups"]
    starts, prefix = _groups(case)
    L, own_len = _shared_lengths(case)
    own_nb = -(-own_len // bs)
    group_of = np.repeat(np.arange(G), np.diff(starts))
    total = int(prefix.sum() + own_nb.sum())
    NB = 1 + total + total // 5
    k = _normal(_pool_shape({**case, "blocks": NB}), gen)
    v = _normal(_pool_shape({**case, "blocks": NB}), gen)
    ids = 1 + torch.randperm(NB - 1, generator=gen, device="cuda")
    # block j of a group's prefix is ids[pre[g] + j]; a sequence's own come after all prefixes
    pre = torch.from_numpy(np.cumsum(prefix) - prefix).cuda()
    mine = torch.from_numpy(int(prefix.sum()) + np.cumsum(own_nb) - own_nb).cuda()
    width = max(1, int((prefix[group_of] + own_nb).max()))
    col = torch.arange(width, device="cuda")
    g = torch.from_numpy(group_of).cuda()
    pb = torch.from_numpy(prefix).cuda()
    nb = pb[g] + torch.from_numpy(own_nb).cuda()
    at = torch.where(col < pb[g][:, None], pre[g][:, None] + col, mine[:, None] + col - pb[g][:, None])
    tables = torch.where(col < nb[:, None], ids[at.clamp(0, NB - 2)], 0).to(torch.int32)
    s.update(q=_normal((S, case["q_heads"], HEAD_DIM), gen), k=k, v=v, tables=tables,
             lens=torch.from_numpy(L).to("cuda", torch.int32),
             starts=torch.from_numpy(starts).to("cuda", torch.int32), prefix=pb.to(torch.int32), scale=HEAD_DIM ** -0.5,
             # sizes a plain form needs on the host, and each sequence's group and place in it
             most=(int(np.diff(starts).max()), int(prefix.max()), max(1, int(own_nb.max()))),
             group=g, place=torch.from_numpy(np.arange(S) - starts[:-1][group_of]).cuda())
    if own:
        from paged_kv_cache_255_gb300 import pagedattn as pa
        s["pa"] = pa
    return s


# -- one pass ----------------------------------------------------------------------

def run(state):
    return _RUN[state["case"]["kind"]](state)


def _run_copy(s):
    if own:
        s["pa"].copy_blocks(s["pools"], s["pairs"])
        return s["all"]
    pairs = s["pairs"].long()
    used = (pairs >= 0).all(1)
    src, dst = torch.where(used, pairs[:, 0], 0), torch.where(used, pairs[:, 1], 0)    # unused: 0 onto itself
    s["all"][:, dst] = s["all"][:, src]
    return s["all"]


def _ints(s):
    return {"refs": s["refs"], "tables": s["tables"], "lens": s["lens"]}


def _run_fork(s):
    s["ints"].copy_(s["saved"])
    if own:
        s["pa"].fork_blocks(s["pools"], s["tables"], s["lens"], s["refs"], s["parents"], s["children"])
        return {"caches": s["all"], **_ints(s)}
    case, refs, tables, lens = s["case"], s["refs"], s["tables"], s["lens"]
    bs = case["block_size"]
    parents, children = s["parents"].long(), s["children"].long()
    L = lens[parents].long()
    full, tail = L // bs, L % bs
    need = tail > 0
    free = refs == 0
    free[0] = False
    # the k-th fork that needs a block takes the k-th lowest free one; others stand at block 0
    new = torch.where(need, torch.searchsorted(free.cumsum(0), need.cumsum(0)), 0)
    col = torch.arange(tables.shape[1], device=tables.device)
    rows = tables[parents].long()
    src = torch.where(need, rows.gather(1, full.clamp(max=tables.shape[1] - 1)[:, None])[:, 0], 0)
    rows = torch.where((col == full[:, None]) & need[:, None], new[:, None], rows)
    tables[children] = rows.to(torch.int32)
    lens[children] = L.to(torch.int32)
    refs.index_add_(0, rows.flatten(), (col < (full + need)[:, None]).flatten().to(torch.int32))
    used = torch.arange(bs, device=tables.device) < tail[:, None]
    used = used[:, None, :, None] if case["head_major"] else used[:, :, None, None]
    s["all"][:, new] = torch.where(used, s["all"][:, src], s["all"][:, new])
    return {"caches": s["all"], **_ints(s)}


def _run_free(s):
    s["ints"].copy_(s["saved"])
    if own:
        s["pa"].free_blocks(s["tables"], s["lens"], s["refs"], s["rows"], s["case"]["block_size"])
        return _ints(s)
    refs, tables, lens = s["refs"], s["tables"], s["lens"]
    rows = s["rows"].long()
    bs = s["case"]["block_size"]
    nb = (lens[rows].long() + bs - 1) // bs
    owned = torch.arange(tables.shape[1], device=tables.device) < nb[:, None]
    refs.index_add_(0, tables[rows].flatten().long(), -owned.flatten().to(torch.int32))
    tables[rows] = torch.where(owned, 0, tables[rows])
    lens[rows] = 0
    return _ints(s)


def _run_compact(s):
    s["ints"].copy_(s["saved"])
    if own:
        remap, num_live = s["pa"].compact_blocks(s["pools"], s["tables"], s["lens"], s["refs"])
        return {"caches": s["all"], "remap": remap, "num_live": num_live, **_ints(s)}
    refs, tables, lens = s["refs"], s["tables"], s["lens"]
    ids = torch.arange(refs.shape[0], device=refs.device)
    live = refs > 0
    live[0] = False
    n = live.sum()
    holes = torch.nonzero(~live & (ids > 0) & (ids <= n))[:, 0]
    high = torch.nonzero(live & (ids > n))[:, 0]
    s["all"][:, holes] = s["all"][:, high]
    remap = torch.where(live, ids, 0)
    remap[high] = holes
    refs[holes] = refs[high]
    refs[high] = 0
    bs = s["case"]["block_size"]
    owned = torch.arange(tables.shape[1], device=tables.device) < ((lens.long() + bs - 1) // bs)[:, None]
    tables.copy_(torch.where(owned, remap[tables.long()].to(torch.int32), tables))
    return {"caches": s["all"], "remap": remap.to(torch.int32), "num_live": n.to(torch.int32).view(1), **_ints(s)}


def _rows_of(pool, blocks, head_major):
    """Token rows of the blocks [..., n] of a pool, in 32 bits: [..., n * block_size, kv_heads, 128]."""
    x = pool[blocks].float()
    return (x.transpose(-3, -2) if head_major else x).flatten(-4, -3)


def _run_shared(s):
    case, q, tables = s["case"], s["q"], s["tables"]
    if own:
        return s["pa"].decode_shared(q, s["k"], s["v"], tables, s["lens"], s["starts"], s["prefix"], s["scale"],
                                     head_major=case["head_major"])
    hm, bs = case["head_major"], case["block_size"]
    S, hq, _ = q.shape
    hkv, G = case["kv_heads"], case["groups"]
    most_seqs, most_prefix, most_own = s["most"]
    g, place, lens = s["group"], s["place"], s["lens"].long()
    qs = q.float().view(S, hkv, hq // hkv, HEAD_DIM) * s["scale"]
    # every group's prefix once, for all its sequences
    first = tables[s["starts"][:-1].long()].long()[:, :most_prefix]
    qg = qs.new_zeros((G, most_seqs) + qs.shape[1:])
    qg[g, place] = qs
    pre = torch.einsum("gnhcd,gthd->gnhct", qg, _rows_of(s["k"], first, hm))[g, place]
    prefix_len = (s["prefix"].long() * bs)[g]
    t = torch.arange(most_prefix * bs, device=q.device)
    pre = pre.masked_fill((t >= prefix_len[:, None])[:, None, None], -torch.inf)
    # each sequence's own tokens
    at = s["prefix"].long()[g][:, None] + torch.arange(most_own, device=q.device)
    mine = tables.long().gather(1, at.clamp(max=tables.shape[1] - 1))
    t = prefix_len[:, None] + torch.arange(most_own * bs, device=q.device)
    seen = t < lens[:, None]
    suf = torch.einsum("shcd,sthd->shct", qs, _rows_of(s["k"], mine, hm))
    suf = suf.masked_fill(~seen[:, None, None], -torch.inf)
    m = torch.maximum(pre.amax(-1) if most_prefix else suf.amax(-1), suf.amax(-1)).clamp(min=-3e38)[..., None]
    p, w = torch.exp(pre - m), torch.exp(suf - m)
    total = p.sum(-1, keepdim=True) + w.sum(-1, keepdim=True)
    pg = p.new_zeros((G, most_seqs) + p.shape[1:])
    pg[g, place] = p
    o = torch.einsum("gnhct,gthd->gnhcd", pg, _rows_of(s["v"], first, hm))[g, place]
    o = o + torch.einsum("shct,sthd->shcd", w, torch.where(seen[..., None, None], _rows_of(s["v"], mine, hm), 0))
    return torch.where(total > 0, o / total, 0).reshape(S, hq, HEAD_DIM).to(torch.bfloat16)


_RUN = {"copy": _run_copy, "fork": _run_fork, "free": _run_free, "compact": _run_compact, "shared": _run_shared}


# -- the definition of the attention in 64 bits ---------------------------------------

def exact(case, seed):
    """softmax(scale q K^T) V of each sequence over its own table alone. The
    page operators move values and compute none."""
    if case["kind"] != "shared":
        return None
    s = prepare(case, seed)
    hkv = case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        blocks = s["tables"][i, :-(-n // case["block_size"])].long()
        K, V = s["k"][blocks], s["v"][blocks]
        if case["head_major"]:
            K, V = K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3)
        K, V = (x.reshape(-1, hkv, HEAD_DIM)[:n].permute(1, 0, 2).double() for x in (K, V))
        q = s["q"][i].double().view(hkv, -1, HEAD_DIM)
        a = torch.softmax(q @ K.transpose(1, 2) * s["scale"], -1)
        out[i] = (a @ V).reshape(-1, HEAD_DIM)
    return out
