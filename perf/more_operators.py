"""Cases for a step of speculative decoding with rotary positions over a paged
KV cache, each with its plain form in torch.

A pool is [num_blocks, block_size, num_kv_heads, 128] bf16, or [num_blocks,
num_kv_heads, block_size, 128] (head_major); token t of a sequence lies in block
block_tables[s, t // block_size] at row t % block_size.

  rotate  the rotation of queries and keys by their positions, with the norm of
          each head's row before it in the same pass
  append  the same on the way of a step's keys and values into the pools
  tree    attention of a tree of drafted tokens per sequence, the last tokens of
          its cache, over everything before them and their own ancestors
  keep    the cache rows of the accepted tokens move to consecutive places
"""
import math
import random

import numpy as np
import torch

own = False

HEAD_DIM = 128
ROW = HEAD_DIM * 2


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # four sequences' new tokens, norms of the heads: the smallest decode step
        dict(name="rotate_step", kind="rotate", tokens=4, q_heads=16, kv_heads=8, rot_dim=128, interleaved=False,
             scaling="plain", factor=1.0, norm=True, far=1024),
        # an odd number of far positions, half of each head rotated in neighbouring pairs
        dict(name="rotate_far", kind="rotate", tokens=997, q_heads=32, kv_heads=8, rot_dim=64, interleaved=True,
             scaling="yarn", factor=32.0, norm=False, far=131072),
        # whole prompts at once
        dict(name="rotate_prompts", kind="rotate", tokens=16384, q_heads=32, kv_heads=8, rot_dim=128,
             interleaved=False, scaling="banded", factor=8.0, norm=True, far=131072),
        # a decode step of 60 sequences
        dict(name="append_step", kind="append", tokens=60, q_heads=16, kv_heads=8, rot_dim=128, interleaved=False,
             scaling="plain", factor=1.0, norm=True, far=1024, block_size=16, head_major=False),
        # chunks of an odd size with padding rows, part of the head rotated
        dict(name="append_chunk", kind="append", tokens=2047, q_heads=32, kv_heads=8, rot_dim=96, interleaved=True,
             scaling="linear", factor=4.0, norm=False, far=32768, block_size=64, head_major=True),
        # whole prompts, many query heads
        dict(name="append_prompts", kind="append", tokens=16384, q_heads=64, kv_heads=8, rot_dim=128,
             interleaved=False, scaling="ntk", factor=8.0, norm=True, far=131072, block_size=16, head_major=False),
        # four short sequences, small trees
        dict(name="tree_tiny", kind="tree", q_heads=16, kv_heads=8, block_size=16, seqs=4, lo=1, hi=300, nodes_lo=1,
             nodes_hi=8, head_major=False),
        # a batch of 60, ragged trees
        dict(name="tree_batch", kind="tree", q_heads=16, kv_heads=8, block_size=16, seqs=60, lo=64, hi=1024,
             nodes_lo=4, nodes_hi=25, head_major=False),
        # wide trees, many query heads: every row of the tensor cores' tiles is used
        dict(name="tree_wide", kind="tree", q_heads=64, kv_heads=8, block_size=64, seqs=32, lo=2048, hi=8192,
             nodes_lo=48, nodes_hi=64, head_major=True),
        # a few long contexts
        dict(name="tree_long", kind="tree", q_heads=32, kv_heads=8, block_size=16, seqs=8, lo=32768, hi=131072,
             nodes_lo=16, nodes_hi=32, head_major=False),
        # one layer, four sequences
        dict(name="keep_step", kind="keep", pools=2, kv_heads=8, block_size=16, seqs=4, lo=1, hi=300, nodes=8, kept=3,
             head_major=False),
        # 16 layers, a batch of 64
        dict(name="keep_layers", kind="keep", pools=32, kv_heads=8, block_size=16, seqs=64, lo=64, hi=1024, nodes=32,
             kept=6, head_major=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng: random.Random):
    kind = rng.choice(["rotate", "append", "append", "tree", "tree", "tree", "keep"])
    bs = 1 << rng.randint(4, 8)
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    hm = rng.random() < 0.5
    if kind in ("rotate", "append"):
        scaling = rng.choice(["plain", "linear", "ntk", "yarn", "banded"])
        far = _log(rng, 64, 1 << 20)
        case = dict(kind=kind, tokens=_log(rng, 1, 16384), q_heads=group * hkv, kv_heads=hkv,
                    rot_dim=16 * rng.randint(1, 8), interleaved=rng.random() < 0.5, scaling=scaling,
                    factor=1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0, 32.0]), norm=rng.random() < 0.5,
                    far=far)
        return case if kind == "rotate" else {**case, "block_size": bs, "head_major": hm}
    if kind == "keep":
        nodes = _log(rng, 1, 64)
        pools = 2 * _log(rng, 1, 16)
        seqs = _log(rng, 1, 64)
        most = max(2, min(2000, (1 << 32) // (pools * hkv * ROW * seqs) - nodes - bs))     # pools of 4 GB at most
        hi = _log(rng, 1, most)
        return dict(kind=kind, pools=pools, kv_heads=hkv, block_size=bs, seqs=seqs, lo=rng.randint(0, hi), hi=hi,
                    nodes=nodes, kept=rng.randint(1, min(nodes, 12)), head_major=hm)
    seqs = _log(rng, 1, 128)
    nodes_hi = _log(rng, 1, 150)
    rows = nodes_hi * group * hkv
    # tokens of context, over all sequences, and their products with the rows
    hi = _log(rng, 1, max(2, min(131072, 600000 // seqs, (1 << 29) // (seqs * rows))))
    return dict(kind="tree", q_heads=group * hkv, kv_heads=hkv, block_size=bs, seqs=seqs, lo=rng.randint(0, hi), hi=hi,
                nodes_lo=rng.randint(0, nodes_hi), nodes_hi=nodes_hi, head_major=hm)


# -- structure that follows from the case alone --------------------------------

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], in a fixed shuffled order."""
    v = lo + (np.arange(n) * (hi - lo)) // max(1, n - 1)
    return np.random.RandomState(n).permutation(v).astype(np.int64)


def _tree_sizes(case):
    """Tokens before each tree, nodes of each tree (nodes of the first: the most)."""
    base = _spread(case["seqs"], case["lo"], case["hi"])
    nodes = _spread(case["seqs"], case["nodes_lo"], case["nodes_hi"])
    nodes[0] = case["nodes_hi"]
    return base, nodes


def work(case):
    kind = case["kind"]
    if kind in ("rotate", "append"):
        heads = case["q_heads"] + case["kv_heads"] * (2 if kind == "append" else 1)
        T = case["tokens"]
        return {"bytes": T * (2 * heads * ROW + (12 if kind == "append" else 4)),
                "flops": T * (case["q_heads"] + case["kv_heads"]) * (3 * case["rot_dim"] + (4 * HEAD_DIM if case["norm"] else 0))}
    if kind == "keep":
        n = case["seqs"] * (case["kept"] - 1)       # the root stays where it is
        return {"bytes": 2 * n * case["pools"] * case["kv_heads"] * ROW + 4 * case["seqs"] * (case["kept"] + 4), "flops": 0}
    base, nodes = _tree_sizes(case)
    L = (base + nodes) * (nodes > 0)
    rows = int(nodes.sum()) * case["q_heads"]
    return {"bytes": int(L.sum()) * case["kv_heads"] * 2 * ROW + 2 * rows * ROW + 8 * int(nodes.sum()),
            "flops": 4 * int((L * nodes).sum()) * case["q_heads"] * HEAD_DIM}


# -- inputs ----------------------------------------------------------------------

BASE, ORIGINAL = 10000.0, 4096       # the rotation's base, the context it was learnt for


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _frequencies(case):
    """Radians a token of every rotated pair, and the factor on the result."""
    r, f = case["rot_dim"], case["factor"]
    i = np.arange(r // 2, dtype=np.float64)
    base, scaling = BASE, case["scaling"]
    if scaling == "ntk":
        base = BASE * f ** (r / (r - 2))
    theta = base ** (-2 * i / r)
    if scaling == "linear":
        theta = theta / f
    elif scaling == "yarn":
        # pairs that turn over 32 times in the original context keep their frequency, those
        # that turn less than once are slowed down, linearly between in their index
        edge = [r * math.log(ORIGINAL / (n * 2 * math.pi)) / (2 * math.log(BASE)) for n in (32, 1)]
        low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
        keep = 1 - np.clip((i - low) / max(high - low, 1e-3), 0, 1)
        theta = theta / f * (1 - keep) + theta * keep
    elif scaling == "banded":
        # by wavelength: shorter than a quarter of the original context kept, longer than it slowed down
        turns = ORIGINAL * theta / (2 * math.pi)
        keep = np.clip((turns - 1) / (4 - 1), 0, 1)
        theta = theta / f * (1 - keep) + theta * keep
    return theta, 0.1 * math.log(f) + 1 if scaling == "yarn" else 1.0


def _rotary(case, pa):
    kinds = {"plain": {}, "linear": dict(scaling="linear", factor=case["factor"]),
             "ntk": dict(scaling="ntk", factor=case["factor"]),
             "yarn": dict(scaling="yarn", factor=case["factor"], original_context=ORIGINAL),
             "banded": dict(scaling="banded", factor=case["factor"], original_context=ORIGINAL)}
    return pa.Rotary(case["rot_dim"], base=BASE, interleaved=case["interleaved"], **kinds[case["scaling"]])


def _pool_shape(case, blocks):
    bs, hkv = case["block_size"], case["kv_heads"]
    return (blocks, hkv, bs, HEAD_DIM) if case["head_major"] else (blocks, bs, hkv, HEAD_DIM)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    {"tree": _prepare_tree, "keep": _prepare_keep}.get(case["kind"], _prepare_heads)(s, case, gen, seed)
    return s


def _prepare_heads(s, case, gen, seed):
    T, hq, hkv = case["tokens"], case["q_heads"], case["kv_heads"]
    # the projection's output: the heads of q, k and v of a token side by side
    qkv = _normal((T, hq + 2 * hkv, HEAD_DIM), gen)
    s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], 1)
    s["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device="cuda", dtype=torch.int32)
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"], s["kw"] = (1 + 0.2 * _normal((HEAD_DIM,), gen).float()).bfloat16(), (1 + 0.2 * _normal((HEAD_DIM,), gen).float()).bfloat16()
    theta, s["amplitude"] = _frequencies(case)
    s["theta"] = torch.from_numpy(theta).cuda()
    s["eps"] = 1e-6
    if case["kind"] == "append":
        bs = case["block_size"]
        blocks = 2 + T // bs * 2
        s["kc"], s["vc"] = _normal(_pool_shape(case, blocks), gen), _normal(_pool_shape(case, blocks), gen)
        # distinct slots outside block 0, a few rows of padding
        slots = bs + torch.randperm((blocks - 1) * bs, generator=gen, device="cuda")[:T]
        if T > 8:
            slots[::9] = -1
        s["slots"] = slots.contiguous()
    if own:
        from paged_kv_cache_255_gb300 import pagedattn as pa
        s["pa"], s["rotary"] = pa, _rotary(case, pa)


def _ancestors(parents):
    """Bit j of entry i: node j is i or one of its ancestors. Python's whole numbers."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    return seen


def _tables(lens, bs, gen):
    """Block tables over blocks in random order, block 0 left out."""
    nb = -(-lens // bs)
    width, total = max(1, int(nb.max())), int(nb.sum())
    NB = 2 + total + total // 8
    ids = 1 + torch.randperm(NB - 1, generator=gen, device="cuda")
    first = torch.from_numpy(np.cumsum(nb) - nb).cuda()
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=NB - 2)
    owned = col < torch.from_numpy(nb).cuda()[:, None]
    return torch.where(owned, ids[at], 0).to(torch.int32), owned, NB


def _prepare_tree(s, case, gen, seed):
    base, nodes = _tree_sizes(case)
    L = base + nodes
    tables, _, NB = _tables(L, case["block_size"], gen)
    starts = np.concatenate([[0], np.cumsum(nodes)])
    T, words = int(starts[-1]), max(1, -(-int(nodes.max()) // 64))
    rng = np.random.RandomState(seed)
    mask = np.zeros((T, words), np.uint64)
    for i, n in enumerate(nodes):
        # the last nodes of every third tree are padding: nobody sees them, they see the context alone
        used = n - n // 5 if i % 3 == 2 else n
        parents = [int(rng.randint(max(0, j // 4), j)) if j else -1 for j in range(used)]
        for j, bits in enumerate(_ancestors(parents)):
            for w in range(words):
                mask[starts[i] + j, w] = bits >> 64 * w & (1 << 64) - 1
    s.update(q=_normal((T, case["q_heads"], HEAD_DIM), gen), k=_normal(_pool_shape(case, NB), gen),
             v=_normal(_pool_shape(case, NB), gen), tables=tables, lens=torch.from_numpy(L).to("cuda", torch.int32),
             starts=torch.from_numpy(starts).to("cuda", torch.int32),
             mask=torch.from_numpy(mask.view(np.int64)).cuda(), scale=HEAD_DIM ** -0.5, most=(int(nodes.max()), int(L.max())))


def _prepare_keep(s, case, gen, seed):
    S, bs = case["seqs"], case["block_size"]
    base = _spread(S, case["lo"], case["hi"])
    L = base + case["nodes"]
    tables, owned, NB = _tables(L, bs, gen)
    s["all"] = _normal((case["pools"],) + _pool_shape(case, NB), gen)
    refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    refs.index_add_(0, tables.flatten().long(), owned.flatten().to(torch.int32))
    lens = torch.from_numpy(L).to("cuda", torch.int32)
    # one buffer for what a pass changes: it starts from this copy each time
    flat = torch.cat([refs, tables.flatten(), lens])
    s["refs"], t, s["lens"] = torch.split(flat, [NB, tables.numel(), S])
    s["tables"] = t.view(tables.shape)
    s["ints"], s["saved"] = flat, flat.clone()
    s["starts"] = torch.arange(S + 1, device="cuda", dtype=torch.int32) * case["nodes"]
    rng = np.random.RandomState(seed)
    kept = np.full((S, case["kept"] + 1), -1, np.int32)      # -1 after the last
    for i in range(S):
        # a path of the tree: the root, then ever later nodes
        kept[i, :case["kept"]] = np.concatenate([[0], 1 + np.sort(rng.choice(case["nodes"] - 1, case["kept"] - 1, False))])
    s["kept"] = torch.from_numpy(kept).cuda()
    if own:
        from paged_kv_cache_255_gb300 import pagedattn as pa
        s["pools"] = pa.CachePools(list(s["all"].unbind(0)), head_major=case["head_major"])


# -- one pass ----------------------------------------------------------------------

def run(state):
    return _RUN[state["case"]["kind"]](state)


def _rotated(s, x, weight):
    """The rows x [T, heads, 128] normed and rotated, in 32 bits."""
    case = s["case"]
    r, half = case["rot_dim"], case["rot_dim"] // 2
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    # far positions: the angle in 64 bits
    angle = s["positions"].double()[:, None] * s["theta"]
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1).to(torch.bfloat16)


def _run_rotate(s):
    if own:
        return s["pa"].rotate(s["q"], s["k"], s["positions"], s["rotary"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"])
    return _rotated(s, s["q"], s["qw"]), _rotated(s, s["k"], s["kw"])


def _run_append(s):
    case = s["case"]
    if own:
        q = s["pa"].append_kvcache(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["positions"], s["rotary"],
                                   q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], head_major=case["head_major"])
        return q, s["kc"], s["vc"]
    bs, slots = case["block_size"], s["slots"]
    used = (slots >= 0)[:, None, None]
    block, row = slots.clamp(min=0) // bs, slots.clamp(min=0) % bs      # padding: row 0 of block 0 onto itself
    for cache, x in ((s["kc"], _rotated(s, s["k"], s["kw"])), (s["vc"], s["v"])):
        at = (block, slice(None), row) if case["head_major"] else (block, row)
        cache[at] = torch.where(used, x, cache[at])
    return _rotated(s, s["q"], s["qw"]), s["kc"], s["vc"]


def _tokens(pool, blocks, head_major):
    """Token rows of the blocks [S, n] of a pool, in 32 bits: [S, kv_heads, n * block_size, 128]."""
    x = pool[blocks].float()
    x = x.transpose(1, 2).flatten(2, 3) if head_major else x.flatten(1, 2).transpose(1, 2)
    return x


def _run_tree(s):
    case, q, mask = s["case"], s["q"], s["mask"]
    if own:
        from paged_kv_cache_255_gb300 import pagedattn as pa
        return pa.decode_tree(q, s["k"], s["v"], s["tables"], s["lens"], s["starts"], mask, s["scale"],
                              head_major=case["head_major"])
    hkv, (most_nodes, most_len) = case["kv_heads"], s["most"]
    T, hq, _ = q.shape
    starts, lens = s["starts"].long(), s["lens"].long()
    n = starts[1:] - starts[:-1]
    S = n.shape[0]
    # the rows of every tree side by side: row (sequence, node) of the batch
    node = torch.arange(most_nodes, device=q.device)
    real = node < n[:, None]
    row = torch.where(real, starts[:-1, None] + node, 0)
    t = torch.arange(most_len, device=q.device)
    j = t - (lens - n)[:, None]                              # [S, L]: node of each token
    word = mask[row].gather(2, (j.clamp(min=0) >> 6).clamp(max=mask.shape[1] - 1)[:, None].expand(-1, most_nodes, -1))
    seen = (j < 0)[:, None] | ((word >> (j & 63)[:, None] & 1) == 1)
    seen &= (t < lens[:, None])[:, None] & real[..., None]
    blocks = s["tables"].long()
    K, V = (_tokens(x, blocks, case["head_major"])[:, :, :most_len] for x in (s["k"], s["v"]))
    qs = (q.float() * s["scale"])[row].view(S, most_nodes, hkv, -1, HEAD_DIM).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (qs @ K.transpose(2, 3)).unflatten(2, (-1, most_nodes)).masked_fill_(~seen[:, None, None], -torch.inf)
    score -= score.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = score.exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ torch.where((t < lens[:, None])[:, None, :, None], V, 0)).unflatten(2, (-1, most_nodes))
    o = torch.where(total > 0, o / total, 0).permute(0, 3, 1, 2, 4).reshape(S, most_nodes, hq, HEAD_DIM)
    return o[real].to(torch.bfloat16)


def _run_keep(s):
    s["ints"].copy_(s["saved"])
    answer = {"caches": s["all"], "refs": s["refs"], "tables": s["tables"], "lens": s["lens"]}
    if own:
        from paged_kv_cache_255_gb300 import pagedattn as pa
        pa.keep_tokens(s["pools"], s["tables"], s["lens"], s["starts"], s["kept"], ref_counts=s["refs"])
        return answer
    case, bs = s["case"], s["case"]["block_size"]
    tables, lens, kept = s["tables"], s["lens"], s["kept"].long()
    old = lens.long()
    base = old - (s["starts"][1:] - s["starts"][:-1]).long()
    count = (kept >= 0).sum(1)
    place = torch.arange(kept.shape[1], device=kept.device)
    used = kept >= 0

    def at(t):      # unused places: row 0 of block 0
        t = torch.where(used, base[:, None] + t, 0)
        block = torch.where(used, tables.long().gather(1, (t // bs).clamp(max=tables.shape[1] - 1)), 0).flatten()
        row = torch.where(used, t % bs, 0).flatten()
        return (slice(None), block, slice(None), row) if case["head_major"] else (slice(None), block, row)
    s["all"][at(place)] = s["all"][at(kept)]
    new = base + count
    lens.copy_(new)
    col = torch.arange(tables.shape[1], device=tables.device)
    gone = (col >= ((new + bs - 1) // bs)[:, None]) & (col < ((old + bs - 1) // bs)[:, None])
    s["refs"].index_add_(0, tables.flatten().long(), -gone.flatten().to(torch.int32))
    tables.copy_(torch.where(gone, 0, tables))
    return answer


_RUN = {"rotate": _run_rotate, "append": _run_append, "tree": _run_tree, "keep": _run_keep}


# -- the definitions in 64 bits --------------------------------------------------------

def _turned(s, x, weight):
    """The definition row by row as complex numbers."""
    case, r = s["case"], s["case"]["rot_dim"]
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / HEAD_DIM + s["eps"]).sqrt() * weight.double()
    theta, amplitude = _frequencies(case)
    phase = torch.outer(s["positions"].double(), torch.from_numpy(theta).cuda())
    turn = torch.polar(torch.full_like(phase, amplitude), phase)[:, None]
    first = x[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
    if not case["interleaved"]:
        first = first.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(first.contiguous()) * turn)
    z = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return torch.cat([z, x[..., r:]], -1)


def _placed(s, pool, x):
    """The pool with the rows x at their slots."""
    bs, out = s["case"]["block_size"], pool.double()
    rows = out.transpose(1, 2) if s["case"]["head_major"] else out
    keep = s["slots"] >= 0
    rows[s["slots"][keep] // bs, s["slots"][keep] % bs] = x[keep]
    return out


def exact(case, seed):
    if case["kind"] == "keep":          # moves values and computes none
        return None
    s = prepare(case, seed)
    if case["kind"] == "rotate":
        return _turned(s, s["q"], s["qw"]), _turned(s, s["k"], s["kw"])
    if case["kind"] == "append":
        return _turned(s, s["q"], s["qw"]), _placed(s, s["kc"], _turned(s, s["k"], s["kw"])), None
    hkv, bs, starts = case["kv_heads"], case["block_size"], s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    words = s["mask"].cpu().numpy().view(np.uint64)
    for i, L in enumerate(s["lens"].tolist()):
        n = starts[i + 1] - starts[i]
        if not n:
            continue
        blocks = s["tables"][i, :-(-L // bs)].long()
        K, V = s["k"][blocks], s["v"][blocks]
        if case["head_major"]:
            K, V = K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3)
        K, V = (x.reshape(-1, hkv, HEAD_DIM)[:L].permute(1, 0, 2).double() for x in (K, V))
        q = s["q"][starts[i]:starts[i + 1]].double().view(n, hkv, -1, HEAD_DIM)
        bits = np.unpackbits(words[starts[i]:starts[i + 1]].view(np.uint8), axis=1, bitorder="little")
        seen = torch.ones(n, L, dtype=torch.bool, device="cuda")
        seen[:, L - n:] = torch.from_numpy(bits[:, :n].astype(bool)).cuda()
        for h in range(hkv):
            a = torch.einsum("ngd,td->ngt", q[:, h], K[h]) * s["scale"]
            a = torch.softmax(a.masked_fill(~seen[:, None], -torch.inf), -1).nan_to_num(0.0)
            out[starts[i]:starts[i + 1]].view(n, hkv, -1, HEAD_DIM)[:, h] = a @ V[h]
    return out
