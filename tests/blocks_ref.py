"""Plain model of the block operations on numpy arrays: one loop per sentence
of their contract, one item after the other. Pools are uint16 arrays
[NB, bs, Hkv, D] ([NB, Hkv, bs, D] with head_major), all changed in place.
Every function returns the set of error codes the device would record."""
import numpy as np

BAD_ENTRY, FORK_REFUSED = 5, 6


def owned(tables, lens, row, bs):
    n = min(max(int(lens[row]), 0), tables.shape[1] * bs)
    return n, -(-n // bs)


def copy(pools, pairs):
    codes = set()
    for src, dst in pairs:
        if src == -1 or dst == -1:
            continue
        if not (0 <= src < pools[0].shape[0] and 0 <= dst < pools[0].shape[0]):
            codes.add(BAD_ENTRY)
            continue
        for p in pools:
            p[dst] = p[src]
    return codes


def fork(pools, tables, lens, refs, parents, children, bs, head_major=False):
    codes = set()
    before, rows, NB = lens.copy(), tables.shape[0], refs.shape[0]
    free = [b for b in range(1, NB) if refs[b] <= 0]
    taken = set()
    old_tables = tables.copy()
    for p, c in zip(parents, children):
        if p == -1 or c == -1:
            continue
        if not (0 <= p < rows and 0 <= c < rows):
            codes.add(BAD_ENTRY)
            continue
        first = int(c) not in taken
        taken.add(int(c))
        if before[c] > 0 or not first:
            codes.add(FORK_REFUSED)
            continue
        L, nb = owned(tables, before, p, bs)
        new = None
        if L % bs and 0 < old_tables[p, nb - 1] < NB:
            if not free:
                codes.add(FORK_REFUSED)
                continue
            new = free.pop(0)
        lens[c] = L
        for j in range(nb):
            b = int(old_tables[p, j])
            if j == nb - 1 and new is not None:
                for q in pools:
                    if head_major:
                        q[new][:, :L % bs] = q[b][:, :L % bs]
                    else:
                        q[new][:L % bs] = q[b][:L % bs]
                tables[c, j], refs[new] = new, 1
                continue
            tables[c, j] = b
            if 0 < b < NB:
                if refs[b] <= 0:
                    codes.add(BAD_ENTRY)
                refs[b] += 1
            elif b != 0:
                codes.add(BAD_ENTRY)
    return codes


def free(tables, lens, refs, rows, bs):
    codes = set()
    for r in rows:
        if r == -1:
            continue
        if not 0 <= r < tables.shape[0]:
            codes.add(BAD_ENTRY)
            continue
        _, nb = owned(tables, lens, r, bs)
        lens[r] = 0
        for j in range(nb):
            b = int(tables[r, j])
            tables[r, j] = 0
            if b == 0:
                continue
            if not 0 < b < refs.shape[0] or refs[b] <= 0:
                codes.add(BAD_ENTRY)
                continue
            refs[b] -= 1
    return codes


def compact(pools, tables, lens, refs, bs):
    """Also returns (remap, number of live blocks)."""
    codes = set()
    NB = refs.shape[0]
    live = [b for b in range(1, NB) if refs[b] > 0]
    n = len(live)
    holes = [b for b in range(1, n + 1) if refs[b] <= 0]
    remap = np.zeros(NB, np.int32)
    for b in live:
        remap[b] = b
    for src, dst in zip([b for b in live if b > n], holes):
        remap[src] = dst
        for p in pools:
            p[dst] = p[src]
        refs[dst], refs[src] = refs[src], 0
    for r in range(tables.shape[0]):
        for j in range(owned(tables, lens, r, bs)[1]):
            b = int(tables[r, j])
            if b == 0:
                continue
            if not 0 < b < NB or remap[b] == 0:
                codes.add(BAD_ENTRY)
                continue
            tables[r, j] = remap[b]
    return codes, remap, n


def draw(rng, rows, width, bs, NB, lens=None, shared=0, spare=0):
    """Consistent tables: `rows` live rows over random blocks, their first
    `shared` entries in common, then `spare` empty rows. Returns tables, lens,
    refs; unused entries hold an id out of range, which nothing may read."""
    if lens is None:
        lens = rng.integers(0, width * bs + 1, size=rows)
    lens = np.concatenate([np.asarray(lens, np.int32), np.zeros(spare, np.int32)])
    ids = list(1 + rng.permutation(NB - 1))
    prefix = [ids.pop() for _ in range(min(shared, width))]
    tables = np.full((rows + spare, width), NB + 7, np.int32)
    refs = np.zeros(NB, np.int32)
    for r in range(rows):
        for j in range(-(-int(lens[r]) // bs)):
            b = prefix[j] if j < len(prefix) else ids.pop()
            tables[r, j] = b
            refs[b] += 1
    return tables, lens, refs


def counts(tables, lens, NB, bs):
    """Counts that the owned entries of the tables give."""
    refs = np.zeros(NB, np.int32)
    for r in range(tables.shape[0]):
        for b in tables[r, :owned(tables, lens, r, bs)[1]]:
            if 0 < b < NB:
                refs[b] += 1
    return refs
