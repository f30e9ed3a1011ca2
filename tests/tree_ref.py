"""Trees of drafted tokens: masks from parents, attention in 64 bits, and the
plain model of keeping accepted tokens."""
import numpy as np
import torch

D = 128


def ancestors(parents):
    """Bit j of entry i: node j is i or one of its ancestors (Python whole numbers)."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    return seen


def words(bits, n):
    """[len(bits), n] int64 mask words of whole numbers."""
    out = np.zeros((len(bits), n), np.uint64)
    for i, b in enumerate(bits):
        for w in range(n):
            out[i, w] = b >> 64 * w & (1 << 64) - 1
    return out.view(np.int64)


def attention(q, k, v, tables, lens, starts, mask, scale, bs, hm):
    """(o, A) in 64 bits, A = sum of weights times |V|, row by row over the tokens that
    it sees alone."""
    T, Hq, _ = q.shape
    NB = k.shape[0]
    Hkv = k.shape[1] if hm else k.shape[2]
    o = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    A = torch.zeros_like(o)
    bits = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=1, bitorder="little").astype(bool)
    starts = [min(max(x, 0), T) for x in starts.tolist()]
    for s, L in enumerate(lens.tolist()):
        L = min(max(L, 0), tables.shape[1] * bs)
        n = starts[s + 1] - starts[s]
        if n <= 0 or L == 0:
            continue
        blocks = tables[s, :-(-L // bs)].long()
        bad = (blocks < 0) | (blocks >= NB)
        K, V = (torch.where(bad[:, None, None, None], 0, x[blocks.clamp(0, NB - 1)]) for x in (k, v))
        if hm:
            K, V = K.transpose(1, 2), V.transpose(1, 2)
        K, V = (x.reshape(-1, Hkv, D)[:L].transpose(0, 1).double() for x in (K, V))
        t = np.arange(L)
        seen = np.zeros((n, L), bool)
        for i in range(n):
            node = t - (L - n)
            seen[i] = (node < 0) | ((node < bits.shape[1]) & bits[starts[s] + i, np.clip(node, 0, bits.shape[1] - 1)])
        for pattern in np.unique(seen, axis=0):
            at = torch.from_numpy(np.nonzero(pattern)[0]).to(q.device)
            if not len(at):
                continue
            rows = starts[s] + torch.from_numpy(np.nonzero((seen == pattern).all(1))[0]).to(q.device)
            qs = q[rows].double().view(len(rows), Hkv, -1, D).transpose(0, 1)
            Ks, Vs = K[:, at], V[:, at]
            p = torch.softmax(torch.einsum("hrgd,htd->hrgt", qs, Ks) * scale, -1)
            o[rows] = torch.einsum("hrgt,htd->rhgd", p, Vs).reshape(len(rows), Hq, D)
            A[rows] = torch.einsum("hrgt,htd->rhgd", p, Vs.abs()).reshape(len(rows), Hq, D)
    return o, A


def keep(pools, tables, lens, starts, kept, refs, bs, hm):
    """The model of keeping tokens on numpy arrays (pools in 16-bit words), in place;
    returns the set of codes that are recorded."""
    codes = set()
    NB = pools[0].shape[0] if pools else refs.shape[0]
    width = tables.shape[1]
    for s in range(len(lens)):
        L = min(max(int(lens[s]), 0), width * bs)
        q0, n = int(starts[s]), int(starts[s + 1]) - int(starts[s])
        if q0 < 0 or n <= 0 or n > L:
            continue
        first, path = L - n, []
        for k in kept[s].tolist():
            if not 0 <= k < n or (path and k <= path[-1]):
                if k != -1:
                    codes.add(5)
                break
            path.append(k)
        moves = []
        for i, k in enumerate(path):
            if i == k:
                continue
            ids = [int(tables[s, (first + x) // bs]) for x in (k, i)]
            if any(b <= 0 or b >= NB for b in ids):
                codes.add(5)
                continue
            moves.append((ids[0], (first + k) % bs, ids[1], (first + i) % bs))
        for p in pools:
            v = p.transpose(0, 2, 1, 3) if hm else p
            rows = [v[a, b].copy() for a, b, _, _ in moves]
            for (_, _, c, d), row in zip(moves, rows):
                v[c, d] = row
        new = first + len(path)
        lens[s] = new
        if refs is not None:
            for e in range(-(-new // bs), -(-L // bs)):
                b = int(tables[s, e])
                tables[s, e] = 0
                if b < 0 or b >= NB:
                    codes.add(5)
                elif b > 0:
                    if refs[b] > 0:
                        refs[b] -= 1
                    else:
                        codes.add(5)
    return codes
