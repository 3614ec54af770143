"""Plain references of the drafted trees, a cache made of random rows, and the attention's tolerance."""
import numpy as np

import evictref


def ancestors(parents):
    """Rows [n, n] of the nodes that each node sees, itself among them; None where it hangs nowhere."""
    rows = []
    for i, a in enumerate(parents):
        row = None
        if a == -1:
            row = np.zeros(len(parents), bool)
        elif 0 <= a < i and rows[a] is not None:
            row = rows[a].copy()
        if row is not None:
            row[i] = True
        rows.append(row)
    return rows


def mask_words(parents):
    """int32 words [n, ceil(n / 32)], and the depth of each node (0 for one that hangs nowhere)."""
    n = len(parents)
    words = np.zeros((n, (n + 31) // 32), np.uint32)
    depth = np.zeros(n, np.int32)
    for i, row in enumerate(ancestors(parents)):
        if row is None:
            continue
        for j in np.flatnonzero(row):
            words[i, j // 32] |= np.uint32(1 << (j % 32))
        depth[i] = row.sum() - 1
    return words.view(np.int32), depth


def walk(parents, draft, target, expected):
    """The accepted path and the token behind it."""
    path, at, token = [], -1, expected
    while True:
        fits = [i for i in range(len(parents)) if parents[i] == at and i > at and draft[i] == token]
        if not fits:
            return path, token
        at = fits[0]
        path.append(at)
        token = target[at]


def words_of(sees):
    """int32 words [n, ceil(n / 32)] of truth values [n, n]."""
    n = len(sees)
    padded = np.zeros((n, (n + 31) // 32 * 32), np.uint8)
    padded[:, :n] = sees
    return np.ascontiguousarray(np.packbits(padded, axis=1, bitorder="little")).view(np.int32)


def random_rows(rng, shape):
    """72-byte NVFP4 rows [*shape, 72]: any code, positive scales from 0.25 to 0.9375."""
    rows = rng.integers(0, 256, (*shape, 72), dtype=np.uint8)
    rows[..., 64:] = rng.integers(0x28, 0x38, (*shape, 8), dtype=np.uint8)
    return rows


class Cache:
    """Random K and V rows [len, H, 144] of every sequence, in a pool whose other bytes are all ones
    (codes of -6, scales that are NaN), its pages scattered."""

    def __init__(self, lens, H, seed, spare=2, pages_behind=1):
        rng = np.random.default_rng(seed)
        self.lens, self.H = list(lens), H
        pages = [(n + 63) // 64 for n in lens]
        self.num_pages = sum(pages) + spare
        order = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(lens), max(pages) + pages_behind), -1, np.int32)
        self.pool = np.full((self.num_pages, 9216 * H), 0xFF, np.uint8)
        self.rows, at = [], 0
        for s, n in enumerate(lens):
            self.table[s, :pages[s]] = order[at:at + pages[s]]
            at += pages[s]
            self.rows.append(np.concatenate([random_rows(rng, (n, H)), random_rows(rng, (n, H))], -1))
        self.write()

    def write(self):
        off = evictref.row_offsets(self.H)
        for s, rows in enumerate(self.rows):
            t = np.arange(len(rows))
            page = self.table[s, t // 64]
            self.pool[page[:, None, None], off[:, t % 64].transpose(1, 0, 2)] = rows


def attend(q, rows, G, sees, sm_scale, good=None):
    """One sequence of n nodes. q [n, Hq, 128] fp64 values, rows [t, H, 144] of its cache, sees [n, n]
    of its nodes, which are the last n rows; good [t]: the row's page is in the pool. Returns the output
    [n, Hq, 128] and its error bound, which evictref.attend derives (the sums and roundings are the
    same); NaN where a visible key's stored K or V holds a NaN."""
    t, n, H = rows.shape[0], q.shape[0], rows.shape[1]
    nan = ((rows & 0x7F) == 0x7F)[..., np.r_[64:72, 136:144]].any(-1)  # [t, H]
    clean = rows.copy()
    clean[..., 64:72][nan] = 0
    clean[..., 136:144][nan] = 0
    k, v = evictref.values(clean[..., :72]), evictref.values(clean[..., 72:])
    ok = np.ones(t, bool) if good is None else good
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for i in range(n):
        see = ok & np.concatenate([np.ones(t - n, bool), sees[i]])
        if not see.any():
            continue
        for g in range(q.shape[1]):
            h = g // G
            if nan[see, h].any():
                out[i, g] = np.nan
                continue
            s = k[see, h] @ q[i, g] * sm_scale
            a = (np.abs(k[see, h]) @ np.abs(q[i, g]) * sm_scale).max()
            p = np.exp(s - s.max())
            p /= p.sum()
            d = 2.0 ** -19 * a + 2.0 ** -16
            out[i, g] = p @ v[see, h]
            tol[i, g] = ((2 * d + 2.0 ** -10) * (p @ np.abs(v[see, h]))
                         + 2.0 ** -25 * np.abs(v[see, h]).sum(0))
    return out, tol + 2.0 ** -8 * (np.abs(out) + tol) + 1e-30


def accept(cache, parents, draft, target, expected, held):
    """Paths, their next tokens and the pool afterwards, of every sequence."""
    pool, off = cache.pool.copy(), evictref.row_offsets(cache.H)
    paths, tokens = [], []
    for s, base in enumerate(held):
        path, token = walk(parents[s], draft[s], target[s], expected[s])
        paths.append(path)
        tokens.append(token)
        move(cache.pool, pool, cache.table[s], off, path, base)
    return paths, tokens, pool


def move(old, new, table, off, path, base):
    """Rows base + path[j] of a sequence to base + j."""
    for j, i in enumerate(path):
        a, b = base + i, base + j
        if 0 <= table[a // 64] < len(old) and 0 <= table[b // 64] < len(old):
            new[table[b // 64], off[:, b % 64]] = old[table[a // 64], off[:, a % 64]]


def random_tree(rng, n, padding=0.0):
    """Parents [n]: mostly one root, chains and branches, and (with a probability) nodes that hang
    nowhere."""
    parents = np.empty(n, np.int32)
    for i in range(n):
        u = rng.random()
        parents[i] = -1 if i == 0 or u < 0.05 else i - 1 if u < 0.5 else rng.integers(0, i)
        if rng.random() < padding:
            parents[i] = rng.choice([-2, i, n, 2 ** 31 - 1, -2 ** 31])
    return parents
