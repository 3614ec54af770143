"""Plain 64-bit references of the eviction operators, and their tolerances, for the tests."""
import numpy as np

import oracle


def row_offsets(H):
    """Byte offsets [H, 64, 144] in a page block of each slot's K codes, K scales, V codes and V
    scales, from the pool layout in the header."""
    off = np.empty((H, 64, 144), np.int64)
    for h in range(H):
        for k in range(64):
            j, b = np.arange(64), np.arange(8)
            off[h, k, :64] = 4096 * h + k // 8 * 512 + j // 16 * 128 + k % 8 * 16 + j % 16
            if h // 2 * 2 + 1 < H:
                off[h, k, 64:72] = (4096 * H + 1024 * (h // 2) + 512 * (b // 4) + 16 * (k % 32)
                                    + 8 * (h % 2) + 4 * (k // 32) + b % 4)
            else:
                off[h, k, 64:72] = (4096 * H + 1024 * (h // 2) + 256 * (b // 4) + 8 * (k % 32)
                                    + 4 * (k // 32) + b % 4)
            off[h, k, 72:136] = 4608 * H + 4096 * h + 64 * k + j
            off[h, k, 136:] = 8704 * H + 512 * h + 8 * k + b
    return off


def cache_rows(pool, table, H, seq, slots):
    """Rows [n, H, 144] of a sequence's slots (pool [num_pages, 9216 H])."""
    off = row_offsets(H)
    slots = np.asarray(slots)
    page = table[seq, slots // 64]
    return pool[page[:, None, None], off[:, slots % 64].transpose(1, 0, 2)]


def values(rows):
    """fp64 values [..., 128] of 72-byte NVFP4 rows (64 code bytes, 8 scales)."""
    flat = np.ascontiguousarray(rows.reshape(-1, 72))
    x = oracle.dequant_rows(np.ascontiguousarray(flat[:, :64]), np.ascontiguousarray(flat[:, 64:]))
    return np.asarray(x, np.float64).reshape(*rows.shape[:-1], 128)


def attend(q, rows, G, q_len, causal, sm_scale, good=None):
    """One sequence. q [q_len, Hq, 128] fp64 values, rows [n, H, 144] of its cache. Returns the
    output [q_len, Hq, 128], the weight sums [H, n], and their error bounds.

    Bounds. A score is a sum of 8 exactly computed 16-element block products; its fp32 sum is off by
    at most 8 steps of 2^-23 (a truncating accumulator) of A = sum |q_j k_j| sm_scale. The
    difference to the row's maximum doubles that, and its product with log2 e, the exponential
    (2^-22) and the sums over keys (64 sequential additions in a lane or fewer, then a tree) add
    less than 2^-16: a probability is off by at most a factor 1 + d, d = 2^-19 A + 2^-16. P enters
    the output product in f16 (half a step: 2^-11 relative, also in its sum on the tile kernel;
    below 2^-14 f16 has steps of 2^-24, so half of one more per key, against a sum of P that is at
    least 1: the largest P of a row is), and the output is rounded to bf16 (half a step: 2^-8
    relative)."""
    n, H = rows.shape[0], rows.shape[1]
    k, v = values(rows[..., :72]), values(rows[..., 72:])
    ok = np.ones(n, bool) if good is None else good
    out = np.zeros_like(q)
    tol = np.zeros_like(q)
    w, wtol = np.zeros((H, n)), np.zeros((H, n))
    for h in range(H):
        for i in range(q_len):
            for g in range(h * G, h * G + G):
                sees = ok & ((np.arange(n) <= n - q_len + i) if causal else True)
                if not sees.any():
                    continue
                s = k[:, h] @ q[i, g] * sm_scale
                a = (np.abs(k[:, h]) @ np.abs(q[i, g]) * sm_scale)[sees].max()
                p = np.where(sees, np.exp(s - s[sees].max()), 0)
                p /= p.sum()
                d = 2.0 ** -19 * a + 2.0 ** -16
                out[i, g] = p @ v[:, h]
                tol[i, g] = ((2 * d + 2.0 ** -10) * (p @ np.abs(v[:, h]))
                             + 2.0 ** -25 * np.abs(v[sees, h]).sum(0))
                w[h] += p
                wtol[h] += 2 * d * p
    return out, tol + 2.0 ** -8 * (np.abs(out) + tol) + 1e-30, w, wtol


def select(w, length, keep, sink, recent):
    """Kept slots of one set, ascending: w [stride] fp32."""
    kept = min(length, keep)
    t = np.arange(length)
    x = w[:length].astype(np.float64)
    rank = np.where(np.isnan(x), -np.inf, np.where(x == -np.inf, -1e300, x))  # NaN below -inf
    rest = ~((t < sink) | (t >= length - recent))
    # lexsort's last key comes first: protected slots (by slot alone), then numbers, then NaN
    order = np.lexsort((t, np.where(rest, -rank, 0), rest & np.isnan(x), rest))
    return np.sort(order[:kept])


def head_sum(w):
    """The heads' weights added in fp32, head 0 first: w [H, n]."""
    s = w[0].astype(np.float32)
    for x in w[1:]:
        s = (s + x).astype(np.float32)
    return s


def compact(pool, table, dst_table, H, index, lens, keep, weights):
    """New pool (bytes) and weights: index [S, H, n], pool [num_pages, 9216 H]."""
    off = row_offsets(H)
    new, w = pool.copy(), None if weights is None else weights.copy()
    for s, (n, m) in enumerate(zip(lens, keep)):
        m = min(n, m)
        j = np.arange(m)
        for h in range(H):
            t = index[s, h, :m]
            new[dst_table[s, j // 64][:, None], off[h, j % 64]] = \
                pool[table[s, t // 64][:, None], off[h, t % 64]]
            if w is not None:
                w[s, h, :m] = weights[s, h, t]
                w[s, h, m:n] = 0
    return new, w
