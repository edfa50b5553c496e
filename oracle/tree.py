"""Plain 64-bit restatement of the drafted-tree operators and the eviction:
numpy, one loop a sequence and head, written from their definitions and
sharing nothing with the CUDA library.  Caches come as the real numbers they
hold ([pages, page_size, H, D] float64); moves act on any row array.
"""
import numpy as np


def e4m3_values(codes):
    """uint8 E4M3 codes -> float64 (0x7f, 0xff: NaN)."""
    c = np.asarray(codes).astype(np.int64)
    exp, man = (c >> 3) & 15, c & 7
    v = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * np.exp2(exp - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def mx_values(codes, scales):
    """MXFP8 rows -> float64: code * 2^(scale - 127), blocks of 32."""
    x = np.exp2(np.asarray(scales).astype(np.float64) - 127)
    return e4m3_values(codes) * np.repeat(x, 32, axis=-1)


def paths(parents):
    """Each token's list of ancestors, root first, itself last; [] for an
    unused one (its chain of parents does not go down to -1)."""
    out = []
    for j, p in enumerate(parents):
        if p >= j or p < -1 or (p >= 0 and not out[p]):
            out.append([])
        else:
            out.append((out[p] if p >= 0 else []) + [j])
    return out


def rows_of(cache, table_row, positions, page_size):
    positions = np.asarray(positions, dtype=np.int64)
    return cache[np.asarray(table_row)[positions // page_size], positions % page_size]


def attention(q, cu, parents, lens, table, k_cache, v_cache, scale):
    """q [T, HQ, D] float64.  Returns out, lse, and bounds for the tests: the
    sum of p |v|, and the largest sum |q_d k_d| * scale over what a row sees."""
    T, HQ, D = q.shape
    H, P = k_cache.shape[2], k_cache.shape[1]
    g = HQ // H
    out, lse = np.zeros((T, HQ, D)), np.full((T, HQ), -np.inf)
    mag, size = np.zeros((T, HQ, D)), np.zeros((T, HQ))
    for i in range(len(lens)):
        a, n, ctx = cu[i], cu[i + 1] - cu[i], int(lens[i])
        k = rows_of(k_cache, table[i], np.arange(ctx + n), P)
        v = rows_of(v_cache, table[i], np.arange(ctx + n), P)
        for j, path in enumerate(paths(parents[a:a + n])):
            if not path:
                continue
            see = np.concatenate([np.arange(ctx), ctx + np.array(path, dtype=np.int64)])
            for hq in range(HQ):
                kk, vv = k[see, hq // g], v[see, hq // g]
                s = kk @ q[a + j, hq] * scale
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                out[a + j, hq] = (p / z) @ vv
                lse[a + j, hq] = m + np.log(z)
                mag[a + j, hq] = (p / z) @ np.abs(vv)
                size[a + j, hq] = (np.abs(kk) @ np.abs(q[a + j, hq])).max() * abs(scale)
    return out, lse, mag, size


def weights(q, lse, cu, parents, lens, table, k_cache, scale, w):
    """The new weights [S, H, positions], and the largest sum |q_d k_d| * scale."""
    T, HQ, D = q.shape
    H, P = k_cache.shape[2], k_cache.shape[1]
    g = HQ // H
    w = np.array(w, dtype=np.float64)
    size = 0.0
    for i in range(len(lens)):
        a, n, ctx = cu[i], cu[i + 1] - cu[i], int(lens[i])
        w[i, :, ctx:ctx + n] = 0
        k = rows_of(k_cache, table[i], np.arange(ctx + n), P)
        for j, path in enumerate(paths(parents[a:a + n])):
            if not path:
                continue
            see = np.concatenate([np.arange(ctx), ctx + np.array(path, dtype=np.int64)])
            for hq in range(HQ):
                if lse[a + j, hq] == -np.inf:
                    continue
                h = hq // g
                w[i, h, see] += np.exp(k[see, h] @ q[a + j, hq] * scale - lse[a + j, hq])
                size = max(size, (np.abs(k[see, h]) @ np.abs(q[a + j, hq])).max() * abs(scale))
    return w, size


def windows(cu, parents, W):
    """For every used packed token its window, oldest first: packed token
    indices, or r - (W - 1) (negative) for row r of the sequence's state."""
    out = {}
    for i in range(len(cu) - 1):
        a = cu[i]
        for j, path in enumerate(paths(parents[a:cu[i + 1]])):
            if path:
                line = [r - (W - 1) for r in range(W - 1)] + [a + t for t in path]
                out[a + j] = (i, line[-W:])
    return out


def evict_pick(w, length, keep, sinks, recent):
    """Kept positions, ascending, of one (sequence, head)."""
    if length <= keep:
        return list(range(length))
    held = list(range(sinks)) + list(range(length - recent, length))

    def rank(p):
        x = w[p]
        return (0, 0.0, p) if np.isnan(x) else (1, -float(x), p)

    rest = sorted(range(sinks, length - recent), key=rank)
    return sorted(held + rest[:keep - sinks - recent])


def place(table_row, p, page_size):
    return table_row[p // page_size], p % page_size
