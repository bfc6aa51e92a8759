"""Rotary positions, the append to a paged key/value cache, and attention over
it (oracle; test infrastructure only; fp64, one row at a time).

Results page, section 3: the target runs one forward pass over the K + 1
positions of the verify block.  Row r of sequence b (rows cu[b] .. cu[b+1]-1,
the newest of its ctx[b] tokens) sits at position p = ctx[b] - cu[b+1] + r;
position p is slot p % page of page table[b][p // page].

    rotation   (x0, x1) -> m (x0 cos t - x1 sin t, x1 cos t + x0 sin t),  t = p f_j
    attention  o = sum_{j <= p} softmax_j(scale q . k_j) v_j

A row before position 0 has no place; a row that sees no key gives zeros; a
key whose page lies outside the cache (or past the table) is neither stored
nor seen.
"""
import numpy as np


def rotate(x, position: int, inv_freq, mscale: float, interleaved: bool) -> np.ndarray:
    """fp64 [heads, d]: the heads of one row at ``position``."""
    y = np.asarray(x, np.float64).copy()
    rot = 2 * len(inv_freq)
    for j, f in enumerate(inv_freq):
        t = float(position) * float(f)
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        x0, x1 = y[:, a].copy(), y[:, b].copy()
        y[:, a] = mscale * (x0 * np.cos(t) - x1 * np.sin(t))
        y[:, b] = mscale * (x1 * np.cos(t) + x0 * np.sin(t))
    return y


def slot_of(table_row, position: int, page: int, num_pages: int):
    """(page, slot) of a position, or None where it has no place."""
    i = position // page
    if position < 0 or i >= len(table_row) or not 0 <= table_row[i] < num_pages:
        return None
    return int(table_row[i]), position % page


def rows_of(cu, ctx, b: int):
    """[(row, position)] of sequence b."""
    lo, hi = int(cu[b]), int(cu[b + 1])
    return [(r, int(ctx[b]) - hi + r) for r in range(lo, hi)]


def rope_append(qkv, k_cache, v_cache, table, cu, ctx, inv_freq, hq: int, mscale=1.0,
                interleaved=False):
    """(q fp64 [n, hq, d] with NaN in the rows that are not written, k_cache, v_cache fp64)."""
    pages, hkv, page, d = k_cache.shape
    x = np.asarray(qkv, np.float64)[:, :(hq + 2 * hkv) * d].reshape(len(qkv), hq + 2 * hkv, d)
    q = np.full((len(qkv), hq, d), np.nan)
    k, v = k_cache.astype(np.float64), v_cache.astype(np.float64)
    for b in range(len(ctx)):
        for r, p in rows_of(cu, ctx, b):
            if p < 0:
                continue
            y = rotate(x[r, :hq + hkv], p, inv_freq, mscale, interleaved)
            q[r] = y[:hq]
            at = slot_of(table[b], p, page, pages)
            if at is not None:
                k[at[0], :, at[1]] = y[hq:]
                v[at[0], :, at[1]] = x[r, hq + hkv:]
    return q, k, v


def attention(q, k_cache, v_cache, table, cu, ctx, scale: float):
    """(out fp64 [n, hq, d], NaN in rows of no sequence; spread fp64 [n, hq, d]: the sum of
    w |v|; reach fp64 [n, hq]: the largest sum of |q| |k| over a visible key; seen int [n])."""
    pages, hkv, page, d = k_cache.shape
    n, hq = q.shape[:2]
    g = hq // hkv
    out = np.full((n, hq, d), np.nan)
    spread = np.zeros((n, hq, d))
    reach = np.zeros((n, hq))
    seen = np.zeros(n, np.int64)
    for b in range(len(ctx)):
        at = [(p, slot_of(table[b], p, page, pages)) for p in range(max(int(ctx[b]), 0))]
        at = [(p, s) for p, s in at if s is not None]
        pos = np.array([p for p, _ in at], np.int64)
        pg = np.array([s[0] for _, s in at], np.int64)
        sl = np.array([s[1] for _, s in at], np.int64)
        for h in range(hkv):
            k = k_cache[pg, h, sl].astype(np.float64).reshape(-1, d)
            v = v_cache[pg, h, sl].astype(np.float64).reshape(-1, d)
            for r, p in rows_of(cu, ctx, b):
                m = pos <= p
                seen[r] = int(m.sum())
                for j in range(h * g, h * g + g):
                    if not m.any():
                        out[r, j] = 0.0
                        continue
                    x = q[r, j].astype(np.float64)
                    s = scale * (k[m] @ x)
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[r, j] = w @ v[m]
                    spread[r, j] = w @ np.abs(v[m])
                    reach[r, j] = (np.abs(k[m]) @ np.abs(x)).max()
    return out, spread, reach, seen
