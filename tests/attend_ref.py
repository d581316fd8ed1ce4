"""Plain 64-bit attention over a paged cache, for the tests: every key of a table, one by one."""
import numpy as np


def cache_rows(pages, table_row, length, page_size, scale):
    """(rows [length, kv_heads, dim] float64, present [length]) of a sequence; ``pages`` is a
    float64 array [pages, page_size, kv_heads, dim].  A key whose page id is not a page is absent
    (its row is zeros)."""
    n = min(max(int(length), 0), len(table_row) * page_size)
    out = np.zeros((n,) + pages.shape[2:])
    present = np.zeros(n, dtype=bool)
    for t in range(n):
        page = int(table_row[t // page_size])
        if 0 <= page < pages.shape[0]:
            out[t] = pages[page, t % page_size] * scale
            present[t] = True
    return out, present


def attend(q, k, v, seen, scale):
    """q [heads, dim], k and v [n, kv_heads, dim], seen [n] -> (out, sum of weights times |v|,
    sum of |q||k| scale at its largest, lse), all float64."""
    heads, dim = q.shape
    group = heads // k.shape[1] if k.shape[1] else 1
    out, mix = np.zeros((heads, dim)), np.zeros((heads, dim))
    lse = np.full(heads, -np.inf)
    keys = np.flatnonzero(seen)
    if keys.size == 0:
        return out, mix, lse
    for h in range(heads):
        kk, vv = k[keys, h // group], v[keys, h // group]
        s = (kk @ q[h]) * scale
        top = s.max()
        w = np.exp(s - top)
        lse[h] = top + np.log(w.sum())
        w /= w.sum()
        out[h] = w @ vv
        mix[h] = w @ np.abs(vv)
    return out, mix, lse
