"""Token sampling in 64 bits, for the tests: sort the row, walk the filters."""
import numpy as np


def sample_row(row, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, logprob) of one row of float64 logits; see bitdelta_sample for the definition."""
    x = np.where(np.isnan(row), -np.inf, row)
    order = np.argsort(-x, kind="stable")
    x = x[order]
    if np.isneginf(x[0]):
        return -1, -np.inf
    if not t > 0:
        return int(order[0]), 0.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == x[0], 1.0, np.exp((x - x[0]) / t))
    n = len(x) if k <= 0 else min(int(k), len(x))
    keep = n
    if p < 1:
        c = np.cumsum(w[:n])
        keep = min(keep, int(np.searchsorted(c, p * c[-1])) + 1)
    if m > 0:
        keep = min(keep, int((w >= m).sum()))
    keep = max(keep, 1)
    c = np.cumsum(w[:keep])
    j = min(int(np.searchsorted(c, max(u, 0.0) * c[-1], side="right")), keep - 1)
    return int(order[j]), float(np.log(w[j] / c[-1]))
