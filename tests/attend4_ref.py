"""Plain forms for the log-sums of 4-bit attention: how a query is held, and queries and keys that show it.

The kernels hold a query's blocks of 32 dims as four e2m3 numbers, 0, 4, 9 and 14 binary places below the
block's scale; what all four leave is at most 2^-19 of the block's largest value."""
import numpy as np

SHIFTS = (0, 4, 9, 14)


def e2m3(x):
    """float64 values rounded to e2m3, to nearest, ties to even, at most 7.5."""
    a = np.abs(x)
    step = np.where(a < 2, 0.125, np.where(a < 4, 0.25, 0.5))
    return np.copysign(np.minimum(np.rint(a / step) * step, 7.5), x)


def held(q, parts=4):
    """float64 values [..., n] as their first `parts` numbers hold them."""
    x = np.asarray(q, np.float64).reshape(*np.shape(q)[:-1], -1, 32)
    top = np.abs(x).max(-1, keepdims=True)
    e = np.ceil(np.log2(np.where(top > 0, top, 1.0) / 7.5))
    left, sum_ = x, np.zeros_like(x)
    for shift in SHIFTS[:parts]:
        unit = np.exp2(e - shift)
        v = e2m3(left / unit) * unit
        left, sum_ = left - v, sum_ + v
    return sum_.reshape(np.shape(q))


def fine_queries(rng, tokens, heads, dim):
    """bf16 queries: in each block one value of 4 to 7, the others of some 2^-8 so that the first three numbers
    leave 12 * 2^-17 of each."""
    q = (131 + 16 * rng.integers(0, 8, (tokens, heads, dim // 32, 32))) * 2.0 ** -15
    at = rng.integers(0, 32, q.shape[:-1])
    np.put_along_axis(q, at[..., None], rng.choice([4.0, 5.0, 6.0, 7.0], at.shape)[..., None], -1)
    return q.reshape(tokens, heads, dim)


def score_bound(q, k, scale):
    """How far one score of query q [dim] and key k [dim] may be from scale * (q . k): sums of dim fp32 terms,
    and what the four numbers leave of each value."""
    return scale * ((q.shape[-1] + 16) * 2.0 ** -24 * (np.abs(q) @ np.abs(k)) + np.abs(q - held(q)) @ np.abs(k))
