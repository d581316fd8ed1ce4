"""Attention over a 4-bit paged cache on the GPU against the plain 64-bit form.

Tolerances, per output element: the result is rounded to bf16 once (half a step, 2^-8 of it) and each
weight once (2^-8 of the weight, so 2^-8 of sum w |v|).  A score is a sum of dim fp32 terms, off by at most
(dim + 16) 2^-24 of the sum of |q||k|, and its query may be held in two parts of 4 bits each of a row's
largest |q|, which are off by at most 2^-17 of that: both are worked out from the inputs (score_error),
and move every weight by that share; so do fp32 exponentials, 2^-20.  The log-sum is off by the score
error plus fp32 rounding."""
import numpy as np
import pytest

import cache_ref as R
import test_gpu_attend as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

BF16 = 2.0 ** -8
EXP = 2.0 ** -20
i32 = A.i32


@pytest.fixture(autouse=True)
def _announce(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"\n[gpu case] {request.node.nodeid}", flush=True)
    yield
    torch.cuda.synchronize()


class Cache4:
    """Pages of normal values in 4 bits (keys with some large channels), head-major ("head"), token-major
    ("token"), or keys and values of a page side by side ("joint")."""

    def __init__(self, rng, pages, page, hk, dim, layout="head", spread=True):
        self.codes, self.byte = [], []
        for which in range(2):
            x = rng.normal(size=(pages, page, hk, dim))
            if which == 0:
                x[..., 5::32] *= 4.0
            elif spread:
                x *= np.exp2(rng.integers(-3, 4, (pages, page, hk, 1)))
            c, b = R.encode4(x)
            self.codes.append(c)
            self.byte.append(b)
        self.layout = layout
        self.upload()

    def upload(self):
        def place(kv):
            kv = [torch.from_numpy(np.ascontiguousarray(x)) for x in kv]
            if self.layout == "token":
                return [x.cuda() for x in kv]
            if self.layout == "head":
                return [x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in kv]
            both = torch.stack([x.transpose(1, 2) for x in kv], 1).contiguous().cuda()
            return [both[:, i].transpose(1, 2) for i in range(2)]

        self.k, self.v = place([R.pack4(c) for c in self.codes])
        self.kb, self.vb = place(self.byte)
        self.kf, self.vf = (R.decode4(c, b) for c, b in zip(self.codes, self.byte))

    def kw(self):
        return {"k_block_scales": self.kb, "v_block_scales": self.vb}


def rows(values, table_row, length, page, scale):
    """(float64 rows of a sequence's first `length` tokens times scale, which are there)."""
    n = min(max(int(length), 0), len(table_row) * page)
    t = np.arange(n)
    pid = np.asarray(table_row, np.int64)[t // page] if n else np.zeros(0, np.int64)
    ok = (pid >= 0) & (pid < values.shape[0])
    out = np.zeros((n,) + values.shape[2:])
    out[ok] = values[pid[ok], t[ok] % page] * scale
    return out, ok


def attend(q, k, v, seen, scale):
    """(out, sum of weights times |v|, log-sum, score error) of one query row per head."""
    heads, dim = q.shape
    group = heads // k.shape[1]
    out, mix = np.zeros((heads, dim)), np.zeros((heads, dim))
    lse, err = np.full(heads, -np.inf), np.zeros(heads)
    keys = np.flatnonzero(seen)
    if keys.size:
        for h in range(heads):
            kk, vv = k[keys, h // group], v[keys, h // group]
            s = (kk @ q[h]) * scale
            w = np.exp(s - s.max())
            lse[h] = s.max() + np.log(w.sum())
            w /= w.sum()
            out[h], mix[h] = w @ vv, w @ np.abs(vv)
            ak, aq = np.abs(kk), np.abs(q[h])
            err[h] = scale * np.max((dim + 16) * 2.0 ** -24 * (ak @ aq) + 2.0 ** -17 * aq.max() * ak.sum(1))
    return out, mix, lse, err


def check(out, lse, ref):
    got, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t, (o, mix, l, err) in enumerate(ref):
        share = BF16 + (2 * err + EXP)[:, None]
        tol = BF16 * np.abs(o) + share * mix + 1e-30
        assert np.array_equal(np.isnan(got[t]), np.isnan(o)), f"token {t}"
        fine = ~np.isnan(o)
        worst = np.where(fine, np.abs(got[t] - o) - tol, -1.0)
        assert worst.max() <= 0, (t, np.unravel_index(worst.argmax(), worst.shape), worst.max())
        dead = np.isneginf(l)
        assert np.array_equal(np.isneginf(z[t]), dead), (t, z[t], l)
        assert np.array_equal(np.isnan(z[t]), np.isnan(l)), (t, z[t], l)
        live = ~dead & ~np.isnan(l)
        off = np.abs(z[t][live] - l[live])
        assert np.all(off <= err[live] + 2e-6 + 1e-6 * np.abs(l[live])), (t, z[t], l, err)


def shared_ref(q, c, page, table, lens, ptable, plens, offs, scales, scale):
    ref = []
    for g in range(len(offs) - 1):
        pk, pp = rows(c.kf, ptable[g], plens[g], page, scales[0])
        pv, _ = rows(c.vf, ptable[g], plens[g], page, scales[1])
        for b in range(offs[g], offs[g + 1]):
            k, p = rows(c.kf, table[b], lens[b], page, scales[0])
            v, _ = rows(c.vf, table[b], lens[b], page, scales[1])
            ref.append(attend(q[b], np.concatenate([pk, k]), np.concatenate([pv, v]),
                              np.concatenate([pp, p]), scale))
    return ref


def window_ref(q, c, page, table, lens, q_lens, window, sinks, scales, scale):
    ref, at = [], 0
    for b, n in enumerate(q_lens):
        length = min(max(lens[b], 0), table.shape[1] * page)
        k, p = rows(c.kf, table[b], length, page, scales[0])
        v, _ = rows(c.vf, table[b], length, page, scales[1])
        j = np.arange(length)
        for i in range(n):
            pos = length - n + i
            ref.append(attend(q[at + i], k, v, p & (j <= pos) & ((pos - j < window) | (j < sinks)), scale))
        at += n
    return ref


SCALES = [(1.0, 1.0), (0.5, 3.0), (1.7, 0.3)]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("case", range(len(A.SHARED)))
def test_shared(case, tiles):
    """(tiles: with prefix tables so wide that sharing the prefixes is worth a launch)"""
    sizes, plens, olens, heads, hk, dim, page, _, extra, layout = A.SHARED[case]
    rng = np.random.default_rng(case + 50 * tiles)
    n = sum(sizes)
    lens = [olens[(i + tiles) % len(olens)] for i in range(n)]
    offs = np.concatenate([[0], np.cumsum(sizes)])
    need = sum(-(-x // page) for x in lens + plens)
    free = list(rng.permutation(need + 3))
    table = A.tables(rng, lens, page, max(-(-max(lens) // page), 0) + extra, free)
    ptable = A.tables(rng, plens, page, max(-(-max(plens) // page), 0) + (0 if tiles else extra), free)
    if tiles:
        if plens[0] > page:  # a page that is none
            ptable[0, 1] = need + 3
        if n > sum(m > 0 for m in sizes):
            ptable = A.widen(ptable, sizes, page, hk, dim // 2, "fp8")
            if (ptable.shape[1] + table.shape[1]) * page > 1 << 30:
                pytest.skip("a table that wide is refused")
    c = Cache4(rng, need + 3, page, hk, dim, layout)
    q, qf = A.make_q(rng, n, heads, dim)
    sc = SCALES[case % 3]
    out, lse = bd.attend_shared(q, c.k, c.v, i32(table), i32(lens), i32(ptable), i32(plens), offs,
                                k_scale=sc[0], v_scale=sc[1], return_lse=True, **c.kw())
    check(out, lse, shared_ref(qf, c, page, table, lens, ptable, plens, offs, sc, dim ** -0.5))


@pytest.mark.parametrize("case", range(len(A.WINDOW)))
def test_window(case):
    q_lens, lens, heads, hk, dim, page, _, window, sinks, extra, layout = A.WINDOW[case]
    rng = np.random.default_rng(100 + case)
    need = sum(-(-x // page) for x in lens)
    free = list(rng.permutation(need + 2))
    table = A.tables(rng, lens, page, -(-max(lens) // page) + extra, free)
    c = Cache4(rng, need + 2, page, hk, dim, "joint" if case % 3 == 2 else layout)
    q, qf = A.make_q(rng, sum(q_lens), heads, dim)
    single = all(n == 1 for n in q_lens)
    offs = None if single else i32(np.concatenate([[0], np.cumsum(q_lens)]))
    sc = SCALES[case % 3]
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), k_scale=sc[0], v_scale=sc[1],
                                return_lse=True, **c.kw())
    check(out, lse, window_ref(qf, c, page, table, lens, q_lens, window, sinks, sc, dim ** -0.5))


# chunks whose units' keys are split into parts: new tokens, tokens with them, heads, kv heads, dim, window,
# sinks, table pages beyond need, and rows to look at (None: all)
SPLIT = [
    ([100], [3000], 8, 2, 128, 5000, 0, 0, None),
    ([33, 70, 0, 1], [5000, 2000, 40, 1], 12, 4, 64, 3000, 5, 9, None),
    ([9, 40], [700, 30], 16, 1, 128, 1200, 2, 500, None),  # parts without keys
    ([1056], [2600], 64, 4, 128, 1400, 4, 0, 61),          # 264 units: 8 of them split
    ([700, 400], [700, 900], 32, 8, 64, 4096, 0, 0, 41),
]


@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_chunks_split_over_workgroups(case):
    q_lens, lens, heads, hk, dim, window, sinks, extra, some = SPLIT[case]
    rng = np.random.default_rng(300 + case)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, heads, hk, dim, extra=extra)
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    assert bd.attend_window_workspace_bytes(c.k, heads, i32(table), sum(q_lens), max(q_lens), window, sinks) > 0
    n = sum(q_lens)
    pick = range(n) if some is None else sorted({0, 1, n - 1, *range(0, n, n // some)})
    at, ref = 0, {}
    for b, m in enumerate(q_lens):
        length = lens[b]
        k, p = rows(c.kf, table[b], length, 16, 1.0)
        v, _ = rows(c.vf, table[b], length, 16, 1.0)
        j = np.arange(length)
        for t in pick:
            if at <= t < at + m:
                pos = length - m + t - at
                ref[t] = attend(qf[t], k, v, p & (j <= pos) & ((pos - j < window) | (j < sinks)), dim ** -0.5)
        at += m
    pick = list(pick)
    check(out[pick], lse[pick], [ref[t] for t in pick])


def _setup(rng, q_lens, lens, heads=8, hk=2, dim=128, page=16, extra=0):
    need = sum(-(-x // page) for x in lens) + 1
    free = list(rng.permutation(need))
    table = A.tables(rng, lens, page, -(-max(lens) // page) + extra, free)
    c = Cache4(rng, need, page, hk, dim)
    q, qf = A.make_q(rng, sum(q_lens), heads, dim)
    return table, c, q, qf, i32(np.concatenate([[0], np.cumsum(q_lens)]))


# single tokens unsplit and split over workgroups, a few tokens, row tiles
KINDS = [([1, 1], [900, 40]), ([1, 1], [1900, 40]), ([2, 3], [1900, 40]), ([80, 20], [300, 40])]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_pages_that_are_no_pages(q_lens, lens, dim):
    rng = np.random.default_rng(5)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, dim=dim, extra=60)
    table[0, 3], table[1, 0], table[0, -60 - 2] = -1, c.k.shape[0], 2 ** 31 - 1
    table[0, 11] = -2 ** 31
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 4000, 2, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    check(out, lse, window_ref(qf, c, 16, table, lens, q_lens, 4000, 2, (1, 1), dim ** -0.5))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_absent_keys_read_nothing_of_page_0(q_lens, lens, dim):
    """Page 0, which belongs to nobody, holds NaN; keys without a page and behind the lists are absent."""
    rng = np.random.default_rng(25)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, dim=dim, extra=60)
    free = list(set(range(c.kf.shape[0])) - set(table[table >= 0].tolist()))[0]
    table = np.where(table == 0, free, table)
    table[0, 2], table[1, 1] = -1, 10 ** 6
    for x in c.byte:
        x[0] = 255
    for x in c.codes:
        x[free] = x[1]
    c.byte[0][free], c.byte[1][free] = c.byte[0][1], c.byte[1][1]
    c.upload()
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 4000, 2, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    check(out, lse, window_ref(qf, c, 16, table, lens, q_lens, 4000, 2, (1, 1), dim ** -0.5))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_keys_and_values_laid_out_differently(q_lens, lens, dim):
    """Keys head by head, values token by token, in pages and heads of an odd number."""
    rng = np.random.default_rng(26)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, heads=9, hk=3, dim=dim, page=7)
    t = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    u = lambda x: x.contiguous()                                 # noqa: E731
    out, lse = bd.attend_window(q, t(c.k), u(c.v), i32(table), i32(lens), 1500, 2, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, k_block_scales=t(c.kb),
                                v_block_scales=u(c.vb))
    check(out, lse, window_ref(qf, c, 7, table, lens, q_lens, 1500, 2, (1, 1), dim ** -0.5))


@pytest.mark.parametrize("heads,hk,dim", [(40, 1, 128), (64, 1, 64), (96, 2, 128)])
def test_single_tokens_of_many_heads(heads, hk, dim):
    """More than 32 query heads a kv head: single tokens by the tile kernel, prefixes by both."""
    rng = np.random.default_rng(27)
    lens = [1400, 0, 33]
    table, c, q, qf, _ = _setup(rng, [1, 1, 1], lens, heads, hk, dim)
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 1000, 4, return_lse=True, **c.kw())
    check(out, lse, window_ref(qf, c, 16, table, lens, [1, 1, 1], 1000, 4, (1, 1), dim ** -0.5))
    out, lse = bd.attend_shared(q, c.k, c.v, i32(table), i32(lens), None, None, [0, 2, 3], return_lse=True, **c.kw())
    check(out, lse, window_ref(qf, c, 16, table, lens, [1, 1, 1], 10 ** 6, 0, (1, 1), dim ** -0.5))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
@pytest.mark.parametrize("window", [37, 4000])
def test_what_no_query_sees_is_not_used(q_lens, lens, window, dim):
    """Blocks of NaN before the windows, beyond the lengths, in the pages of nobody."""
    rng = np.random.default_rng(7)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, dim=dim)
    sinks = 3
    seen = np.zeros(c.kf.shape[:2], bool)
    for b, n in enumerate(q_lens):
        for i in range(n):
            pos = lens[b] - n + i
            for j in range(pos + 1):
                if pos - j < window or j < sinks:
                    seen[table[b, j // 16], j % 16] = True
    ref = window_ref(qf, c, 16, table, lens, q_lens, window, sinks, (1, 1), dim ** -0.5)
    for x in (*c.byte, ):
        x[~seen] = 255
    c.upload()
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    check(out, lse, ref)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_blocks_of_nan_reach_the_rows_that_see_them(q_lens, lens, which, dim):
    """A key's NaN makes the rows NaN that see it, a value's the 32 dims of its block of those."""
    rng = np.random.default_rng(11)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, dim=dim)
    for b, n in enumerate(q_lens):
        at = lens[b] - max(1, n // 2)  # seen by some rows of the chunk only
        c.byte[which][table[b, at // 16], at % 16, b % 2, b % (dim // 32)] = 255
        at = lens[b] - n - 9           # leaves the window in the chunk
        if at >= 0:
            c.byte[which][table[b, at // 16], at % 16, 1 - b % 2, 1] = 255
    c.upload()
    window = 9 + max(q_lens) // 2
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), window, 0, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    ref = window_ref(qf, c, 16, table, lens, q_lens, window, 0, (1, 1), dim ** -0.5)
    got, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t, (o, mix, l, err) in enumerate(ref):
        assert np.array_equal(np.isnan(got[t]), np.isnan(o)), t
        # (a log-sum over NaN scores is NaN; over NaN values it is not)
        assert np.array_equal(np.isnan(z[t]), np.isnan(l)), t
    if which == 1:
        check(out, lse, ref)


@pytest.mark.parametrize("dim", [64, 128])
def test_extreme_scales_and_queries(dim):
    """Blocks of a row 2^200 apart; queries of one large and many small values; rows of zeros."""
    rng = np.random.default_rng(13)
    n = 700
    table, c, q, qf, offs = _setup(rng, [1, 3], [n, n], dim=dim)
    c.byte[0][..., 1] -= 100
    c.byte[0][::3, ..., 0] -= 20
    c.byte[1][..., 0] = 2     # the smallest that are written
    c.byte[1][..., 1] = 200
    c.codes[1][..., -1] = 0
    c.upload()
    x = q.float()
    x[0] *= 1e-6
    x[0, :, 7] = 3.0
    x[1] = 0.0
    x[2] *= 2.0 ** -30
    q = x.bfloat16()
    qf = q.double().cpu().numpy()
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32([n, n]), 5000, 0, q_offsets=offs, max_q_len=3,
                                return_lse=True, **c.kw())
    check(out, lse, window_ref(qf, c, 16, table, [n, n], [1, 3], 5000, 0, (1, 1), dim ** -0.5))


def test_queries_that_are_not_finite():
    """Such a row is NaN; the others are not touched by it."""
    rng = np.random.default_rng(14)
    for q_lens, lens in KINDS:
        table, c, q, qf, offs = _setup(rng, q_lens, lens)
        want = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 5000, 0, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
        bad = q.clone()
        bad[0, 3, 5], bad[1, 0, 127], bad[-1, 7, 0] = float("nan"), float("inf"), float("-inf")
        got = bd.attend_window(bad, c.k, c.v, i32(table), i32(lens), 5000, 0, q_offsets=offs,
                               max_q_len=max(q_lens), return_lse=True, **c.kw())
        hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        hit[0, 3] = hit[1, 0] = hit[-1, 7] = True
        assert torch.isnan(got[0][hit]).all() and torch.isnan(got[1][hit]).all()
        assert torch.equal(got[0][~hit], want[0][~hit]) and torch.equal(got[1][~hit], want[1][~hit])


def test_offsets_beyond_32_bits():
    hk, dim, page = 2, 128, 16
    apart = (1 << 32) + (1 << 12)
    raw = [torch.zeros(apart + (1 << 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    blocks = [torch.zeros(apart // 16 + (1 << 12), dtype=torch.uint8, device="cuda") for _ in "kv"]
    pages = [t.as_strided((2, page, hk, dim // 2), (apart, dim // 2, page * dim // 2, 1)) for t in raw]
    small = [t.as_strided((2, page, hk, dim // 32), (apart // 16, dim // 32, page * dim // 32, 1)) for t in blocks]
    rng = np.random.default_rng(4)
    c = Cache4(rng, 2, page, hk, dim)
    for big, x in zip((*pages, *small), (c.k, c.v, c.kb, c.vb)):
        big.copy_(x)
    table, lens = i32([[1, 0]] * 40), i32([30] * 40)
    q, qf = A.make_q(rng, 40, 8, dim)
    kw = dict(k_block_scales=small[0], v_block_scales=small[1], return_lse=True)
    for extra in (dict(), dict(q_offsets=i32([0, 40]), max_q_len=40)):
        t, l = (table[:1].contiguous(), i32([32])) if extra else (table, lens)
        got = bd.attend_window(q, *pages, t, l, 64, 0, **extra, **kw)
        want = bd.attend_window(q, c.k, c.v, t, l, 64, 0, **extra, return_lse=True, **c.kw())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_like_a_bf16_cache_of_the_same_values(q_lens, lens, dim):
    """cache_read's values in a bf16 cache give the same attention: the two roundings to bf16 and the
    weights' aside, which each side has once."""
    rng = np.random.default_rng(15)
    table, c, q, qf, offs = _setup(rng, q_lens, lens, dim=dim)
    pages, page, hk = c.kf.shape[:3]
    every = i32(np.arange(pages)[:, None])
    full = i32([page] * pages)
    at = i32(np.arange(pages + 1) * page)
    k, v = bd.cache_read(c.k, c.v, every, full, q_offsets=at, tokens=pages * page, **c.kw())
    assert np.array_equal(k.double().cpu().numpy().reshape(c.kf.shape), c.kf)
    a = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 700, 2, q_offsets=offs, max_q_len=max(q_lens),
                         return_lse=True, **c.kw())
    b = bd.attend_window(q, k.view(pages, page, hk, dim), v.view(pages, page, hk, dim), i32(table), i32(lens),
                         700, 2, q_offsets=offs, max_q_len=max(q_lens), return_lse=True)
    ref = window_ref(qf, c, 16, table, lens, q_lens, 700, 2, (1, 1), dim ** -0.5)
    check(*a, ref)
    check(*b, ref)


def test_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn with eager work between."""
    rng = np.random.default_rng(16)
    q_lens, lens = [1] * 6, [2500, 1, 700, 0, 1900, 64]
    table, c, q, qf, offs = _setup(rng, q_lens, lens)
    t, l = i32(table), i32(lens)
    need = max(bd.attend_window_workspace_bytes(c.k, 8, t, 6, 1, w, 4) for w in (4000, 2100))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]

    def call(i, out):
        return bd.attend_window(q, c.k, c.v, t, l, (4000, 2100)[i], 4, out=out, workspace=ws, **c.kw())

    graphs = []
    for i in range(2):
        call(i, outs[i])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, outs[i])
        graphs.append(g)
    for turn in range(4):
        q.copy_(torch.randn_like(q))
        l.copy_(i32([x + turn for x in [2400, 1, 700, 0, 1800, 60]]))
        for i in (0, 1, 1, 0):
            graphs[i].replay()
            eager = call(i, torch.empty_like(q))
            torch.cuda.synchronize()
            assert torch.equal(outs[i], eager)


def test_graph_of_a_split_chunk():
    """Parts of a chunk's keys and what joins them, captured, replayed with other queries and lengths."""
    rng = np.random.default_rng(31)
    table, c, q, qf, offs = _setup(rng, [70, 30], [2500, 900])
    t, l = i32(table), i32([2500, 900])
    out = torch.empty_like(q)

    def call(to):
        return bd.attend_window(q, c.k, c.v, t, l, 1900, 4, q_offsets=offs, max_q_len=70, out=to, **c.kw())

    call(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for turn in range(4):
        q.copy_(torch.randn_like(q))
        l.copy_(i32([2500 - 300 * turn, 70 + turn]))
        g.replay()
        eager = call(torch.empty_like(q))
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_repeated_calls_agree_and_other_streams():
    rng = np.random.default_rng(17)
    for q_lens, lens in KINDS:
        table, c, q, qf, offs = _setup(rng, q_lens, lens)
        args = (q, c.k, c.v, i32(table), i32(lens), 1500, 4)
        kw = dict(q_offsets=offs, max_q_len=max(q_lens), return_lse=True, **c.kw())
        want = bd.attend_window(*args, **kw)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        for got in (bd.attend_window(*args, **kw), bd.attend_window(*args, **kw, stream=s.cuda_stream)):
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_behind_the_last_sequence_stay():
    rng = np.random.default_rng(18)
    for q_lens, lens in (([2, 3], [40, 300]), ([70, 50], [100, 90])):
        table, c, q, qf, offs = _setup(rng, q_lens, lens)
        n = sum(q_lens)
        more = torch.cat([q, q[:3]])
        out = torch.full_like(more, 9.0)
        lse = torch.full(more.shape[:2], 9.0, device="cuda")
        bd.attend_window(more, c.k, c.v, i32(table), i32(lens), 50, 1, q_offsets=offs, max_q_len=max(q_lens),
                         out=out, lse=lse, **c.kw())
        assert (out[n:] == 9).all() and (lse[n:] == 9).all()
        check(out[:n], lse[:n], window_ref(qf, c, 16, table, lens, q_lens, 50, 1, (1, 1), 128 ** -0.5))


def test_refusals_of_the_binding():
    rng = np.random.default_rng(1)
    table, c, q, qf, offs = _setup(rng, [1, 1], [40, 30])
    args = (q, c.k, c.v, i32(table), i32([40, 30]), 50)
    with pytest.raises(TypeError):
        bd.attend_window(*args)
    with pytest.raises(ValueError):
        bd.attend_window(*args, k_block_scales=c.kb.contiguous(), v_block_scales=c.vb)
    with pytest.raises(ValueError):
        bd.attend_window(q[:, :, :64], *args[1:], **c.kw())
    with pytest.raises(bd.BitDeltaError):
        bd.attend_window(*args, k_scale=-1.0, **c.kw())
    k = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        bd.attend_window(q, k, k, *args[3:], **c.kw())


@pytest.mark.parametrize("dim", [64, 128])
def test_workers_pass_over_empty_sequences(dim):
    """(a table so wide that units are split; a workgroup's run then goes over several short units)"""
    rng = np.random.default_rng(dim)
    lens = [int(x) for x in rng.integers(1, 700, 300)]
    for i in (0, 1, 17, 18, 19, 20, 150, 297, 298, 299, *rng.integers(0, 300, 80)):
        lens[i] = 0
    lens[64] = 4000
    table, c, q, qf, _ = _setup(rng, [1] * 300, lens, 4, 2, dim, extra=60)
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 5000, return_lse=True, **c.kw())
    assert bd.attend_window_workspace_bytes(c.k, 4, i32(table), 300, 1, 5000, 0) > 0
    check(out, lse, window_ref(qf, c, 16, table, lens, [1] * 300, 5000, 0, (1.0, 1.0), dim ** -0.5))


def test_refusals_of_the_workspace_query():
    pages = torch.zeros((4, 16, 2, 64), dtype=torch.uint8, device="cuda")
    table = i32([[0, 1], [2, 3]])
    assert bd.attend_window_workspace_bytes(pages, 8, table, 2, 1, 50, 0) >= 0
    for bad, error in ((pages[0], ValueError), (pages.cpu(), TypeError), (None, TypeError)):
        with pytest.raises(error):
            bd.attend_window_workspace_bytes(bad, 8, table, 2, 1, 50, 0)
        with pytest.raises(error):
            bd.attend_shared_workspace_bytes(bad, 8, table, None, [0, 2])
