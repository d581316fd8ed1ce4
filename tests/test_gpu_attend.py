"""Paged attention on the GPU against the plain 64-bit form.

Tolerances, per output element: the result is rounded to bf16 once (half a step, 2^-8 of it) and
each weight once (2^-8 of the weight, so 2^-8 of sum w |v|); fp32 scores are off by at most about
(dim + 8) 2^-24 sum |q||k| scale, below 2e-4 for these inputs, which moves every weight by that
share.  The log-sum is off by the score error plus fp32 rounding."""
import numpy as np
import pytest

import attend_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

BF16 = 2.0 ** -8
SCORE = 2e-4


@pytest.fixture(autouse=True)
def _announce(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"\n[gpu case] {request.node.nodeid}", flush=True)
    yield
    torch.cuda.synchronize()


def make_cache(rng, pages, page, hk, dim, kv, layout="head"):
    """(k, v device views [pages, page, hk, dim], their stored float64 values, scales)."""
    out, vals = [], []
    for _ in range(2):
        x = torch.from_numpy(rng.normal(size=(pages, page, hk, dim)).astype(np.float32))
        x = (x * 16.0).to(torch.float8_e4m3fn) if kv == "fp8" else x.to(torch.bfloat16)
        vals.append(x.float().double().numpy())
        if layout == "head":
            raw = x.view(torch.uint8) if kv == "fp8" else x
            dev = raw.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
            dev = dev.view(torch.float8_e4m3fn) if kv == "fp8" else dev
        else:
            dev = x.cuda()
        out.append(dev)
    return out[0], out[1], vals[0], vals[1], ((1 / 16, 1 / 8) if kv == "fp8" else (1.0, 1.0))


def make_q(rng, tokens, heads, dim):
    q = torch.from_numpy(rng.normal(scale=1.5, size=(tokens, heads, dim)).astype(np.float32))
    q = q.to(torch.bfloat16)
    return q.cuda(), q.double().numpy()


def tables(rng, lengths, page, width, free):
    t = np.full((len(lengths), width), -1, dtype=np.int32)
    for i, n in enumerate(lengths):
        for j in range(-(-n // page)):
            t[i, j] = free.pop()
    return t


def i32(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def check(out, lse, ref):
    """ref: list of (out, mix, lse) per token."""
    got, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t, (o, mix, l) in enumerate(ref):
        tol = BF16 * np.abs(o) + (BF16 + SCORE) * mix
        assert np.all(np.isfinite(got[t])), f"token {t}"
        worst = np.abs(got[t] - o) - tol
        assert worst.max() <= 1e-30, (t, np.unravel_index(worst.argmax(), worst.shape), worst.max())
        dead = np.isneginf(l)
        assert np.array_equal(np.isneginf(z[t]), dead), (t, z[t], l)
        assert np.all(np.abs(z[t][~dead] - l[~dead]) <= SCORE + 1e-6 * np.abs(l[~dead])), (t, z[t], l)


def shared_ref(q, kv, vv, page, table, lens, ptable, plens, offs, scales, scale):
    ref = []
    for g in range(len(offs) - 1):
        pk, pp = R.cache_rows(kv, ptable[g], plens[g], page, scales[0])
        pv, _ = R.cache_rows(vv, ptable[g], plens[g], page, scales[1])
        for b in range(offs[g], offs[g + 1]):
            k, p = R.cache_rows(kv, table[b], lens[b], page, scales[0])
            v, _ = R.cache_rows(vv, table[b], lens[b], page, scales[1])
            ref.append(R.attend(q[b], np.concatenate([pk, k]), np.concatenate([pv, v]),
                                np.concatenate([pp, p]), scale))
    return ref


# sizes per segment, prefix lengths, own lengths (cycled), heads, kv heads, dim, page, type, table
# widths beyond need (wide tables take the split kernels), cache layout
SHARED = [
    ([3], [40], [5, 1, 0], 8, 2, 64, 16, "bf16", 0, "head"),
    ([1, 2, 4], [100, 0, 33], [17, 64, 0, 3], 16, 2, 128, 16, "bf16", 0, "token"),
    ([2, 0, 5], [65, 9, 300], [130, 1, 0, 77], 12, 4, 128, 24, "bf16", 80, "head"),
    ([7], [1], [1], 8, 8, 64, 7, "fp8", 300, "token"),
    ([40, 3], [513, 70], [0, 129, 31], 32, 4, 128, 64, "bf16", 30, "head"),
    ([9, 9], [200, 64], [63, 65, 128], 64, 8, 64, 16, "fp8", 90, "head"),
    ([5, 1], [1030, 300], [300, 0], 12, 4, 128, 24, "fp8", 60, "token"),
    ([1, 1, 1], [700, 0, 5], [900, 0, 40], 6, 2, 128, 16, "bf16", 40, "head"),
    ([3, 2], [150, 90], [20], 20, 1, 64, 16, "bf16", 90, "head"),
    ([6], [333], [50, 0], 128, 2, 128, 32, "bf16", 60, "head"),
    ([4], [0], [0], 8, 2, 128, 16, "bf16", 100, "head"),
    ([300], [97], [3, 40], 8, 1, 64, 16, "bf16", 70, "head"),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared(case):
    sizes, plens, olens, heads, hk, dim, page, kv, extra, layout = SHARED[case]
    rng = np.random.default_rng(case)
    n = sum(sizes)
    lens = [olens[i % len(olens)] for i in range(n)]
    offs = np.concatenate([[0], np.cumsum(sizes)])
    need = sum(-(-x // page) for x in lens + plens)
    free = list(rng.permutation(need + 3))
    table = tables(rng, lens, page, max(-(-max(lens) // page), 0) + extra, free)
    ptable = tables(rng, plens, page, max(-(-max(plens) // page), 0) + extra, free)
    k, v, kf, vf, sc = make_cache(rng, need + 3, page, hk, dim, kv, layout)
    q, qf = make_q(rng, n, heads, dim)
    out, lse = bd.attend_shared(q, k, v, i32(table), i32(lens), i32(ptable), i32(plens), offs,
                                k_scale=sc[0], v_scale=sc[1], return_lse=True)
    check(out, lse, shared_ref(qf, kf, vf, page, table, lens, ptable, plens, offs, sc, dim ** -0.5))


def widen(ptable, sizes, page, hk, dim, kv):
    """The prefix table with unused columns until sharing the prefixes is worth the tile kernel."""
    saved = (sum(sizes) - sum(n > 0 for n in sizes)) * page * hk * 2 * dim * (1 if kv == "fp8" else 2)
    more = np.full((len(ptable), -(-(130 << 20) // saved)), -1, dtype=np.int32)
    return np.concatenate([ptable, more], axis=1)


@pytest.mark.parametrize("case", [i for i, c in enumerate(SHARED) if max(c[0]) > 1])
def test_shared_prefix_in_tiles(case):
    sizes, plens, olens, heads, hk, dim, page, kv, extra, layout = SHARED[case]
    rng = np.random.default_rng(50 + case)
    n = sum(sizes)
    lens = [olens[(i + 1) % len(olens)] for i in range(n)]
    offs = np.concatenate([[0], np.cumsum(sizes)])
    need = sum(-(-x // page) for x in lens + plens)
    free = list(rng.permutation(need + 3))
    table = tables(rng, lens, page, max(-(-max(lens) // page), 0) + extra, free)
    ptable = tables(rng, plens, page, max(-(-max(plens) // page), 0), free)
    if plens[0] > page:  # a page that is none
        ptable[0, 1] = need + 3
    ptable = widen(ptable, sizes, page, hk, dim, kv)
    k, v, kf, vf, sc = make_cache(rng, need + 3, page, hk, dim, kv, layout)
    q, qf = make_q(rng, n, heads, dim)
    assert bd.attend_shared_workspace_bytes(k, heads, i32(table), i32(ptable), offs) > \
        bd.attend_shared_workspace_bytes(k, heads, i32(table), i32(ptable[:, :1]), offs)
    out, lse = bd.attend_shared(q, k, v, i32(table), i32(lens), i32(ptable), i32(plens), offs,
                                k_scale=sc[0], v_scale=sc[1], return_lse=True)
    check(out, lse, shared_ref(qf, kf, vf, page, table, lens, ptable, plens, offs, sc, dim ** -0.5))


# new tokens per sequence, cached lengths, heads, kv heads, dim, page, type, window, sinks, extra
# table width, cache layout
WINDOW = [
    ([1, 1, 1], [1, 0, 50], 8, 2, 64, 16, "bf16", 20, 4, 0, "head"),
    ([1, 1], [300, 129], 64, 8, 128, 16, "bf16", 64, 3, 0, "token"),
    ([1, 1, 1, 1], [2000, 7, 1300, 0], 12, 4, 128, 24, "fp8", 1500, 16, 0, "head"),
    ([1], [4000], 8, 8, 64, 64, "bf16", 4096, 0, 0, "head"),
    ([1, 1], [1500, 800], 40, 2, 64, 16, "fp8", 2000, 1, 0, "token"),
    ([1, 1], [1500, 800], 64, 1, 128, 16, "bf16", 2000, 1, 0, "head"),
    ([2, 4, 1, 0], [30, 4, 90, 10], 8, 2, 64, 16, "bf16", 8, 2, 0, "head"),
    ([3, 1], [1400, 1300], 12, 2, 128, 16, "bf16", 1200, 5, 20, "head"),
    ([4, 2], [1300, 2], 16, 1, 128, 16, "fp8", 3000, 0, 0, "head"),
    ([70, 1, 33], [70, 1, 90], 8, 2, 64, 16, "bf16", 16, 4, 0, "head"),
    ([200], [200], 12, 4, 128, 24, "bf16", 4096, 0, 0, "token"),
    ([65, 130, 0, 3], [400, 130, 20, 3], 64, 8, 128, 64, "bf16", 100, 4, 0, "head"),
    ([129], [700], 32, 8, 128, 16, "fp8", 64, 16, 0, "head"),
    ([90], [300], 16, 16, 64, 16, "fp8", 1, 0, 0, "token"),
    ([300], [300], 8, 1, 128, 7, "bf16", 50, 70, 0, "head"),
    ([40, 20], [25, 0], 64, 1, 64, 16, "bf16", 30, 2, 2, "head"),
    ([33], [33], 10, 2, 128, 16, "bf16", 10, 0, 0, "head"),
]


def window_ref(q, kf, vf, page, table, lens, q_lens, window, sinks, scales, scale):
    ref, at = [], 0
    for b, n in enumerate(q_lens):
        length = min(lens[b], table.shape[1] * page)
        k, p = R.cache_rows(kf, table[b], length, page, scales[0])
        v, _ = R.cache_rows(vf, table[b], length, page, scales[1])
        j = np.arange(length)
        for i in range(n):
            pos = length - n + i
            seen = p & (j <= pos) & ((pos - j < window) | (j < sinks))
            ref.append(R.attend(q[at + i], k, v, seen, scale))
        at += n
    return ref


@pytest.mark.parametrize("case", range(len(WINDOW)))
def test_window(case):
    q_lens, lens, heads, hk, dim, page, kv, window, sinks, extra, layout = WINDOW[case]
    rng = np.random.default_rng(100 + case)
    need = sum(-(-x // page) for x in lens)
    free = list(rng.permutation(need + 2))
    table = tables(rng, lens, page, -(-max(lens) // page) + extra, free)
    k, v, kf, vf, sc = make_cache(rng, need + 2, page, hk, dim, kv, layout)
    q, qf = make_q(rng, sum(q_lens), heads, dim)
    single = all(n == 1 for n in q_lens)
    offs = None if single else i32(np.concatenate([[0], np.cumsum(q_lens)]))
    out, lse = bd.attend_window(q, k, v, i32(table), i32(lens), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), k_scale=sc[0], v_scale=sc[1],
                                return_lse=True)
    check(out, lse, window_ref(qf, kf, vf, page, table, lens, q_lens, window, sinks, sc,
                               dim ** -0.5))


def _window_setup(rng, q_lens, lens, heads=8, hk=2, dim=128, page=16, extra=0):
    need = sum(-(-x // page) for x in lens) + 1
    free = list(rng.permutation(need))
    table = tables(rng, lens, page, -(-max(lens) // page) + extra, free)
    k, v, kf, vf, sc = make_cache(rng, need, page, hk, dim, "bf16")
    q, qf = make_q(rng, sum(q_lens), heads, dim)
    return table, k, v, kf, vf, q, qf, i32(np.concatenate([[0], np.cumsum(q_lens)]))


@pytest.mark.parametrize("q_lens,lens,window", [([1, 1], [900, 40], 4000), ([1, 1], [1900, 40], 4000),
                                                ([2, 3], [1900, 40], 50), ([80, 20], [300, 40], 70)])
def test_window_pages_that_are_no_pages(q_lens, lens, window):
    """Keys whose table entry is no page are absent, wherever they are."""
    rng = np.random.default_rng(5)
    table, k, v, kf, vf, q, qf, offs = _window_setup(rng, q_lens, lens, extra=60)
    table[0, 3], table[1, 0], table[0, -60 - 2] = -1, k.shape[0], 2 ** 31 - 1
    table[0, 11] = -2 ** 31
    out, lse = bd.attend_window(q, k, v, i32(table), i32(lens), window, 2, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True)
    check(out, lse, window_ref(qf, kf, vf, 16, table, lens, q_lens, window, 2, (1, 1), 128 ** -0.5))


@pytest.mark.parametrize("wide", [0, 80])
def test_shared_pages_that_are_no_pages(wide):
    rng = np.random.default_rng(6)
    lens, plens, offs = [50, 0, 90, 20], [200, 40], [0, 3, 4]
    free = list(rng.permutation(40))
    table, ptable = tables(rng, lens, 16, 6 + wide, free), tables(rng, plens, 16, 13 + wide, free)
    k, v, kf, vf, sc = make_cache(rng, 40, 16, 2, 64, "bf16")
    q, qf = make_q(rng, 4, 8, 64)
    ptable[0, 5], ptable[1, :3], table[0, 0], table[3, :2] = -7, 40, 4000, -1
    out, lse = bd.attend_shared(q, k, v, i32(table), i32(lens), i32(ptable), i32(plens), offs,
                                return_lse=True)
    check(out, lse, shared_ref(qf, kf, vf, 16, table, lens, ptable, plens, offs, sc, 64 ** -0.5))


@pytest.mark.parametrize("q_lens,lens", [([1, 1], [40, 90]), ([1, 1], [40, 2000]),
                                         ([3, 2], [40, 2000]), ([70, 40], [70, 300])])
def test_window_unseen_cache_is_never_used(q_lens, lens):
    """NaN in every slot that no query of the call sees changes nothing, and lengths beyond the
    table or below zero count as its capacity and as none."""
    rng = np.random.default_rng(7)
    window, sinks = 30, 3
    table, k, v, kf, vf, q, qf, offs = _window_setup(rng, q_lens, lens, extra=2)
    used = np.zeros(k.shape[:2], dtype=bool)
    for b, n in enumerate(q_lens):
        for j in range(lens[b]):
            if j >= lens[b] - n - window + 1 or j < sinks:
                used[table[b, j // 16], j % 16] = True
    bad = torch.from_numpy(~used).cuda()
    k[bad], v[bad] = float("nan"), float("nan")
    out, lse = bd.attend_window(q, k, v, i32(table), i32(lens), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True)
    check(out, lse, window_ref(qf, kf, vf, 16, table, lens, q_lens, window, sinks, (1, 1),
                               128 ** -0.5))
    lens2 = [-5, table.shape[1] * 16 + 100]
    table2 = np.where(table < 0, 0, table)
    k.nan_to_num_(), v.nan_to_num_()
    kf2, vf2 = k.double().cpu().numpy(), v.double().cpu().numpy()
    out, lse = bd.attend_window(q, k, v, i32(table2), i32(lens2), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True)
    check(out, lse, window_ref(qf, kf2, vf2, 16, table2, [0, table.shape[1] * 16], q_lens, window,
                               sinks, (1, 1), 128 ** -0.5))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_window_value_seen_by_some_tokens_only(value):
    """A value or key that is not finite reaches the tokens that see it and no other."""
    rng = np.random.default_rng(8)
    n, window = 150, 20
    table, k, v, kf, vf, q, qf, offs = _window_setup(rng, [n], [n])
    at = [37, 100]
    v[int(table[0, at[0] // 16]), at[0] % 16, 0, 5] = value
    k[int(table[0, at[1] // 16]), at[1] % 16, 1, 7] = float("nan")
    out, lse = bd.attend_window(q, k, v, i32(table), i32([n]), window, 0, q_offsets=offs,
                                max_q_len=n, return_lse=True)
    o = out.double().cpu().numpy()
    sees = lambda t, j: j <= t < j + window
    ref = window_ref(qf, kf, vf, 16, table, [n], [n], window, 0, (1, 1), 128 ** -0.5)
    for t in range(n):
        hit = np.zeros((8, 128), dtype=bool)
        if sees(t, at[0]):
            hit[:4, 5] = True
            assert not np.isfinite(o[t, :4, 5]).any(), t
        if sees(t, at[1]):
            hit[4:] = True
            assert np.isnan(o[t, 4:]).all(), t
        ro, mix, _ = ref[t]
        ok = np.abs(o[t] - ro) <= BF16 * np.abs(ro) + (BF16 + SCORE) * mix
        assert (ok | hit).all(), (t, np.argwhere(~(ok | hit))[:4])


def test_strided_rows_and_own_outputs():
    """q as a slice of a wider projection, out and lse given, a cache with separate strides."""
    rng = np.random.default_rng(9)
    lens = [70, 33]
    table, k, v, kf, vf, _, _, _ = _window_setup(rng, [1, 1], lens)
    wide, widef = make_q(rng, 2, 12, 128)
    q = wide[:, 2:10]
    hold = torch.full((2, 20, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    out = hold[:, 5:13, :128]
    lse = torch.empty((2, 8), dtype=torch.float32, device="cuda")
    v2 = torch.empty((v.shape[0], 16, 3, 2, 128), dtype=torch.bfloat16, device="cuda")[:, :, 1]
    v2.copy_(v)
    got = bd.attend_window(q, k, v2, i32(table), i32(lens), 50, 2, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(out, lse, window_ref(widef[:, 2:10], kf, vf, 16, table, lens, [1, 1], 50, 2, (1, 1),
                               128 ** -0.5))
    hold[:, 5:13, :128] = 7.0
    assert bool((hold == 7.0).all())


def test_cache_beyond_32_bit_offsets():
    """Pages past 4 GiB of a cache are reached by both kernels and both operators."""
    page, hk, dim = 16, 2, 64
    pages = (5 << 30) // (page * hk * dim * 2)
    k = torch.zeros((pages, page, hk, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    rng = np.random.default_rng(10)
    ids = [pages - 1, pages - 2, pages // 2, 3, 1, pages - 9]
    sk, sv, kf, vf, sc = make_cache(rng, len(ids), page, hk, dim, "bf16", "token")
    idx = torch.tensor(ids, device="cuda")
    k[idx], v[idx] = sk, sv
    table = np.array([[0, 1, 2, 3, 4, 5]], dtype=np.int32)
    far = i32(np.array([ids], dtype=np.int32))
    for n in (1, 90):
        q, qf = make_q(rng, n, 8, dim)
        out, lse = bd.attend_window(q, k, v, far, i32([95]), 4000, 0, q_offsets=i32([0, n]),
                                    max_q_len=n, return_lse=True)
        check(out, lse, window_ref(qf, kf, vf, page, table, [95], [n], 4000, 0, sc, dim ** -0.5))
    q, qf = make_q(rng, 3, 8, dim)
    wide = torch.full((1, 80), -1, dtype=torch.int32, device="cuda")
    wide[:, :6] = far
    out, lse = bd.attend_shared(q, k, v, wide.repeat(3, 1)[:, 3:].contiguous(), i32([20, 0, 40]),
                                wide, i32([48]), [0, 3], return_lse=True)
    check(out, lse, shared_ref(qf, kf, vf, page, table[:, 3:].repeat(3, 0), [20, 0, 40], table, [48],
                               [0, 3], sc, dim ** -0.5))


@pytest.mark.parametrize("batch,hk,group,most", [(16, 4, 16, 3), (48, 4, 12, 2), (64, 8, 1, 1)])
def test_window_kernel_choice(batch, hk, group, most):
    """Many units of 33..64 rows, of 17..32 rows (tile kernel), and single tokens over lists of up
    to 12 steps that no workgroup shares."""
    rng = np.random.default_rng(batch)
    page, width = 16, 12 if most > 1 else 90
    q_lens = rng.integers(0 if most > 1 else 1, most + 1, batch).tolist()
    q_lens[3] = most
    lens = [int(rng.integers(n, 60)) for n in q_lens]
    lens[3], lens[5] = (180 if most > 1 else 1400), q_lens[5]
    need = sum(-(-x // page) for x in lens)
    table = tables(rng, lens, page, width, list(rng.permutation(need)))
    k, v, kf, vf, sc = make_cache(rng, need, page, hk, 64, "bf16")
    q, qf = make_q(rng, sum(q_lens), hk * group, 64)
    offs = i32(np.concatenate([[0], np.cumsum(q_lens)])) if most > 1 else None
    window = 40 if most > 1 else 2000
    out, lse = bd.attend_window(q, k, v, i32(table), i32(lens), window, 2, q_offsets=offs,
                                max_q_len=most, return_lse=True)
    check(out, lse, window_ref(qf, kf, vf, page, table, lens, q_lens, window, 2, sc, 0.125))


def _graph_call(kind):
    rng = np.random.default_rng(11)
    if kind == "shared":
        lens, plens, offs = [50, 700, 90, 20], [2000, 400], [0, 3, 4]
        free = list(rng.permutation(300))
        table, ptable = tables(rng, lens, 16, 50, free), tables(rng, plens, 16, 130, free)
        k, v, *_ = make_cache(rng, 300, 16, 2, 128, "bf16")
        q, _ = make_q(rng, 4, 16, 128)
        t, l, pt, pl = i32(table), i32(lens), i32(ptable), i32(plens)
        ws = torch.empty(max(1, bd.attend_shared_workspace_bytes(k, 16, t, pt, offs)),
                         dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        return q, l, lambda: bd.attend_shared(q, k, v, t, l, pt, pl, offs, out=out, workspace=ws,
                                              return_lse=True)
    q_lens, lens = ([1, 1], [1900, 500]) if kind == "decode" else ([100, 30], [300, 80])
    table, k, v, _, _, q, _, offs = _window_setup(rng, q_lens, lens)
    t, l = i32(table), i32(lens)
    ws = torch.empty(max(1, bd.attend_window_workspace_bytes(k, 8, t, q.shape[0], max(q_lens), 4000, 4)),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    return q, l, lambda: bd.attend_window(q, k, v, t, l, 4000, 4, q_offsets=offs,
                                          max_q_len=max(q_lens), out=out, workspace=ws,
                                          return_lse=True)


@pytest.mark.parametrize("kind", ["shared", "decode", "prefill"])
def test_graph_replays_and_other_streams(kind):
    """Captured calls replay like eager ones, bit for bit, also with lengths and queries that
    changed since; and a call on another stream equals one on the current stream."""
    q, lens, call = _graph_call(kind)
    eager = [x.clone() for x in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = [x.clone() for x in call()]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(eager, side))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = call()
    for i in range(4):
        q.copy_(torch.randn(q.shape, device="cuda").to(torch.bfloat16))
        lens.sub_(3)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in res]
        torch.randn(1 << 20, device="cuda").sum().item()
        want = [x.clone() for x in call()]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_graph_replays_prefix_tiles():
    rng = np.random.default_rng(12)
    sizes, plens, page, hk, dim = [3, 20], [900, 400], 16, 2, 128
    lens, offs = rng.integers(20, 300, 23).tolist(), [0, 3, 23]
    free = list(rng.permutation(600))
    table, ptable = tables(rng, lens, page, 50, free), tables(rng, plens, page, 60, free)
    ptable = widen(ptable, sizes, page, hk, dim, "bf16")
    k, v, kf, vf, sc = make_cache(rng, 600, page, hk, dim, "bf16")
    q, _ = make_q(rng, 23, 16, dim)
    t, l, pt, pl = i32(table), i32(lens), i32(ptable), i32(plens)
    call = lambda: bd.attend_shared(q, k, v, t, l, pt, pl, offs, return_lse=True)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = call()
    for i in range(4):
        new, qf = make_q(rng, 23, 16, dim)
        q.copy_(new)
        l.sub_(3)
        pl.sub_(70)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in res]
        torch.randn(1 << 20, device="cuda").sum().item()
        assert all(torch.equal(a, b) for a, b in zip(got, call())), i
    check(*got, shared_ref(qf, kf, vf, page, table, l.tolist(), ptable, pl.tolist(), offs, sc, dim ** -0.5))


def test_binding_refusals():
    rng = np.random.default_rng(12)
    table, k, v, _, _, q, _, offs = _window_setup(rng, [1, 1], [40, 33])
    t, l = i32(table), i32([40, 33])
    with pytest.raises(TypeError):
        bd.attend_window(q.float(), k, v, t, l, 8)
    with pytest.raises(TypeError):
        bd.attend_window(q, k.float(), v.float(), t, l, 8)
    with pytest.raises(TypeError):
        bd.attend_window(q, k, v, t.long(), l, 8)
    with pytest.raises(ValueError):
        bd.attend_window(q, k, v, t[:1], l, 8)
    with pytest.raises(ValueError):
        bd.attend_window(q, k, v[..., ::2], t, l, 8)
    with pytest.raises(ValueError):
        bd.attend_shared(q, k, v, t, l, t, None, [0, 2])
    with pytest.raises(bd.BitDeltaError):
        bd.attend_window(q, k, v, t, l, 0)
    with pytest.raises(bd.BitDeltaError):
        bd.attend_shared(q, k, v, t, l, t[:1], l[:1], [0, 1])
