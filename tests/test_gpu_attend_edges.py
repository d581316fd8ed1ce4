"""Paged attention on the GPU at the ends of its arguments and with values that are not finite, against
the plain 64-bit form, with the tolerances of test_gpu_attend.py."""
import numpy as np
import pytest

import test_gpu_attend as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _announce(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"\n[gpu case] {request.node.nodeid}", flush=True)
    yield
    torch.cuda.synchronize()


def setup(rng, q_lens, lens, heads, hk, dim=128, page=16, kv="bf16", extra=0):
    need = sum(-(-x // page) for x in lens) + 1
    table = A.tables(rng, lens, page, -(-max(lens) // page) + extra, list(rng.permutation(need)))
    k, v, kf, vf, sc = A.make_cache(rng, need, page, hk, dim, kv)
    q, qf = A.make_q(rng, sum(q_lens), heads, dim)
    return table, k, v, kf, vf, sc, q, qf, A.i32(np.concatenate([[0], np.cumsum(q_lens)]))


def poke(pages, page, slot, head, d, value):
    """One stored value; e4m3 by its byte (all ones below the sign: NaN)."""
    if pages.dtype == torch.float8_e4m3fn:
        assert np.isnan(value)
        pages.view(torch.uint8)[page, slot, head, d] = 0x7F
    else:
        pages[page, slot, head, d] = value


# new tokens, cached lengths, heads, kv heads, dim, window: tiles of 256 and of 32 tokens where some
# waves see all of an edge step's keys and others do not; a window whose left edge crosses tiles; the row
# kernel with several tokens, in one piece and split
SEEN = [
    ([300], [300], 4, 4, 128, 4096),
    ([200], [210], 16, 2, 128, 4096),
    ([200], [210], 16, 2, 64, 4096),
    ([280], [400], 3, 3, 64, 90),
    ([130, 90], [130, 100], 8, 2, 128, 70),
    ([4], [30], 8, 2, 128, 4096),
    ([3, 2], [1900, 40], 8, 2, 64, 4096),
    ([8, 5], [1900, 300], 8, 2, 128, 100),
]


@pytest.mark.parametrize("kv,value", [("bf16", NAN), ("bf16", INF), ("bf16", -INF), ("fp8", NAN)])
@pytest.mark.parametrize("case", range(len(SEEN)))
def test_window_value_that_is_not_finite_reaches_every_token_that_sees_it(case, kv, value):
    q_lens, lens, heads, hk, dim, window = SEEN[case]
    rng = np.random.default_rng(300 + case)
    table, k, v, kf, vf, sc, q, qf, offs = setup(rng, q_lens, lens, heads, hk, dim, kv=kv)
    at = {}  # sequence, kv head -> (key, dim of the value)
    for b, (n, length) in enumerate(zip(q_lens, lens)):
        for g in range(hk):
            j = [length - n + min(10, n // 2), length - 1, max(length - n - 20, 0), length - n // 2][(b + g) % 4]
            at[b, g] = j, int(rng.integers(dim))
            poke(v, int(table[b, j // 16]), j % 16, g, at[b, g][1], value)
    out, lse = bd.attend_window(q, k, v, A.i32(table), A.i32(lens), window, 0, q_offsets=offs,
                                max_q_len=max(q_lens), k_scale=sc[0], v_scale=sc[1], return_lse=True)
    o = out.double().cpu().numpy()
    ref = A.window_ref(qf, kf, vf, 16, table, lens, q_lens, window, 0, sc, dim ** -0.5)
    t = 0
    for b, (n, length) in enumerate(zip(q_lens, lens)):
        for pos in range(length - n, length):
            hit = np.zeros((heads, dim), dtype=bool)
            for g in range(hk):
                j, d = at[b, g]
                if j <= pos < j + window:
                    hit[g * (heads // hk):(g + 1) * (heads // hk), d] = True
            assert not np.isfinite(o[t][hit]).any(), (b, pos)
            ro, mix, _ = ref[t]
            ok = np.abs(o[t] - ro) <= A.BF16 * np.abs(ro) + (A.BF16 + A.SCORE) * mix
            assert (ok | hit).all(), (b, pos, np.argwhere(~(ok | hit))[:4])
            t += 1


@pytest.mark.parametrize("q_lens,lens", [([1, 1], [40, 90]), ([1, 1], [40, 2000]), ([3, 2], [40, 2000]),
                                         ([70, 40], [70, 300])])
def test_window_unseen_e4m3_cache_is_never_used(q_lens, lens):
    """NaN in every slot of an e4m3 cache that no query of the call sees changes nothing."""
    rng = np.random.default_rng(21)
    window, sinks = 30, 3
    table, k, v, kf, vf, sc, q, qf, offs = setup(rng, q_lens, lens, 8, 2, kv="fp8", extra=2)
    used = np.zeros(k.shape[:2], dtype=bool)
    for b, n in enumerate(q_lens):
        for j in range(lens[b]):
            if j >= lens[b] - n - window + 1 or j < sinks:
                used[table[b, j // 16], j % 16] = True
    bad = torch.from_numpy(~used).cuda()
    k.view(torch.uint8)[bad], v.view(torch.uint8)[bad] = 0x7F, 0xFF
    out, lse = bd.attend_window(q, k, v, A.i32(table), A.i32(lens), window, sinks, q_offsets=offs,
                                max_q_len=max(q_lens), k_scale=sc[0], v_scale=sc[1], return_lse=True)
    A.check(out, lse, A.window_ref(qf, kf, vf, 16, table, lens, q_lens, window, sinks, sc, 128 ** -0.5))


# new tokens, cached lengths, heads, kv heads, a chunk limit below the longest: single tokens, the row
# kernel (one piece, split), the tile kernel
CUT = [
    ([5, 1, 3], [40, 30, 90], 8, 2, 1),
    ([5, 1, 3], [1900, 30, 1300], 8, 2, 1),
    ([7, 2, 9], [40, 30, 90], 8, 2, 3),
    ([7, 2, 9], [1900, 2, 1300], 8, 2, 4),
    ([150, 40], [300, 40], 8, 2, 100),
    ([150, 40, 3], [149, 20, 3], 16, 1, 77),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(CUT)))
def test_rows_beyond_max_q_len_are_left_out_and_the_others_keep_their_places(case, kv):
    q_lens, lens, heads, hk, most = CUT[case]
    rng = np.random.default_rng(400 + case)
    table, k, v, kf, vf, sc, q, qf, offs = setup(rng, q_lens, lens, heads, hk, kv=kv)
    window, sinks = 60, 2
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    bd.attend_window(q, k, v, A.i32(table), A.i32(lens), window, sinks, q_offsets=offs, max_q_len=most,
                     k_scale=sc[0], v_scale=sc[1], out=out, lse=lse)
    ref = A.window_ref(qf, kf, vf, 16, table, lens, q_lens, window, sinks, sc, 128 ** -0.5)
    done = np.concatenate([np.arange(n) < most for n in q_lens])
    A.check(out[torch.from_numpy(done).cuda()], lse[torch.from_numpy(done).cuda()],
            [r for r, d in zip(ref, done) if d])
    left = torch.from_numpy(~done).cuda()
    assert bool((out[left] == 7.0).all()) and bool((lse[left] == 7.0).all())


@pytest.mark.parametrize("first,cut", [(0, 4), (-3, 0), (-2, 5)])
@pytest.mark.parametrize("q_lens,lens", [([9, 8], [300, 100]), ([9, 8], [1900, 1300]), ([90, 80], [300, 100])])
def test_rows_outside_the_tokens_are_left_out_and_the_others_keep_their_places(q_lens, lens, first, cut):
    """Offsets that begin before row 0 or end past the last row."""
    rng = np.random.default_rng(41)
    table, k, v, kf, vf, sc, q, qf, _ = setup(rng, q_lens, lens, 8, 2)
    total = sum(q_lens)
    offs = np.concatenate([[0], np.cumsum(q_lens)]) + first
    rows = slice(max(-first, 0), total - cut)  # of the whole list of tokens, those that are given
    out, lse = bd.attend_window(q[rows].contiguous(), k, v, A.i32(table), A.i32(lens), 60, 2,
                                q_offsets=A.i32(offs), max_q_len=max(q_lens), return_lse=True)
    ref = A.window_ref(qf, kf, vf, 16, table, lens, q_lens, 60, 2, sc, 128 ** -0.5)
    A.check(out, lse, ref[rows])


@pytest.mark.parametrize("most", [None, 500])
@pytest.mark.parametrize("q_lens,lens", [([1, 1], [40, 300]), ([3, 1, 0, 2], [40, 300, 5, 900]),
                                         ([90, 33], [300, 40])])
def test_max_q_len_above_the_longest_chunk(q_lens, lens, most):
    """A limit that no chunk reaches; without one it is the number of rows."""
    rng = np.random.default_rng(42)
    table, k, v, kf, vf, sc, q, qf, offs = setup(rng, q_lens, lens, 8, 2)
    kw = {} if most is None else {"max_q_len": most}
    out, lse = bd.attend_window(q, k, v, A.i32(table), A.i32(lens), 60, 2, q_offsets=offs, return_lse=True, **kw)
    A.check(out, lse, A.window_ref(qf, kf, vf, 16, table, lens, q_lens, 60, 2, sc, 128 ** -0.5))


@pytest.mark.parametrize("q_lens,lens", [([1, 1], [40, 300]), ([3, 1, 0, 2], [40, 300, 5, 900]),
                                         ([90, 33], [300, 40])])
def test_max_q_len_of_no_limit(q_lens, lens):
    """The largest limit there is."""
    rng = np.random.default_rng(43)
    table, k, v, kf, vf, sc, q, qf, offs = setup(rng, q_lens, lens, 8, 2)
    out, lse = bd.attend_window(q, k, v, A.i32(table), A.i32(lens), 60, 2, q_offsets=offs,
                                max_q_len=2 ** 31 - 1, return_lse=True)
    A.check(out, lse, A.window_ref(qf, kf, vf, 16, table, lens, q_lens, 60, 2, sc, 128 ** -0.5))


def test_segment_offsets_are_checked_without_prefixes():
    rng = np.random.default_rng(61)
    table, k, v, kf, vf, sc, q, qf, _ = setup(rng, [1, 1], [40, 33], 8, 2)
    t, l = A.i32(table), A.i32([40, 33])
    ref = A.window_ref(qf, kf, vf, 16, table, [40, 33], [1, 1], 4000, 0, sc, 128 ** -0.5)
    for offs in ([0, 2], [0, 1, 2], [0, 0, 2, 2]):
        A.check(*bd.attend_shared(q, k, v, t, l, None, None, offs, return_lse=True), ref)
    for offs in ([0, 1], [1, 2], [0, 3], [0, 2, 1, 2], [0], [0] * 66 + [2]):
        with pytest.raises(bd.BitDeltaError):
            bd.attend_shared(q, k, v, t, l, None, None, offs)


@pytest.mark.parametrize("n,length", [(1, 7), (3, 2000)])
def test_single_heads_with_any_stride(n, length):
    """q, out and the cache of one head, whose head dimension has a stride of 1."""
    rng = np.random.default_rng(71)
    table, k, v, kf, vf, sc, q, qf, offs = setup(rng, [n], [length], 1, 1, 64)
    lay = lambda x: x.squeeze(-2).contiguous().unsqueeze(-1).transpose(-1, -2)  # noqa: E731
    q1, k1, v1 = lay(q), lay(k), lay(v)
    out = lay(torch.empty_like(q))
    assert q1.stride(-2) == k1.stride(-2) == out.stride(-2) == 1
    _, lse = bd.attend_window(q1, k1, v1, A.i32(table), A.i32([length]), 1500, 2, q_offsets=offs, max_q_len=n,
                              out=out, return_lse=True)
    A.check(out, lse, A.window_ref(qf, kf, vf, 16, table, [length], [n], 1500, 2, sc, 64 ** -0.5))
