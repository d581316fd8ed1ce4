"""4-bit pages whose scale bytes cache_write never makes (0, 1, 253, 254), as another writer may: what they
stand for, 2^128 and more as an infinity, and that a row sees nothing of keys that are hidden from it.

Tolerances are those of test_gpu_attend4."""
import numpy as np
import pytest

import cache_ref as R
import test_gpu_attend as A
import test_gpu_attend4 as F

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

_announce = F._announce
i32 = A.i32
FAR = [0, 1, 253, 254]
KINDS = F.KINDS


def infinite(x):
    """float64 values as bf16 and fp32 hold them: 2^128 and more is an infinity."""
    return np.where(np.abs(x) >= 2.0 ** 128, np.copysign(np.inf, x), x)


@pytest.mark.parametrize("scale", [1.0, 0.125, 2.0 ** 90, 0.7])
def test_read_of_every_code_and_scale_byte(scale):
    codes = np.tile(np.arange(16), 256 * 2).reshape(256, 1, 1, 32)  # token b: byte b
    codes = np.concatenate([codes, np.roll(codes, 5, -1)], -1).astype(np.uint8).reshape(16, 16, 1, 64)
    byte = np.repeat(np.arange(256), 2).astype(np.uint8).reshape(16, 16, 1, 2)
    pages, blocks = torch.from_numpy(R.pack4(codes)).cuda(), torch.from_numpy(byte).cuda()
    k, v = bd.cache_read(pages, pages, i32(np.arange(16)[None]), i32([256]), q_offsets=i32([0, 256]), tokens=256,
                         k_scale=scale, v_scale=1.0, k_block_scales=blocks, v_block_scales=blocks)
    x = R.decode4(codes, byte).reshape(256, 1, 64)
    with np.errstate(over="ignore"):
        want = [torch.from_numpy((infinite(x).astype(np.float32) * np.float32(s))).bfloat16() for s in (scale, 1.0)]
    for got, w in zip((k, v), want):
        assert np.array_equal(got.double().cpu().numpy(), w.double().numpy(), equal_nan=True)


def _unseen(c, table, q_lens, lens, window, sinks):
    seen = np.zeros(c.kf.shape[:2], bool)
    for b, n in enumerate(q_lens):
        for i in range(n):
            pos = lens[b] - n + i
            for j in range(pos + 1):
                if pos - j < window or j < sinks:
                    seen[table[b, j // 16], j % 16] = True
    return ~seen


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
@pytest.mark.parametrize("window", [37, 4000])
def test_what_no_query_sees_is_not_used(q_lens, lens, window, dim):
    rng = np.random.default_rng(41)
    table, c, q, qf, offs = F._setup(rng, q_lens, lens, dim=dim)
    ref = F.window_ref(qf, c, 16, table, lens, q_lens, window, 3, (1, 1), dim ** -0.5)
    hidden = _unseen(c, table, q_lens, lens, window, 3)
    for codes, byte in zip(c.codes, c.byte):
        byte[hidden] = rng.choice(FAR, byte[hidden].shape)
        codes[hidden] = rng.integers(0, 16, codes[hidden].shape)
    c.upload()
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), window, 3, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    F.check(out, lse, ref)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("byte", [253, 254])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_infinite_values_reach_the_rows_that_see_them(q_lens, lens, byte, dim):
    """A value of 2^128 and more makes its dim of the rows that see it infinite; other dims, of its block too,
    and other rows stay as they are."""
    rng = np.random.default_rng(43)
    table, c, q, qf, offs = F._setup(rng, q_lens, lens, dim=dim)
    for b, n in enumerate(q_lens):
        for at, head in ((lens[b] - max(1, n // 2), b % 2), (lens[b] - n - 9, 1 - b % 2)):
            if at < 0:
                continue
            # seen by some rows of the chunk only; leaves the window in the chunk
            page, slot, block = table[b, at // 16], at % 16, (b + head) % (dim // 32)
            c.byte[1][page, slot, head, block] = byte
            code = np.zeros(32, np.uint8)
            code[[1, 6, 17, 31]] = 7, 15, 8 + 6, 6
            if byte == 254:
                code[[3, 20]] = 4, 13
            c.codes[1][page, slot, head, 32 * block:32 * block + 32] = code
    c.upload()
    window = 9 + max(q_lens) // 2
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), window, 0, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    c.vf = infinite(c.vf)
    far = np.isinf(c.vf)
    # the finite ones' sums, the infinite ones' signs
    vf, c.vf = c.vf, np.where(far, 0.0, c.vf)
    ref = F.window_ref(qf, c, 16, table, lens, q_lens, window, 0, (1, 1), dim ** -0.5)
    signs = []
    for sign in (1, -1):
        c.vf = np.where(far & (np.sign(vf) == sign), 1.0, 0.0)
        signs.append([o > 0 for o, *_ in F.window_ref(qf, c, 16, table, lens, q_lens, window, 0, (1, 1), dim ** -0.5)])
    got = out.double().cpu().numpy()
    assert sum(s.sum() for s in signs[0]) > 0
    for t, (o, mix, l, err) in enumerate(ref):
        plus, minus = signs[0][t], signs[1][t]
        want = np.where(plus, np.inf, np.where(minus, -np.inf, 0.0))
        want[plus & minus] = np.nan
        one = plus | minus
        assert np.array_equal(got[t][one], want[one], equal_nan=True), t
        got[t][one] = o[one]
    F.check(torch.from_numpy(got), lse, ref)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_largest_finite_values(q_lens, lens, dim):
    """Codes of the largest scales that stay below 2^128 count as they are, beside others of their block.
    (Queries of zeros: every weight is the same, so the sums stay in range as well.)"""
    rng = np.random.default_rng(44)
    table, c, q, qf, offs = F._setup(rng, q_lens, lens, dim=dim)
    c.codes[1][:], c.byte[1][:] = 0, 127
    for b, n in enumerate(q_lens):
        at = lens[b] - max(1, n // 2)
        page, slot = table[b, at // 16], at % 16
        c.byte[1][page, slot, :, 0], c.byte[1][page, slot, :, 1] = 253, 254
        c.codes[1][page, slot, :, 3], c.codes[1][page, slot, :, 9] = 1, 13     # 2^125, -3 * 2^126
        c.codes[1][page, slot, :, 35], c.codes[1][page, slot, :, 50] = 9, 2    # -2^126, 2^127
    c.upload()
    q.zero_()
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 5000, 0, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, v_scale=2.0 ** -100, **c.kw())
    F.check(out, lse, F.window_ref(0 * qf, c, 16, table, lens, q_lens, 5000, 0, (1, 2.0 ** -100), dim ** -0.5))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_smallest_values(q_lens, lens, dim):
    """Values of the smallest scales, under a scale that brings them back."""
    rng = np.random.default_rng(45)
    table, c, q, qf, offs = F._setup(rng, q_lens, lens, dim=dim)
    c.byte[1] = rng.integers(0, 5, c.byte[1].shape).astype(np.uint8)
    c.upload()
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 5000, 0, q_offsets=offs,
                                max_q_len=max(q_lens), return_lse=True, v_scale=2.0 ** 120, **c.kw())
    F.check(out, lse, F.window_ref(qf, c, 16, table, lens, q_lens, 5000, 0, (1, 2.0 ** 120), dim ** -0.5))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("low", [True, False])
@pytest.mark.parametrize("q_lens,lens", KINDS)
def test_keys_of_the_smallest_and_largest_scales(q_lens, lens, low, dim):
    rng = np.random.default_rng(46)
    table, c, q, qf, offs = F._setup(rng, q_lens, lens, dim=dim)
    c.byte[0] = rng.choice([0, 1, 2] if low else [252, 253, 254], c.byte[0].shape).astype(np.uint8)
    c.upload()
    # scores of a few units: q of 2^60 against 2^-127, 2^-100 against 2^127, under a scale of keys
    q = (q.float() * 2.0 ** (60 if low else -100)).bfloat16()
    k_scale = 2.0 ** (66 if low else -28)
    out, lse = bd.attend_window(q, c.k, c.v, i32(table), i32(lens), 5000, 0, q_offsets=offs, k_scale=k_scale,
                                max_q_len=max(q_lens), return_lse=True, **c.kw())
    F.check(out, lse, F.window_ref(q.double().cpu().numpy(), c, 16, table, lens, q_lens, 5000, 0, (k_scale, 1),
                                   dim ** -0.5))
