"""Log-sums of 4-bit attention over one key, which are scores, against the bound of how a query is held
(attend4_ref.score_bound); three of its four numbers would exceed that a hundred times (test_attend4_cpu)."""
import numpy as np
import pytest

import attend4_ref as Q
import cache_ref as R
import test_gpu_attend4 as F
import test_gpu_attend4_prefix as P

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

_announce = F._announce
i32 = F.i32


def _one_key(rng, tokens, heads, hk, dim, exact):
    """Queries and, for each token, a page of one key: 6 everywhere but at the queries' largest values (exact: the
    bound is then 1e-5 and less), or anything."""
    if exact:
        qf = Q.fine_queries(rng, tokens, heads, dim)
        same = qf.reshape(tokens, hk, heads // hk, dim)
        same[:] = same[:, :, :1]  # one key fits the heads of a kv head
        k = np.where(same[:, :, 0] > 1, 0.0, 6.0)
    else:
        qf = rng.integers(128, 256, (tokens, heads, dim)) * np.exp2(rng.integers(-22, -6, (tokens, heads, dim)))
        qf = np.copysign(qf, rng.normal(size=qf.shape))
        k = rng.choice(R.GRID[1:], (tokens, hk, dim)) * rng.choice([-1, 1], (tokens, hk, dim))
    c = F.Cache4(rng, tokens, 1, hk, dim)
    codes, byte = R.encode4(k[:, None])
    keep = R.decode4(codes, byte) == k[:, None]
    assert keep.all()
    c.codes[0], c.byte[0] = codes, byte
    c.upload()
    q = torch.from_numpy(qf).bfloat16()
    assert np.array_equal(q.double().numpy(), qf)
    return c, q.cuda(), qf


def _check_scores(lse, qf, k, scale):
    """k [tokens, heads, dim]: the key that each row sees"""
    z = lse.double().cpu().numpy()
    for t in range(len(qf)):
        for h in range(qf.shape[1]):
            s = scale * (qf[t, h] @ k[t, h])
            # (beyond the score: its factor in base 2 and the way back, two fp32 roundings each; the exponential
            # and logarithm of a sum of 1, a few 2^-23)
            bound = Q.score_bound(qf[t, h], k[t, h], scale) + 2.0 ** -22 * abs(s) + 2.0 ** -21
            assert abs(z[t, h] - s) <= bound, (t, h, z[t, h], s, bound)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("tokens,heads,hk", [(1, 8, 2), (3, 16, 2), (1, 40, 2), (1, 64, 1), (40, 8, 2), (70, 12, 4)])
def test_log_sums_of_windows(tokens, heads, hk, exact, dim):
    """Each token sees its own key only: one token a sequence, a few, and row tiles."""
    rng = np.random.default_rng(560)
    n = 2 * tokens
    c, q, qf = _one_key(rng, n, heads, hk, dim, exact)
    table = i32(np.arange(n).reshape(2, tokens))
    _, lse = bd.attend_window(q, c.k, c.v, table, i32([tokens] * 2), 1, q_offsets=i32([0, tokens, n]),
                              max_q_len=tokens, return_lse=True, **c.kw())
    _check_scores(lse, qf, np.repeat(c.kf[:, 0], heads // hk, 1), dim ** -0.5)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("heads,hk", [(16, 2), (40, 2), (64, 1)])
def test_log_sums_of_prefixes(heads, hk, tiles, exact, dim):
    """Two segments of prefixes of one key; "tiles": of more and of fewer rows than half a tile."""
    rng = np.random.default_rng(561)
    sizes = [19, 2]
    c, q, qf = _one_key(rng, 21, heads, hk, dim, exact)
    if exact:  # a segment's queries have their large values in the same places
        for a, b in ((0, 19), (19, 21)):
            qf[a:b] = qf[a:a + 1]
        q = torch.from_numpy(qf).bfloat16().cuda()
    ptable, offs = np.array([[0], [19]], np.int32), [0, 19, 21]
    if tiles:
        ptable = P.widen(ptable, sizes, 1, hk, dim)
    p, t = i32(ptable), i32(np.zeros((21, 1)))
    need = bd.attend_shared_workspace_bytes(c.k, heads, t, p, offs)
    assert need > 1 << 20 if tiles else need == 0
    _, lse = bd.attend_shared(q, c.k, c.v, t, i32([0] * 21), p, i32([1, 1]), offs, return_lse=True, **c.kw())
    k = np.repeat(c.kf[[0] * 19 + [19] * 2, 0], heads // hk, 1)
    _check_scores(lse, qf, k, dim ** -0.5)
