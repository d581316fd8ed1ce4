"""attend_shared over 4-bit pages by each of its ways: prefixes read with every sequence's own keys by one
workgroup ("direct") or several ("split"), or once per segment by the tile kernel ("tiles"), which tables
wide enough choose.

Tolerances are those of test_gpu_attend4."""
import numpy as np
import pytest

import test_gpu_attend as A
import test_gpu_attend4 as F

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

_announce = F._announce
i32 = A.i32
SHARE_BYTES = 400 << 20  # of 4-bit keys and values that sharing has to save
WAYS = ["direct", "split", "tiles"]


def pad(table, columns):
    return np.concatenate([table, np.full((len(table), columns), -1, np.int32)], 1)


def widen(ptable, sizes, page, hk, dim):
    """The prefix table with unused columns until sharing the prefixes is worth the tile kernel."""
    saved = (sum(sizes) - sum(n > 0 for n in sizes)) * page * hk * (dim + dim // 16)
    return pad(ptable, -(-SHARE_BYTES // saved))


class Call:
    """Sequences of segments `sizes` behind prefixes of `plens` tokens with own keys of `olens` (cycled), page 0
    nobody's, tables for one of the ways."""

    def __init__(self, rng, way, sizes, plens, olens, heads, hk, dim, page=16, layout="head"):
        self.page, self.sizes, self.plens, self.dim = page, sizes, plens, dim
        n = sum(sizes)
        self.lens = [olens[i % len(olens)] for i in range(n)]
        self.offs = np.concatenate([[0], np.cumsum(sizes)])
        need = sum(-(-x // page) for x in self.lens + plens)
        free = [int(x) + 1 for x in rng.permutation(need + 2)]
        self.table = A.tables(rng, self.lens, page, -(-max(self.lens) // page), free)
        self.ptable = A.tables(rng, plens, page, -(-max(plens) // page), free)
        if way != "direct":
            self.table = pad(self.table, -(-4200 // page))
        if way == "tiles":
            self.ptable = widen(self.ptable, sizes, page, hk, dim)
        self.c = F.Cache4(rng, need + 3, page, hk, dim, layout)
        self.q, self.qf = A.make_q(rng, n, heads, dim)
        t, p = i32(self.table), i32(self.ptable)
        if way == "tiles":
            assert bd.attend_shared_workspace_bytes(self.c.k, heads, t, p, self.offs) > \
                bd.attend_shared_workspace_bytes(self.c.k, heads, t, p[:, :1].contiguous(), self.offs) + (1 << 20)
        else:
            assert (bd.attend_shared_workspace_bytes(self.c.k, heads, t, p, self.offs) == 0) == (way == "direct")

    def run(self):
        return bd.attend_shared(self.q, self.c.k, self.c.v, i32(self.table), i32(self.lens), i32(self.ptable),
                                i32(self.plens), self.offs, return_lse=True, **self.c.kw())

    def ref(self):
        return F.shared_ref(self.qf, self.c, self.page, self.table, self.lens, self.ptable, self.plens, self.offs,
                            (1.0, 1.0), self.dim ** -0.5)

    def seen(self):
        """[pages, page]: slots that some sequence sees"""
        seen = np.zeros(self.c.kf.shape[:2], bool)
        for table, lens in ((self.ptable, self.plens), (self.table, self.lens)):
            for row, n in zip(table, lens):
                for j in range(n):
                    if 0 <= row[j // self.page] < len(seen):
                        seen[row[j // self.page], j % self.page] = True
        return seen


@pytest.mark.parametrize("case", [i for i, c in enumerate(A.SHARED) if max(c[0]) > 1])
def test_prefixes_in_tiles(case):
    sizes, plens, olens, heads, hk, dim, page, _, _, layout = A.SHARED[case]
    rng = np.random.default_rng(500 + case)
    x = Call(rng, "tiles", sizes, plens, olens, heads, hk, dim, page, layout)
    if plens[0] > page:  # a page that is none
        x.ptable[0, 1] = len(x.c.kf)
    F.check(*x.run(), x.ref())


# sizes per segment, prefix and own lengths, heads, kv heads, page.  Rows of a segment up to 128: two 64-key
# tiles a step; prefixes of an odd and an even number of tiles, ends within and at the end of one; runs of one
# and of several steps, of one and several units
TILES = [
    ([6, 5], [4200, 4133], [3, 0, 200], 16, 8, 16),       # 66 and 65 tiles
    ([20, 3, 9], [3000, 65, 1], [40, 7], 64, 4, 16),      # 320, 48 and 144 rows: two tiles of rows, half, one
    ([2, 2, 2, 2, 2], [64, 65, 128, 129, 192], [0], 8, 2, 16),
    ([8, 9, 1, 0, 16], [700, 701, 63, 50, 0], [40], 16, 1, 24),  # 128 and 144 rows
    ([50, 86], [500, 333], [10, 0], 12, 4, 7),            # 3 heads a kv head: 86 sequences are two tiles
    ([3, 2], [1000, 90], [30], 64, 1, 16),                # 192 and 128 rows of 64 heads
]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("case", range(len(TILES)))
def test_tiles_of_all_sizes(case, dim):
    """(some pages of the prefixes are none, page 0 holds NaN)"""
    sizes, plens, olens, heads, hk, page = TILES[case]
    rng = np.random.default_rng(520 + case)
    x = Call(rng, "tiles", sizes, plens, olens, heads, hk, dim, page)
    for g, n in enumerate(plens):
        if n > 2 * page:
            x.ptable[g, [1, n // page // 2]] = (-1, len(x.c.kf), 2 ** 31 - 1, -2 ** 31)[g % 4], -5
    for byte in x.c.byte:
        byte[0] = 255
    x.c.upload()
    F.check(*x.run(), x.ref())


SMALL = ([5, 1, 3], [300, 70, 129], [20, 0, 33], 16, 2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("heads", [16, 40, 128])
def test_what_no_sequence_sees_is_not_used(way, heads, dim):
    """NaN and infinities behind the lengths, in absent pages' place (page 0) and in pages of nobody."""
    rng = np.random.default_rng(540)
    x = Call(rng, way, *SMALL[:3], heads, SMALL[4], dim)
    x.ptable[0, 3] = -1
    x.ptable[2, 0] = 10 ** 6
    ref = x.ref()
    hidden = ~x.seen()
    for codes, byte in zip(x.c.codes, x.c.byte):
        byte[hidden] = rng.choice([253, 254, 255, 255], byte[hidden].shape)
        codes[hidden] = rng.integers(0, 16, codes[hidden].shape)
    x.c.upload()
    F.check(*x.run(), ref)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("which", [0, 1])
def test_blocks_of_nan_reach_the_sequences_that_see_them(way, which, dim):
    """One in a prefix its whole segment, one among a sequence's own keys that sequence."""
    rng = np.random.default_rng(541)
    x = Call(rng, way, *SMALL, dim)
    byte = x.c.byte[which]
    byte[x.ptable[0, 299 // 16], 299 % 16, 1, 0] = 255
    byte[x.ptable[2, 4], 0, 0, 1] = 255
    byte[x.table[3, 1], 3, 0, dim // 32 - 1] = 255
    x.c.upload()
    ref = x.ref()
    nan = np.array([np.isnan(o).any() for o, *_ in ref])
    assert list(np.flatnonzero(~nan)) == [5]
    F.check(*x.run(), ref)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("way", WAYS)
def test_infinite_values_of_prefixes(way, dim):
    rng = np.random.default_rng(542)
    x = Call(rng, way, *SMALL, dim)
    ref = x.ref()
    at = x.ptable[0, 2], 5
    for codes, head, block, byte in ((7, 0, 0, 253), (8 + 4, 1, 1, 254)):
        x.c.byte[1][at][head, block] = byte
        x.c.codes[1][at][head, 32 * block:32 * block + 32] = 0
        x.c.codes[1][at][head, 32 * block + 9] = codes
    x.c.upload()
    out, lse = x.run()
    got = out.double().cpu().numpy()
    assert (got[:5, :8, 9] == np.inf).all() and (got[:5, 8:, 41] == -np.inf).all()
    got[:5, :8, 9] = got[:5, 8:, 41] = 0
    assert np.isfinite(got).all()
    F.check(out[5:], lse[5:], ref[5:])


def test_captured_prefixes():
    """The prefixes' launch, the own keys' and what joins them, replayed with other queries and lengths."""
    rng = np.random.default_rng(543)
    x = Call(rng, "tiles", [20, 3, 9], [3000, 65, 1000], [40, 7], 64, 4, 128)
    t, l, p, m = i32(x.table), i32(x.lens), i32(x.ptable), i32(x.plens)
    out = torch.empty_like(x.q)

    def call(to):
        return bd.attend_shared(x.q, x.c.k, x.c.v, t, l, p, m, x.offs, out=to, **x.c.kw())

    call(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for turn in range(4):
        x.q.copy_(torch.randn_like(x.q))
        l.copy_(i32([n - turn for n in x.lens]))
        m.copy_(i32([3000 - 700 * turn, 65 - turn, 1000]))
        g.replay()
        eager = call(torch.empty_like(x.q))
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
