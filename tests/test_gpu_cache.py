"""Writing and reading the paged cache on the GPU.  Everything here is defined to the last bit: a stored
value is one fp32 quotient rounded once, a value read is one fp32 product rounded once."""
import numpy as np
import pytest

import cache_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")


@pytest.fixture(autouse=True)
def _announce(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"\n[gpu case] {request.node.nodeid}", flush=True)
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def tables(rng, lens, page, width, pages):
    """Page tables of distinct pages, -1 beyond a sequence's end."""
    free = list(rng.permutation(pages))
    t = np.full((len(lens), width), -1, dtype=np.int32)
    for i, n in enumerate(lens):
        for j in range(min(width, max(0, -(-n // page)))):
            t[i, j] = free.pop()
    return t


class Pages:
    """A cache filled with a byte pattern, head-major ("head") or token-major pages."""

    def __init__(self, pages, page, hk, dim, kv, layout="head", fill=0x35):
        self.kv, self.dim = kv, dim
        width, dtype = {"bf16": (dim * 2, torch.bfloat16), "fp8": (dim, torch.float8_e4m3fn),
                        "fp4": (dim // 2, torch.uint8)}[kv]

        def make(n):
            shape = (pages, hk, page, n) if layout == "head" else (pages, page, hk, n)
            t = torch.full(shape, fill, dtype=torch.uint8, device="cuda")
            return t.transpose(1, 2) if layout == "head" else t

        self.raw = [make(width) for _ in "kv"]
        self.k, self.v = (t if kv == "fp4" else t.view(dtype) for t in self.raw)
        self.blocks = [make(dim // 32) for _ in "kv"] if kv == "fp4" else []

    def kw(self):
        return dict(zip(("k_block_scales", "v_block_scales"), self.blocks))

    def bytes(self):
        return [t.cpu().numpy() for t in (*self.raw, *self.blocks)]

    def values(self, which, scale):
        """float64 [pages, page, hk, dim] of what is stored, times the scale in fp32, rounded to bf16."""
        raw = self.raw[which].cpu().contiguous()
        if self.kv == "fp4":
            x = R.decode4(R.unpack4(raw.numpy()), self.blocks[which].cpu().numpy())
        else:
            x = raw.view(torch.bfloat16 if self.kv == "bf16" else torch.float8_e4m3fn).double().numpy()
        with np.errstate(over="ignore"):
            return R.bf16(x.astype(np.float32) * np.float32(scale))


def expected_bytes(cache, x, scale):
    """(stored bytes, scale bytes or None) of bf16 rows x (a torch tensor on the host)."""
    if not x.numel():
        return np.zeros(x.shape, np.uint8), np.zeros(x.shape, np.uint8)
    f = x.float().numpy()
    if cache.kv == "fp4":
        codes, byte = R.encode4(f, scale)
        return R.pack4(codes), byte
    if cache.kv == "fp8":
        return torch.from_numpy(R.encode8(f, scale)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), None
    if scale == 1.0:
        return x.contiguous().view(torch.uint8).numpy(), None
    y = torch.from_numpy(R.quotient(f, scale)).float().bfloat16()
    return y.view(torch.uint8).numpy(), None


def check_written(cache, before, new, scales, place):
    """Every byte of the cache: the rows written, and all else as it was."""
    want = [b.copy() for b in before]
    for which in range(2):
        data, blocks = expected_bytes(cache, new[which], scales[which])
        for row, _, pid, slot in place:
            if pid < 0:
                continue
            want[which][pid, slot] = data[row]
            if blocks is not None:
                want[2 + which][pid, slot] = blocks[row]
    got = cache.bytes()
    for g, w, name in zip(got, want, ("k", "v", "k blocks", "v blocks")):
        diff = np.argwhere(g != w)
        assert diff.size == 0, (name, len(diff), diff[:3], g[tuple(diff[0])], w[tuple(diff[0])])


def rows_of(rng, n, hk, dim, spread=True):
    x = rng.normal(size=(n, hk, dim))
    if spread:
        x *= np.exp2(rng.integers(-6, 6, (n, hk, 1)))
        x.reshape(-1)[::131] *= 40.0
    return torch.from_numpy(x).float().bfloat16() if n else torch.empty((0, hk, dim), dtype=torch.bfloat16)


# new tokens per sequence, tokens with the new ones, heads, dim, page, extra table width, layout
SIZES = [
    ([1, 1, 1], [1, 40, 17], 2, 64, 16, 0, "head"),
    ([1] * 9, [5, 0, 16, 33, -3, 64, 2, 7, 100], 3, 128, 24, 2, "token"),
    ([5, 0, 1, 70, 0, 0, 3], [5, 9, 1, 100, 0, 50, 2], 8, 128, 64, 0, "head"),
    ([333], [400], 1, 64, 7, 0, "token"),
    ([33, 65], [33, 300], 16, 64, 1, 0, "head"),
    ([2] * 40, list(range(1, 41)), 5, 128, 16, 0, "token"),
    ([0, 0], [3, 4], 2, 128, 16, 0, "head"),
]


@pytest.mark.parametrize("kv,scales", [("fp4", (1.0, 1.0)), ("fp4", (0.3, 2.0)), ("fp8", (0.0625, 0.0571)),
                                       ("bf16", (1.0, 1.0)), ("bf16", (0.5, 0.7))])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_write_then_read(case, kv, scales):
    q_lens, lens, hk, dim, page, extra, layout = SIZES[case]
    rng = np.random.default_rng(10 * case + len(kv))
    pages = sum(max(0, -(-n // page)) for n in lens) + 2
    width = max(1, max(-(-n // page) for n in lens)) + extra
    table = tables(rng, lens, page, width, pages)
    if table.shape[1] > 2:  # pages that are none
        table[0, 0], table[-1, 0] = pages, -2 ** 31
    cache = Pages(pages, page, hk, dim, kv, layout)
    n = sum(q_lens)
    new = [rows_of(rng, n, hk, dim) for _ in "kv"]
    place = R.places(q_lens, lens, table, page, pages)
    one = all(m == 1 for m in q_lens)
    offs = None if one else i32(np.concatenate([[0], np.cumsum(q_lens)]))
    kw = dict(q_offsets=offs, k_scale=scales[0], v_scale=scales[1], **cache.kw())
    before = cache.bytes()
    bd.cache_write(new[0].cuda(), new[1].cuda(), cache.k, cache.v, i32(table), i32(lens), **kw)
    check_written(cache, before, new, scales, place)
    got = bd.cache_read(cache.k, cache.v, i32(table), i32(lens), tokens=n, **kw)
    for which in range(2):
        vals = cache.values(which, scales[which])
        want = np.zeros((n, hk, dim))
        for row, _, pid, slot in place:
            if pid >= 0:
                want[row] = vals[pid, slot]
        assert np.array_equal(got[which].double().cpu().numpy(), want)


def special_rows(dim):
    """Rows of everything that can go wrong in a block."""
    rows = [np.zeros(dim), np.full(dim, -0.0), np.full(dim, 1e-40), np.full(dim, 3.3e38)]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    for e in (-130, -127, -126, -125, -124, -20, 0, 3, 100, 124, 125):
        for top in (7.0, 6.0, 4.0, 3.5, 7.0625):
            r = np.zeros(dim)
            t = np.concatenate([ties, -ties, ties * 1.0078125, ties * 0.9921875])
            r[:32] = t
            r[31] = top
            r[32:64] = np.roll(t, 5)
            with np.errstate(over="ignore"):
                rows.append(r * 2.0 ** e)
    for bad in (np.inf, -np.inf, np.nan):
        for at in (0, 31, 32, dim - 1):
            r = np.linspace(-3, 3, dim)
            r[at] = bad
            rows.append(r)
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.array(rows)).float().bfloat16()[:, None]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv,scales", [("fp4", (1.0, 0.3)), ("fp4", (1e-3, 2.0 ** 60)), ("fp4", (2.0 ** -140, 1e30)),
                                       ("fp8", (1.0, 0.3)), ("fp8", (1e-30, 1e30)), ("bf16", (1.0, 1.0))])
def test_write_special_values(kv, scales, dim):
    x = special_rows(dim)
    n = len(x)
    cache = Pages(n, 1, 1, dim, kv)
    table, lens = np.arange(n, dtype=np.int32)[:, None], [1] * n
    kw = dict(k_scale=scales[0], v_scale=scales[1], **cache.kw())
    before = cache.bytes()
    bd.cache_write(x.cuda(), x.cuda(), cache.k, cache.v, i32(table), i32(lens), **kw)
    got = cache.bytes()
    place = R.places(lens, lens, table, 1, n)
    if kv == "fp8":  # one NaN is as good as another
        for which in range(2):
            want = expected_bytes(cache, x, scales[which])[0]
            nan = (want & 0x7F) == 0x7F
            g = got[which][:, 0]
            assert np.array_equal(nan, (g & 0x7F) == 0x7F) and np.array_equal(g[~nan], want[~nan])
    else:
        check_written(cache, before, [x, x], scales, place)
    back = bd.cache_read(cache.k, cache.v, i32(table), i32(lens), **kw)
    for which in range(2):
        want = cache.values(which, scales[which])[:, 0]
        assert np.array_equal(back[which].double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("kv", ["fp4", "fp8", "bf16"])
def test_rows_of_no_sequence_and_tables_too_short(kv):
    """Rows before the first and behind the last sequence, lengths beyond the table, descending offsets."""
    rng = np.random.default_rng(3)
    hk, dim, page = 2, 64, 16
    table, lens = tables(rng, [48, 48], page, 3, 7), [60, 20]
    cache = Pages(7, page, hk, dim, kv)
    offs = [4, 30, 41]  # rows 0..3 and 41..49 are of no sequence
    new = [rows_of(rng, 50, hk, dim) for _ in "kv"]
    place = [(4 + row, b, pid, slot) for row, b, pid, slot in R.places([26, 11], lens, table, page, 7)]
    before = cache.bytes()
    bd.cache_write(new[0].cuda(), new[1].cuda(), cache.k, cache.v, i32(table), i32(lens), q_offsets=i32(offs),
                   **cache.kw())
    check_written(cache, before, new, (1.0, 1.0), place)
    out = [torch.full((50, hk, dim), 7.5, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    bd.cache_read(cache.k, cache.v, i32(table), i32(lens), q_offsets=i32(offs), k_out=out[0], v_out=out[1],
                  **cache.kw())
    for which in range(2):
        want = np.full((50, hk, dim), 7.5)
        vals = cache.values(which, 1.0)
        for row, _, pid, slot in place:
            want[row] = vals[pid, slot] if pid >= 0 else 0.0
        assert np.array_equal(out[which].double().cpu().numpy(), want)
    # offsets that descend or lie outside the rows claim no row, or some row of the call: nothing else
    state = cache.bytes()
    for offs in ([60, 70, 80], [-50, -40, -30], [50, 20, 0], [-2 ** 31, -2 ** 31, -2 ** 31]):
        bd.cache_write(new[0].cuda(), new[1].cuda(), cache.k, cache.v, i32(table), i32(lens),
                       q_offsets=i32(offs), **cache.kw())
        torch.cuda.synchronize()
        assert all(np.array_equal(a, b) for a, b in zip(cache.bytes(), state)), offs


def test_many_sequences():
    """As many sequences as a call takes, most of them empty, and rows of many heads."""
    rng = np.random.default_rng(8)
    q_lens = [0] * 1024
    for b, n in ((0, 3), (5, 1), (511, 200), (512, 1), (700, 64), (1023, 2)):
        q_lens[b] = n
    lens = [n + b % 5 for b, n in enumerate(q_lens)]
    page, hk, dim = 16, 40, 64
    pages = sum(-(-n // page) for n in lens)
    table = tables(rng, lens, page, max(-(-n // page) for n in lens), pages)
    cache = Pages(pages, page, hk, dim, "fp4")
    n = sum(q_lens)
    new = [rows_of(rng, n, hk, dim) for _ in "kv"]
    offs = i32(np.concatenate([[0], np.cumsum(q_lens)]))
    before = cache.bytes()
    bd.cache_write(new[0].cuda(), new[1].cuda(), cache.k, cache.v, i32(table), i32(lens), q_offsets=offs,
                   **cache.kw())
    check_written(cache, before, new, (1.0, 1.0), R.places(q_lens, lens, table, page, pages))


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_strided_rows(kv):
    """Rows cut out of a joint projection, read back into one; a single head and token with any stride."""
    rng = np.random.default_rng(9)
    hk, dim, page, n = 3, 128, 16, 21
    joint = rows_of(rng, n, 3 * hk, dim).cuda()
    k, v = joint[:, hk:2 * hk], joint[:, 2 * hk:]
    table, lens = tables(rng, [n], page, 2, 4), [n]
    cache = Pages(4, page, hk, dim, kv, "token")
    offs = i32([0, n])
    before = cache.bytes()
    bd.cache_write(k, v, cache.k, cache.v, i32(table), i32(lens), q_offsets=offs, **cache.kw())
    check_written(cache, before, [k.cpu(), v.cpu()], (1.0, 1.0), R.places([n], lens, table, page, 4))
    out = torch.zeros((n, 3 * hk, dim), dtype=torch.bfloat16, device="cuda")
    a, b = bd.cache_read(cache.k, cache.v, i32(table), i32(lens), q_offsets=offs, **cache.kw(), tokens=n)
    bd.cache_read(cache.k, cache.v, i32(table), i32(lens), q_offsets=offs, k_out=out[:, :hk], v_out=out[:, 2 * hk:],
                  **cache.kw())
    assert torch.equal(out[:, :hk], a) and torch.equal(out[:, 2 * hk:], b) and not out[:, hk:2 * hk].any()
    one = Pages(1, 1, 1, dim, kv)
    x = joint[0, :1].as_strided((1, 1, dim), (3, 5, 1))
    bd.cache_write(x, x, one.k, one.v, i32([[0]]), i32([1]), **one.kw())
    got = bd.cache_read(one.k, one.v, i32([[0]]), i32([1]), **one.kw())[0]
    want, byte = expected_bytes(one, x.cpu(), 1.0)
    assert np.array_equal(one.bytes()[0].reshape(-1), want.reshape(-1)) and torch.isfinite(got).all()


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 bytes apart (their scale bytes more than 2^28)."""
    hk, dim, page = 2, 128, 16
    apart = (1 << 32) + (1 << 12)
    raw = [torch.zeros(apart + (1 << 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    blocks = [torch.zeros(apart // 16 + (1 << 12), dtype=torch.uint8, device="cuda") for _ in "kv"]
    pages = [t.as_strided((2, page, hk, dim // 2), (apart, dim // 2, page * dim // 2, 1)) for t in raw]
    small = [t.as_strided((2, page, hk, dim // 32), (apart // 16, dim // 32, page * dim // 32, 1)) for t in blocks]
    rng = np.random.default_rng(4)
    new = [rows_of(rng, 20, hk, dim) for _ in "kv"]
    kw = dict(q_offsets=i32([0, 20]), k_block_scales=small[0], v_block_scales=small[1])
    bd.cache_write(new[0].cuda(), new[1].cuda(), *pages, i32([[0, 1]]), i32([20]), **kw)
    got = bd.cache_read(*pages, i32([[0, 1]]), i32([20]), tokens=20, **kw)
    for which in range(2):
        codes, byte = R.encode4(new[which].float().numpy())
        assert np.array_equal(pages[which][1, :4].cpu().numpy(), R.pack4(codes[16:]))
        assert np.array_equal(small[which][1, :4].cpu().numpy(), byte[16:])
        assert np.array_equal(got[which].double().cpu().numpy(), R.decode4(codes, byte))
        # nothing else was written
        assert int((raw[which] != 0).sum()) == int((R.pack4(codes) != 0).sum())


@pytest.mark.parametrize("kv", ["fp4", "fp8"])
def test_captured_and_replayed(kv):
    """A step's write and read in a graph, replayed with other tables and values."""
    rng = np.random.default_rng(6)
    hk, dim, page, n = 2, 128, 16, 6
    cache = Pages(9, page, hk, dim, kv)
    k, v = (rows_of(rng, n, hk, dim).cuda() for _ in "kv")
    table, lens = i32(tables(rng, [30] * n, page, 1, 9)), i32([1] * n)
    out = [torch.zeros((n, hk, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def step():
        bd.cache_write(k, v, cache.k, cache.v, table, lens, **cache.kw())
        bd.cache_read(cache.k, cache.v, table, lens, k_out=out[0], v_out=out[1], **cache.kw())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        k.copy_(rows_of(rng, n, hk, dim))
        v.copy_(rows_of(rng, n, hk, dim))
        lens.fill_(1 + 3 * i)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        after = cache.bytes()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out))
        assert all(np.array_equal(a, b) for a, b in zip(after, cache.bytes()))


def test_on_another_stream():
    rng = np.random.default_rng(12)
    hk, dim, page, n = 2, 64, 16, 40
    cache = Pages(4, page, hk, dim, "fp4")
    k, v = (rows_of(rng, n, hk, dim).cuda() for _ in "kv")
    table, lens, offs = i32([[2, 0, 3]]), i32([n]), i32([0, n])
    bd.cache_write(k, v, cache.k, cache.v, table, lens, q_offsets=offs, **cache.kw())
    want = bd.cache_read(cache.k, cache.v, table, lens, q_offsets=offs, tokens=n, **cache.kw())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = set()
    for x in want:
        held = [torch.empty_like(x) for _ in range(4)]
        freed |= {h.data_ptr() for h in held}
        del held
    got = bd.cache_read(cache.k, cache.v, table, lens, q_offsets=offs, tokens=n, stream=s.cuda_stream, **cache.kw())
    assert not freed & {x.data_ptr() for x in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_the_binding():
    rng = np.random.default_rng(1)
    c4, c8 = Pages(4, 16, 2, 64, "fp4"), Pages(4, 16, 2, 64, "fp8")
    k = rows_of(rng, 3, 2, 64).cuda()
    table, lens = i32([[0], [1], [2]]), i32([1, 1, 1])

    def write(cache=c4, k=k, v=None, table=table, lens=lens, **kw):
        return bd.cache_write(k, k if v is None else v, cache.k, cache.v, table, lens,
                              **{**cache.kw(), **kw})

    write()
    bad = torch.zeros((4, 16, 2, 2), dtype=torch.uint8, device="cuda")  # not head-major
    for kw, kind in [(dict(k_block_scales=None), TypeError), (dict(k_block_scales=bad), ValueError),
                     (dict(v_block_scales=c4.blocks[1][:, :8]), ValueError),
                     (dict(v_block_scales=c4.blocks[1].cpu()), TypeError),
                     (dict(v_block_scales=c4.blocks[1].view(torch.int8)), TypeError),
                     (dict(k=k.float()), TypeError), (dict(k=k.cpu()), TypeError), (dict(k=k[:, :1]), ValueError),
                     (dict(k=k[:2]), bd.BitDeltaError), (dict(lens=i32([1, 1])), ValueError),
                     (dict(table=table[:2]), ValueError), (dict(table=table.long()), TypeError),
                     (dict(q_offsets=i32([0, 1])), ValueError),
                     (dict(cache=c8, k_block_scales=c4.blocks[0]), ValueError),
                     (dict(k=k.transpose(1, 2)), ValueError)]:
        with pytest.raises(kind):
            write(**kw)
    with pytest.raises(bd.BitDeltaError):
        write(k_scale=0.0)
    with pytest.raises(ValueError):
        bd.cache_read(c4.k, c4.v, table, lens, q_offsets=i32([0, 1, 2, 3]), **c4.kw())
    with pytest.raises(ValueError):
        bd.cache_read(c4.k, c4.v, table, lens, k_out=k, **c4.kw())
    with pytest.raises(ValueError):
        bd.cache_read(c4.k, c4.v, table, lens, tokens=2, k_out=k, v_out=k, **c4.kw())
    assert bd.cache_write(k[:0], k[:0], c4.k, c4.v, table[:0], lens[:0], **c4.kw())[0] is c4.k
