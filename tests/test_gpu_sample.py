"""Token sampling on the GPU against the 64-bit form.  Tokens have to be equal; the log-probability
is rounded to float32 once (half a step, 2^-24 of it) from fp64 sums."""
import numpy as np
import pytest

import sample_ref as R

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


def f32(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).cuda()


def run(logits, u, t=None, k=None, p=None, m=None, **kw):
    """(tokens, logprob) as arrays for host parameter arrays."""
    arg = lambda x: None if x is None else f32(x)
    kk = None if k is None else torch.from_numpy(np.asarray(k, dtype=np.int32)).cuda()
    tok, lp = bd.sample(logits, f32(u), temperature=arg(t), top_k=kk, top_p=arg(p), min_p=arg(m),
                        return_logprob=True, **kw)
    return tok.cpu().numpy(), lp.cpu().numpy()


def check(logits, u, t=None, k=None, p=None, m=None, **kw):
    tok, lp = run(logits, u, t, k, p, m, **kw)
    x = logits.double().cpu().numpy()
    pick = lambda a, r, d: d if a is None else float(np.float32(a[r]))
    for r in range(x.shape[0]):
        want, wl = R.sample_row(x[r], float(np.float32(u[r])), pick(t, r, 1.0),
                                0 if k is None else int(k[r]), pick(p, r, 1.0), pick(m, r, 0.0))
        what = (r, u[r], pick(t, r, 1.0), None if k is None else k[r], pick(p, r, 1.0), pick(m, r, 0.0))
        assert tok[r] == want, (what, tok[r], want)
        if want < 0:
            assert np.isneginf(lp[r]), what
        else:
            assert abs(lp[r] - wl) <= 2.0 ** -24 * abs(wl) + 1e-12, (what, lp[r], wl)


def peaked(rng, rows, vocab, dtype):
    x = rng.normal(scale=2.0, size=(rows, vocab))
    for r in range(rows):
        hot = rng.integers(0, vocab, size=min(24, vocab))
        x[r, hot] = rng.normal(13, 2.5, size=hot.size)
    x = torch.from_numpy(x.astype(np.float32)).cuda()
    return x.to(dtype)


def settings(rng, rows):
    return dict(t=rng.choice([0.0, 0.3, 0.7, 1.0, 1.5], size=rows),
                k=rng.choice([0, 0, 1, 2, 40, 200, 1000, 1024], size=rows),
                p=rng.choice([1.0, 1.0, 0.3, 0.9, 0.95, 0.999], size=rows),
                m=rng.choice([0.0, 0.0, 0.0, 0.05, 0.3], size=rows))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 63, 64, 65, 500, 1024, 1025, 4099, 32000, 50001])
def test_sizes(vocab, dtype):
    rng = np.random.default_rng(vocab)
    rows = 24 if vocab < 5000 else 12
    check(peaked(rng, rows, vocab, dtype), rng.random(rows), **settings(rng, rows))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_flat_rows(dtype):
    """Distributions whose kept tokens are most of the vocabulary."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(scale=0.7, size=(14, 20011)).astype(np.float32)).cuda().to(dtype)
    u = rng.random(14)
    u[:3] = 0.0, 1.0 - 2.0 ** -24, 0.5
    check(x, u)
    check(x, u, p=np.linspace(0.05, 0.999, 14))
    check(x, u, m=np.linspace(0.01, 0.9, 14))
    check(x, u, k=rng.integers(1025, 20011, size=14), p=np.linspace(0.2, 1.0, 14))
    check(x, u, k=rng.integers(1025, 20011, size=14))
    check(x, u, k=rng.integers(1025, 20011, size=14), m=np.full(14, 0.05))
    check(x, u, t=np.linspace(0.1, 8.0, 14), p=np.full(14, 0.9), m=np.full(14, 0.01))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [5, 3001])
def test_ties(vocab, dtype):
    """Equal logits go by index, however many there are, -0 and +0 among them."""
    rng = np.random.default_rng(2)
    x = torch.full((10, vocab), 1.5, device="cuda")
    x[1] = 0.0
    x[1, ::2] = -0.0
    x[2, vocab // 2] = 3.0
    x[3:6] = torch.from_numpy(rng.integers(0, 3, size=(3, vocab)).astype(np.float32)).cuda()
    x[6:] = torch.from_numpy(rng.integers(0, 40, size=(4, vocab)).astype(np.float32) / 8).cuda()
    x = x.to(dtype)
    u = rng.random(10)
    check(x, u)
    check(x, u, p=np.linspace(0.1, 0.9, 10))
    check(x, u, k=rng.integers(1, vocab + 3, size=10))
    check(x, u, t=np.zeros(10))
    check(x, u, m=np.full(10, 0.5), p=np.full(10, 0.6))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [8192, 9001, 70003])
def test_thousands_of_nearly_equal_logits(vocab, dtype):
    """More tokens around a border than are ever collected."""
    rng = np.random.default_rng(vocab)
    x = torch.zeros((12, vocab), device="cuda")
    x[1, ::2] = -0.0
    x[2:4] = torch.from_numpy(rng.integers(0, 2, size=(2, vocab)).astype(np.float32))
    x[4:8] = torch.from_numpy(rng.normal(scale=0.004, size=(4, vocab)).astype(np.float32))
    x[8:] = torch.from_numpy(rng.normal(loc=-20, scale=0.004, size=(4, vocab)).astype(np.float32))
    x[9, 5], x[11, 77] = -10.0, -19.0
    x[5, 100:200], x[6, ::3], x[10, 1::2] = float("nan"), -float("inf"), -float("inf")
    x = x.to(dtype)
    u = rng.random(12)
    u[0], u[1], u[4], u[8] = 0.5, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24, 0.0
    check(x, u)
    check(x, u, p=np.linspace(0.1, 0.9, 12))
    check(x, u, k=rng.integers(1, 60, size=12))
    check(x, u, k=rng.integers(1025, vocab, size=12), p=np.linspace(0.2, 1.0, 12))
    check(x, u, m=np.full(12, 0.5), p=np.linspace(1.0, 0.3, 12))
    check(x, u, t=np.linspace(0.01, 4, 12), m=np.full(12, 0.9))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_infinite_and_nan_logits(dtype):
    rng = np.random.default_rng(3)
    x = peaked(rng, 12, 9001, torch.float32).cpu().numpy()
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2, :-1] = -np.inf
    x[3, rng.random(9001) < 0.99] = -np.inf
    x[4, rng.random(9001) < 0.5] = np.nan
    x[5] = np.nan
    x[6, [10, 5000, 9000]] = np.inf
    x[7, 17] = np.inf
    x[8] = np.finfo(np.float32).min
    x[8, 4000:4003] = -np.inf
    x[9] *= 1e30
    x[10, 5:] = -np.inf
    x[11, ::2] = -np.inf
    x = torch.from_numpy(x).cuda().to(dtype)
    u = rng.random(12)
    for kw in (dict(), dict(k=np.full(12, 50)), dict(p=np.full(12, 0.9)), dict(m=np.full(12, 0.1)),
               dict(k=np.full(12, 800), p=np.full(12, 0.99), t=np.full(12, 2.0)),
               dict(t=np.zeros(12)), dict(k=np.full(12, 2000), p=np.full(12, 0.5))):
        check(x, u, **kw)


def test_parameters_at_their_ends():
    """Off values, NaN, values beyond their range."""
    rng = np.random.default_rng(4)
    x = peaked(rng, 16, 3000, torch.float32)
    u = rng.random(16)
    base = run(x, u)
    nan = np.full(16, np.nan)
    for kw in (dict(k=np.full(16, -3)), dict(k=np.full(16, 5000)), dict(p=np.full(16, 1.5)),
               dict(p=nan), dict(m=np.full(16, -0.5)), dict(m=nan), dict(t=np.ones(16))):
        assert all(np.array_equal(a, b) for a, b in zip(base, run(x, u, **kw))), kw
    top = x.argmax(1).cpu().numpy()
    for kw in (dict(t=nan), dict(t=np.full(16, -1.0)), dict(p=np.zeros(16)), dict(p=np.full(16, -1.0)),
               dict(m=np.full(16, 1.5)), dict(k=np.ones(16)), dict(t=np.full(16, 1e-30))):
        tok, lp = run(x, u, **kw)
        assert np.array_equal(tok, top) and not lp.any(), kw
    check(x, np.full(16, 0.0)), check(x, np.full(16, 1.0 - 2.0 ** -24))
    lo, hi = run(x, np.full(16, -1.0)), run(x, np.full(16, 2.0), k=np.full(16, 7))
    assert np.array_equal(lo[0], run(x, np.zeros(16))[0])
    order = torch.argsort(x, dim=1, descending=True, stable=True).cpu().numpy()
    assert np.array_equal(hi[0], order[:, 6])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_offsets(dtype):
    """Rows that are slices of wider ones, at every offset from a 16-byte border."""
    rng = np.random.default_rng(5)
    wide = peaked(rng, 6, 2100, dtype)
    for off in range(9):
        for n in (2050, 2053):
            check(wide[:, off:off + n], rng.random(6), k=np.full(6, 40), p=np.full(6, 0.95))


def test_rows_beyond_the_bins():
    """More than 2^20 tokens: no bins; borders by bisection where there is no top-k."""
    rng = np.random.default_rng(8)
    vocab = (1 << 20) + 77
    x = torch.from_numpy(rng.normal(scale=2.0, size=(3, vocab)).astype(np.float32)).cuda()
    x[1, 1 << 20] = 14.0
    x[2, ::2] = 0.25
    u = rng.random(3)
    check(x, u)
    check(x, u, p=np.array([0.9, 0.5, 0.99]), k=np.array([0, 30, 5000]))
    check(x, u, t=np.array([0.5, 0.0, 2.0]), m=np.array([0.1, 0.0, 0.01]))


def test_rows_beyond_32_bit_offsets():
    vocab, rows = 200000, 11000  # 4.4 GB of bf16
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    x[-1, 123456], x[-2, 77] = 30.0, 30.0
    tok = bd.sample(x, f32(np.full(rows, 0.25)), top_k=torch.full((rows,), 4, dtype=torch.int32, device="cuda"))
    assert int(tok[-1]) == 123456 and int(tok[-2]) == 77
    assert bool((tok[:-2] == 1).all())


def test_graph_replays_and_other_streams():
    rng = np.random.default_rng(6)
    x, u = peaked(rng, 9, 30011, torch.bfloat16), f32(rng.random(9))
    p = f32(np.full(9, 0.97))
    call = lambda: bd.sample(x, u, top_p=p, return_logprob=True)
    eager = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = [t.clone() for t in call()]
    by_handle = bd.sample(x, u, top_p=p, return_logprob=True, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for got in (side, by_handle):
        assert all(torch.equal(a, b) for a, b in zip(eager, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = call()
    for _ in range(4):
        u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        torch.randn(1 << 20, device="cuda").sum().item()
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_draws_follow_the_distribution():
    """Many u over one row: each token's share is its weight's."""
    n = 4096
    w = np.array([0.4, 0.3, 0.2, 0.1])
    x = f32(np.tile(np.log(w), (n, 1)))
    tok = bd.sample(x, f32((np.arange(n) + 0.5) / n)).cpu().numpy()
    assert np.all(np.abs(np.bincount(tok, minlength=4) / n - w) <= 1.0 / n)


def test_binding_refusals():
    x, u = torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(TypeError):
        bd.sample(x.half(), u)
    with pytest.raises(TypeError):
        bd.sample(x.cpu(), u)
    with pytest.raises(TypeError):
        bd.sample(x, u.double())
    with pytest.raises(ValueError):
        bd.sample(x[:, ::2], u)
    with pytest.raises(ValueError):
        bd.sample(x, u[:1])
    with pytest.raises(ValueError):
        bd.sample(x[0], u)
    with pytest.raises(TypeError):
        bd.sample(x, u, top_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert bd.sample(x[:0], u[:0]).numel() == 0
