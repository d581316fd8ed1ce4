"""Token sampling at the ends of its settings, against the 64-bit form: tokens have to be equal, the
log-probability is rounded to float32 once from fp64 sums (half a step, 2^-24 of it)."""
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


def put(x, dtype=np.float32):
    return None if x is None else torch.from_numpy(np.asarray(x, dtype=dtype)).cuda()


def check(logits, u, t=None, k=None, p=None, m=None):
    """Against the 64-bit form; an infinite temperature weighs every token that is not masked alike,
    as 1e300 does in 64 bits."""
    tok, lp = bd.sample(logits, put(u), put(t), put(k, np.int32), put(p), put(m), return_logprob=True)
    tok, lp, x = tok.cpu().numpy(), lp.cpu().numpy(), logits.double().cpu().numpy()
    pick = lambda a, r, d: d if a is None else float(np.float32(a[r]))  # noqa: E731
    for r in range(x.shape[0]):
        want, wl = R.sample_row(x[r], pick(u, r, 0.0), min(pick(t, r, 1.0), 1e300),
                                0 if k is None else int(k[r]), pick(p, r, 1.0), pick(m, r, 0.0))
        assert tok[r] == want, (r, tok[r], want)
        assert abs(lp[r] - wl) <= 2.0 ** -24 * abs(wl) + 1e-12, (r, lp[r], wl)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,allowed", [(7, 1.0), (1025, 1.0), (2048, 1.0), (4096, 1.0), (9001, 1.0),
                                           (100003, 0.02), (100003, 0.0002)])
def test_infinite_temperature_is_a_uniform_draw(vocab, allowed, dtype):
    rng = np.random.default_rng(vocab)
    rows = 8
    x = rng.normal(scale=3.0, size=(rows, vocab)).astype(np.float32)
    if allowed < 1:
        x[rng.random(x.shape) >= allowed] = -np.inf
        x[:, 17] = 2.0
    x = torch.from_numpy(x).cuda().to(dtype)
    u, t = rng.random(rows), np.full(rows, np.inf)
    check(x, u, t)
    check(x, u, t, p=np.linspace(0.1, 0.95, rows))
    check(x, u, t, m=np.full(rows, 0.5))
    check(x, u, t, m=np.full(rows, 0.5), p=np.linspace(0.95, 0.1, rows))
    check(x, u, t, k=np.full(rows, 40))
    check(x, u, t, k=np.full(rows, 1500), p=np.full(rows, 0.7))
    check(x, u, np.where(np.arange(rows) % 2, np.inf, 0.8))
    check(x, u, np.full(rows, 3e38))


def test_draws_from_a_long_tail_of_equal_logits():
    """One large logit and 2^17 equal ones far below: a draw among those is at the token where the
    definition puts it.  Sums of weights are off by 2^-30 each (header), the running one and the whole,
    so the token by at most 2^-29 / w, plus one for a border."""
    vocab, rows = (1 << 17) - 1, 24
    # of the floats around ln 1e-9 the one whose weight is farthest from a multiple of 2^-43
    cand = np.float32(-20.7) - np.arange(4000, dtype=np.float32) * np.float32(2.0 ** -19)
    w = np.exp(cand.astype(np.float64))
    at = np.argmin(np.abs(w * 2.0 ** 43 % 1.0 - 0.45))
    x = np.full((rows, vocab), cand[at], np.float32)
    x[:, 5] = 0.0
    u = (1.0 - np.arange(1, rows + 1) * 2.0 ** -18).astype(np.float32)
    tok, lp = bd.sample(torch.from_numpy(x).cuda(), put(u), return_logprob=True)
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    total = 1.0 + (vocab - 1) * w[at]
    for r in range(rows):
        j = np.floor((float(u[r]) * total - 1.0) / w[at])  # of the equal ones, in the order of indices
        assert 0 < j < vocab - 1
        want = j if j < 5 else j + 1
        assert abs(tok[r] - want) <= 2.0 ** -29 / w[at] + 1, (r, tok[r], want)
        assert abs(lp[r] - (np.log(w[at]) - np.log(total))) <= 2.0 ** -24 * abs(lp[r]) + 2.0 ** -29


def test_more_rows_than_one_launch_takes():
    """2^22 rows of 1024 threads are more than a grid holds."""
    rows = (1 << 22) + 3
    x = torch.zeros((rows, 3), device="cuda")
    x[::2, 1], x[1::2, 2] = 5.0, 5.0
    x[-1] = torch.tensor([9.0, 0.0, 0.0])
    u = torch.zeros(rows, device="cuda")
    tok, lp = bd.sample(x, u, top_k=torch.ones(rows, dtype=torch.int32, device="cuda"),
                        return_logprob=True)
    want = 1 + torch.arange(rows, device="cuda", dtype=torch.int32) % 2
    want[-1] = 0
    assert torch.equal(tok, want) and not bool(lp.any())


@pytest.mark.parametrize("vocab", [5, 1500, 9001])
def test_min_p_of_one_at_an_infinite_temperature_keeps_every_token(vocab):
    rng = np.random.default_rng(vocab)
    x = rng.normal(size=(6, vocab)).astype(np.float32)
    x[3:, ::3] = -np.inf
    u = np.linspace(0.01, 0.99, 6)
    check(torch.from_numpy(x).cuda(), u, np.full(6, np.inf), m=np.ones(6))
    check(torch.from_numpy(x).cuda(), u, np.full(6, 3e38), m=np.ones(6))
    check(torch.from_numpy(np.round(x)).cuda(), u, m=np.ones(6))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("equal", [2, 6, 48, 64, 66, 1062, 2048, 4096])
def test_borders_between_equal_tokens(equal, dtype):
    """Half, a quarter and three quarters of the weight of n equal tokens are whole numbers of them; what
    else the row holds weighs less than fp64 resolves, or is masked."""
    rng = np.random.default_rng(equal)
    vocab, rows = 5003, 9
    x = np.full((rows, vocab), -60.0, np.float32)
    x[3:6] = -np.inf
    x[6:] = -1000.0 - 4.0 * rng.integers(0, 50, size=(3, vocab))
    for r in range(rows):
        x[r, rng.permutation(vocab)[:equal]] = (0.0, 3.0, -7.5)[r % 3]
    x = torch.from_numpy(x).cuda().to(dtype)
    share = np.tile([0.5, 0.25, 0.75], 3)
    check(x, share)
    check(x, np.full(rows, 1.0 - 2.0 ** -24), p=share)
    check(x, share, p=share)
    check(x, np.tile([0.25, 0.5, 0.5], 3), p=share, m=np.full(rows, 0.9))
    check(x, share, k=np.full(rows, 4500))
    check(x, np.full(rows, 1.0 - 2.0 ** -24), k=np.full(rows, 4500), p=share)
    check(x, share, t=np.full(rows, 0.1), p=share)
