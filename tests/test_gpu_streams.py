"""Calls on a stream given by its handle: what they allocate belongs to that stream."""
import numpy as np
import pytest

import test_gpu_attend as A

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


def _calls():
    """(name, call by stream handle) of each operator that makes its results itself."""
    rng = np.random.default_rng(51)
    table, k, v, _, _, q, _, _ = A._window_setup(rng, [1, 1], [1900, 300])
    t, l = A.i32(table), A.i32([1900, 300])
    x, u = torch.randn((9, 5000), device="cuda"), torch.rand(9, device="cuda")
    return [
        ("shared", lambda **kw: bd.attend_shared(q, k, v, t, l, t[:1].contiguous(), l[:1].contiguous(),
                                                 [0, 2], return_lse=True, **kw)),
        ("window", lambda **kw: bd.attend_window(q, k, v, t, l, 4000, 4, return_lse=True, **kw)),
        ("sample", lambda **kw: bd.sample(x, u, return_logprob=True, **kw)),
    ]


@pytest.mark.parametrize("which", range(3))
def test_results_on_another_stream_take_no_memory_of_the_current_one(which):
    """A call on a stream given by its handle runs without an order to the current stream's work, so
    that memory freed on the current stream, which that work may still use, must not become its results."""
    name, call = _calls()[which]
    want = [x.clone() for x in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = set()
    for x in want:  # blocks of the results' sizes, free on the current stream
        held = [torch.empty_like(x) for _ in range(4)]
        freed |= {h.data_ptr() for h in held}
        del held
    got = call(stream=s.cuda_stream)
    assert not freed & {x.data_ptr() for x in got}, name
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    # nor do later results on that stream take memory that the current stream may still read
    place = {x.data_ptr() for x in got}
    torch.cuda._sleep(20_000_000)  # about 10 ms of the current stream's time
    copies = [x.clone() for x in got]
    del got, x
    again = call(stream=s.cuda_stream)
    assert not place & {y.data_ptr() for y in again}, name
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)), name
    assert all(torch.equal(a, b) for a, b in zip(again, want)), name


def test_workspace_on_another_stream_takes_no_memory_of_the_current_one():
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = torch.empty(5 << 20, dtype=torch.uint8, device="cuda")
    place = held.data_ptr()
    del held
    ws = bd._temp(5 << 20, torch.device("cuda:0"), s.cuda_stream)
    assert ws.data_ptr() != place and ws.numel() == 5 << 20


def test_calls_on_the_default_stream_by_its_handle_from_another():
    s = torch.cuda.Stream()
    for name, call in _calls():
        want = [x.clone() for x in call()]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            got = call(stream=torch.cuda.default_stream().cuda_stream)
            same = call(stream=s.cuda_stream)
        torch.cuda.synchronize()
        for a, b, c in zip(got, same, want):
            assert torch.equal(a, c) and torch.equal(b, c), name


def test_fused_linears_on_another_stream_take_no_memory_of_the_current_one():
    rng = np.random.default_rng(52)
    w = torch.from_numpy(rng.normal(size=(512, 256)).astype(np.float32)).bfloat16().cuda()
    words = torch.empty((512, 8), dtype=torch.int32, device="cuda")
    alpha = torch.empty(1, dtype=torch.float32, device="cuda")
    bd.compress(torch.from_numpy(rng.normal(size=(512, 256)).astype(np.float32)).cuda(), words, alpha)
    x = torch.randn((3, 256), device="cuda").bfloat16()
    s = torch.cuda.Stream()
    calls = [lambda **kw: bd.matmul(x, w, [(words, alpha)], [0, 3], [0], **kw),
             lambda **kw: bd.reconstruct(w, (words, alpha), **kw)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        held = [torch.empty_like(want) for _ in range(4)]
        freed = {h.data_ptr() for h in held}
        del held
        got = call(stream=s.cuda_stream)
        assert got.data_ptr() not in freed
        torch.cuda.synchronize()
        assert torch.equal(got, want)
