"""The decoder of examples/decode.py with a quantised cache: every attention call of its steps against the
same call over a bf16 cache that holds what the quantised one stands for (read back by cache_read).

Both sides round each weight to bf16 (2^-8 of it, so 2^-8 of a row's largest value together) and the result
(2^-8 of it)."""
import dataclasses

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

import test_gpu_decode_example as T  # noqa: E402

D = T.D


@pytest.mark.parametrize("kv", ["fp8", "fp4"])
def test_decode_from_a_quantised_cache(kv, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    device = torch.device("cuda:0")
    cfg = dataclasses.replace(D.Config(), kv=kv)
    rng = np.random.default_rng(6)
    model = D.Model(cfg, device, seed=4)
    variant = np.array([2, 0, 0, 1, 2])
    prompts = [rng.integers(0, cfg.vocab, cfg.page * n) for n in (9, 2, 4)]
    calls = []
    real = {"attend_window": bd.attend_window, "attend_shared": bd.attend_shared}

    def checked(name):
        def call(q, k, v, *args, **kw):
            scales = {n: kw.pop(n) for n in list(kw) if n.endswith("scale") or n.endswith("scales")}
            got = real[name](q, k, v, *args, **kw, **scales)
            pages, page = k.shape[:2]
            every = torch.arange(pages, dtype=torch.int32, device=device)
            plain = bd.cache_read(k, v, every[:, None].contiguous(), torch.full_like(every, page),
                                  q_offsets=torch.arange(pages + 1, dtype=torch.int32, device=device) * page,
                                  tokens=pages * page, **scales)
            want = real[name](q, *(x.view(pages, page, cfg.kv_heads, cfg.head_dim) for x in plain), *args, **kw)
            a, b = got.double(), want.double()
            tol = 2 * 2.0 ** -8 * (b.abs() + plain[1].double().abs().max()) + 1e-5
            assert ((a - b).abs() <= tol).all() and torch.isfinite(a).all()
            calls.append(name)
            return got
        return call

    for name in real:
        monkeypatch.setattr(D.bd, name, checked(name))
    engine = D.Engine(model, variant, prompts, cfg.page + 3, device)
    engine.prefill()
    for _ in range(cfg.page + 3):
        tokens = torch.from_numpy(rng.integers(0, cfg.vocab, len(variant))).to(device)
        assert torch.isfinite(engine.decode(tokens)).all()
    assert calls.count("attend_shared") == 2 * (cfg.page + 3)
    assert calls.count("attend_window") == 4 + 2 * (cfg.page + 3)
