"""The decoder of examples/decode.py against the model recomputed in 64 bits, within a bound that a mask
wrong by one token exceeds (decode_model.py derives it; test_decode_bound_cpu.py shows what it tells
apart)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

import decode_model as M  # noqa: E402


def test_decode_logits_within_the_roundings():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    device = torch.device("cuda:0")
    cfg = M.D.Config()
    rng = np.random.default_rng(9)
    model = M.D.Model(cfg, device, seed=3)
    variant = np.array([1, 0, 2, 0, 1])
    prompts = [rng.integers(0, cfg.vocab, cfg.page * n) for n in (4, 2, 9)]
    steps = cfg.page + 2
    engine = M.D.Engine(model, variant, prompts, steps, device)
    engine.prefill()
    lists = [list(prompts[variant[r]]) for r in engine.perm]
    for step in range(steps):
        tokens = rng.integers(0, cfg.vocab, len(variant))
        for b, t in enumerate(tokens):
            lists[b].append(int(t))
        got = engine.decode(torch.from_numpy(tokens).to(device)).cpu().double().numpy()
        if step in (0, 1, cfg.page - 1, cfg.page, steps - 1):
            for b in range(len(variant)):
                err = M.error(got[b], M.T.plain_logits(model, variant[engine.perm[b]], np.array(lists[b])))
                print(f"step {step} request {b}: {err:.2e}", flush=True)
                assert err <= M.BOUND, (step, b, err)
