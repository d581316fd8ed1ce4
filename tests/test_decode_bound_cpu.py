"""The bound that the decoder of examples/decode.py is held to, without a GPU: the roundings it allows for
stay well below it, and a mask that is wrong by one token in the layers with a window exceeds it."""
import dataclasses

import numpy as np
import pytest

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

import decode_model as M  # noqa: E402


@pytest.fixture(scope="module")
def model():
    return M.HostModel(M.D.Config(), torch.device("cpu"), seed=3)


@pytest.mark.parametrize("variant,n", [(1, 34), (0, 74), (2, 160)])
def test_roundings_fit_the_bound_and_wrong_masks_do_not(model, variant, n):
    tokens = np.random.default_rng(n).integers(0, model.cfg.vocab, n)
    cfg = model.cfg
    ref = M.T.plain_logits(model, variant, tokens)
    assert M.error(M.rounded_logits(model, variant, tokens), ref) <= M.BOUND / 2
    for wrong in (dict(sinks=0), dict(sinks=cfg.sinks - 1), dict(window=cfg.window - 1),
                  dict(window=cfg.window + 1), dict(window=10 ** 6)):
        model.cfg = dataclasses.replace(cfg, **wrong)
        try:
            off = M.error(M.T.plain_logits(model, variant, tokens), ref)
        finally:
            model.cfg = cfg
        assert off > M.BOUND, (wrong, off)
