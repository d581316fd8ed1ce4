"""The decoder of examples/decode.py against the same model recomputed in 64 bits from whole
token lists: no cache, no sharing, every mask written out.

Tolerance on a row of logits (relative L2): the library's linears are allowed 2e-2 each in other
tests and reach a few 2^-8; what a layer rounds to bf16 on the way (norm, q, k, v, attention
weights and output, o, sum, norm, gate, up, their product, down, sum) is 13 half steps of 2^-8
relative, which add up at worst, through 4 layers and the last norm to 53 of them."""
import os
import sys

import numpy as np
import pytest

import sample_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode as D  # noqa: E402

TOL = 53 * 2.0 ** -8


def weights(linear, v):
    """W_base + alpha sign of a variant, float64."""
    w, variants = linear
    words, alpha, _ = variants[v]
    bits = np.unpackbits(words.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    return w.double().cpu().numpy() + float(alpha) * (2.0 * bits - 1.0)


def norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)


def rotary(x):
    half = x.shape[-1] // 2
    angle = np.arange(len(x))[:, None] * 10000.0 ** (-np.arange(half) / half)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, a * s + b * c], -1)


def plain_logits(model, v, tokens):
    """Logits of the last token of a request of variant v, from its whole list of tokens."""
    cfg = model.cfg
    x = model.embed.double().cpu().numpy()[tokens]
    n = len(tokens)
    back = np.arange(n)[:, None] - np.arange(n)[None, :]
    for i, layer in enumerate(model.layers):
        w = {name: weights(lin, v) for name, lin in layer.items()}
        y = norm(x)
        q, k, val = ((y @ w[c].T).reshape(n, -1, cfg.head_dim) for c in "qkv")
        q, k = rotary(q), rotary(k)
        seen = back >= 0
        if i % 2:
            seen &= (back < cfg.window) | (np.arange(n)[None, :] < cfg.sinks)
        out = np.empty_like(q)
        for h in range(cfg.heads):
            g = h // (cfg.heads // cfg.kv_heads)
            s = np.where(seen, q[:, h] @ k[:, g].T / np.sqrt(cfg.head_dim), -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            out[:, h] = (p / p.sum(1, keepdims=True)) @ val[:, g]
        x = x + out.reshape(n, -1) @ w["o"].T
        y = norm(x)
        gate, up = y @ w["gate"].T, y @ w["up"].T
        x = x + (gate / (1 + np.exp(-gate)) * up) @ w["down"].T
    return norm(x[-1]) @ weights(model.head, v).T


def test_decode_matches_plain_recomputation():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    device = torch.device("cuda:0")
    cfg = D.Config()
    rng = np.random.default_rng(5)
    model = D.Model(cfg, device, seed=3)
    variant = np.array([2, 0, 0, 2, 2, 0, 1, 0, 2])
    prompts = [rng.integers(0, cfg.vocab, cfg.page * n) for n in (9, 2, 4)]
    steps = 20  # past a page
    engine = D.Engine(model, variant, prompts, steps, device)
    engine.prefill()
    n = len(variant)
    tokens = torch.from_numpy(rng.integers(0, cfg.vocab, n)).to(device)
    temperature = np.array([0, 1, 0.7, 1.3, 1, 1, 0.9, 1, 1], np.float32)
    top_k = np.array([0, 0, 7, 40, 1, 0, 0, 3, 100], np.int32)
    top_p = np.array([1, 0.9, 1, 0.8, 1, 1, 0.5, 1, 0.95], np.float32)
    min_p = np.array([0, 0, 0, 0.02, 0, 0.1, 0, 0, 0], np.float32)
    knobs = [torch.from_numpy(a).to(device) for a in (temperature, top_k, top_p, min_p)]
    lists = [list(prompts[variant[r]]) for r in engine.perm]
    for step in range(steps):
        for b, t in enumerate(tokens.cpu().tolist()):
            lists[b].append(t)
        logits = engine.decode(tokens)
        u = rng.random(n).astype(np.float32)
        tokens, lp = bd.sample(logits, torch.from_numpy(u).to(device), *knobs, return_logprob=True)
        got = logits.cpu().double().numpy()
        for b in range(n):
            want, wlp = sample_ref.sample_row(got[b], float(u[b]), float(temperature[b]), int(top_k[b]),
                                              float(top_p[b]), float(min_p[b]))
            assert tokens[b].item() == want, (step, b)
            assert abs(lp[b].item() - wlp) <= 1e-5 * max(1.0, abs(wlp)), (step, b)
            if step in (0, 1, cfg.page - 1, cfg.page, steps - 1):
                ref = plain_logits(model, variant[engine.perm[b]], np.array(lists[b]))
                err = np.linalg.norm(got[b] - ref) / np.linalg.norm(ref)
                assert err <= TOL, (step, b, err)
                print(f"step {step} request {b}: {err:.2e}", flush=True)
