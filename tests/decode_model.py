"""The model of examples/decode.py on the host, for the tests: its weights compressed by the oracle, and
its logits from a whole list of tokens with every intermediate result rounded to bf16 where the engine
rounds it.

A row of logits is off (relative L2) by the 13 roundings of a layer (norm, q, k, v, attention weights and
output, o, sum, norm, gate, up, their product, down, sum) through 4 layers and the last norm: 53 of at most
half a step, 2^-8.  They are independent, so that their squares add: BOUND counts each at its largest (the
mean over a step is 0.41 of it), and mistakes in a mask have to exceed it."""
import numpy as np
import torch

import test_gpu_decode_example as T
from oracle import bitdelta_oracle as O

D = T.D
BOUND = 53 ** 0.5 * 2.0 ** -8


class HostModel(D.Model):
    def _linear(self, shape, gen, device, scale=1.0):
        d_out, d_in = shape
        w = (torch.randn(shape, generator=gen) * (scale / d_in ** 0.5)).bfloat16()
        variants = []
        for _ in range(self.cfg.variants):
            words, alpha = O.compress_ref((torch.randn(shape, generator=gen) * (0.2 * scale / d_in ** 0.5)).numpy())
            variants.append((torch.from_numpy(words.view(np.int32).reshape(d_out, d_in // 32)),
                             torch.tensor([float(alpha)]), None))
        return w, variants


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).bfloat16().double().numpy()


def rounded_logits(model, v, tokens):
    cfg = model.cfg
    x = model.embed.double().cpu().numpy()[tokens]
    n = len(tokens)
    back = np.arange(n)[:, None] - np.arange(n)[None, :]
    for i, layer in enumerate(model.layers):
        w = {name: T.weights(lin, v) for name, lin in layer.items()}
        y = bf16(T.norm(x))
        q, k, val = (bf16(y @ w[c].T).reshape(n, -1, cfg.head_dim) for c in "qkv")
        q, k = bf16(T.rotary(q)), bf16(T.rotary(k))
        seen = back >= 0
        if i % 2:
            seen &= (back < cfg.window) | (np.arange(n)[None, :] < cfg.sinks)
        out = np.empty_like(q)
        for h in range(cfg.heads):
            g = h // (cfg.heads // cfg.kv_heads)
            s = np.where(seen, q[:, h] @ k[:, g].T / np.sqrt(cfg.head_dim), -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            out[:, h] = bf16(bf16(p) @ val[:, g] / p.sum(1, keepdims=True))
        x = bf16(x + bf16(out.reshape(n, -1) @ w["o"].T))
        y = bf16(T.norm(x))
        gate, up = bf16(y @ w["gate"].T), bf16(y @ w["up"].T)
        x = bf16(x + bf16(bf16(bf16(gate / (1 + np.exp(-gate))) * up) @ w["down"].T))
    return bf16(T.norm(x[-1])) @ T.weights(model.head, v).T


def error(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)
