"""A small multi-tenant decoder, from prompts to sampled tokens, on the library's operators.

    python examples/decode.py [bf16|fp8|fp4]

Every linear of the model has one base matrix and a 1-bit delta per variant.  Requests of one
variant share that variant's system prompt, so its keys and values are written once (``prefill``)
and every request's own tokens follow in pages of its own.  One step of ``decode`` is:

* the batch, grouped by variant (``plan_segments``), through the grouped fused linears;
* ``cache_write`` puts the new keys and values into the paged cache, in bf16, e4m3 or 4 bits;
* ``attend_shared`` in the layers that see everything (each prompt is read once per variant, not
  once per request), ``attend_window`` in the layers with a sliding window and a few first tokens;
* ``sample`` on the logits.

torch does what is left: embedding, norms, rotary positions.  Weights are random.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tenant_serving_bitdelta_amd as bd  # noqa: E402


@dataclass
class Config:
    hidden: int = 512
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    ffn: int = 1024
    vocab: int = 2048
    layers: int = 4          # even ones see everything, odd ones a window
    window: int = 24
    sinks: int = 4
    variants: int = 3
    page: int = 16
    kv: str = "bf16"         # what the cache holds: bf16, fp8 (e4m3), fp4 (e2m1 and a scale per 32 values)

    def linears(self):
        q, kv = self.heads * self.head_dim, self.kv_heads * self.head_dim
        return {"q": (q, self.hidden), "k": (kv, self.hidden), "v": (kv, self.hidden),
                "o": (self.hidden, q), "gate": (self.ffn, self.hidden),
                "up": (self.ffn, self.hidden), "down": (self.hidden, self.ffn)}


class Model:
    """Random base weights, and each variant's compressed delta of every linear."""

    def __init__(self, cfg: Config, device, seed=0):
        gen = torch.Generator(device="cpu").manual_seed(seed)
        self.cfg = cfg
        self.embed = torch.randn(cfg.vocab, cfg.hidden, generator=gen).bfloat16().to(device)
        self.layers = [{name: self._linear(shape, gen, device) for name, shape in cfg.linears().items()}
                       for _ in range(cfg.layers)]
        self.head = self._linear((cfg.vocab, cfg.hidden), gen, device, scale=3.0)

    def _linear(self, shape, gen, device, scale=1.0):
        d_out, d_in = shape
        w = (torch.randn(shape, generator=gen) * (scale / d_in ** 0.5)).bfloat16().to(device)
        variants = []
        for _ in range(self.cfg.variants):
            delta = (torch.randn(shape, generator=gen) * (0.2 * scale / d_in ** 0.5)).to(device)
            words = torch.empty((d_out, d_in // 32), dtype=torch.int32, device=device)
            tiled = torch.empty(bd.sign_words_t128(d_out, d_in), dtype=torch.int32, device=device)
            alpha = torch.empty(1, dtype=torch.float32, device=device)
            bd.compress(delta, words, alpha, tiled=tiled)
            variants.append((words, alpha, tiled))
        return w, variants


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def rotary(x, pos):
    """x [tokens, heads, dim], pos [tokens]."""
    half = x.shape[-1] // 2
    angle = pos[:, None].float() * 10000.0 ** (-torch.arange(half, device=x.device) / half)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x.float().split(half, dim=-1)
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1).bfloat16()


class Cache:
    """One layer's pages, [pages, page, kv_heads, ..], stored head by head; ``scales``: what the cache's
    calls take beside them.  e4m3 gets 16 times the values, so up to 28: keys are norms of a few, and rotated."""

    def __init__(self, cfg: Config, pages: int, device):
        def make(width, dtype):
            shape = (pages, cfg.kv_heads, cfg.page, width)
            return torch.zeros(shape, dtype=dtype, device=device).transpose(1, 2)

        width, dtype = {"bf16": (cfg.head_dim, torch.bfloat16), "fp8": (cfg.head_dim, torch.float8_e4m3fn),
                        "fp4": (cfg.head_dim // 2, torch.uint8)}[cfg.kv]
        self.k, self.v = make(width, dtype), make(width, dtype)
        self.scales = {}
        if cfg.kv == "fp8":
            self.scales = {"k_scale": 1 / 16, "v_scale": 1 / 16}
        elif cfg.kv == "fp4":
            self.scales = {"k_block_scales": make(cfg.head_dim // 32, torch.uint8),
                           "v_block_scales": make(cfg.head_dim // 32, torch.uint8)}


class Engine:
    """A batch of requests of several variants and the pages that hold their keys and values."""

    def __init__(self, model: Model, token_variant, prompts, max_new: int, device):
        cfg = self.cfg = model.cfg
        self.model, self.device = model, device
        self.perm, self.offs, self.segv = bd.plan_segments(token_variant, cfg.variants)
        batch, nseg = len(self.perm), len(self.segv)
        # whole pages of prompt, so that a request's own pages can follow them in one table
        self.prompts = [prompts[v] for v in self.segv]
        assert all(len(p) % cfg.page == 0 for p in self.prompts)
        pages_of = [len(p) // cfg.page for p in self.prompts]
        own = -(-max_new // cfg.page)
        ids = iter(torch.randperm(sum(pages_of) + batch * own).tolist())
        width = max(pages_of)
        prefix = np.zeros((nseg, width), np.int32)
        for g, n in enumerate(pages_of):
            prefix[g, :n] = [next(ids) for _ in range(n)]
        table = np.array([[next(ids) for _ in range(own)] for _ in range(batch)], np.int32)
        # the same keys as one list per request, for the layers with a window
        joined = np.zeros((batch, width + own), np.int32)
        first = np.zeros(batch, np.int32)
        for g, n in enumerate(pages_of):
            for b in range(self.offs[g], self.offs[g + 1]):
                joined[b, :n], joined[b, n:n + own] = prefix[g, :n], table[b]
                first[b] = n * cfg.page
        put = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
        self.prefix, self.table, self.joined, self.first = put(prefix), put(table), put(joined), put(first)
        self.prefix_lens = put(np.array([len(p) for p in self.prompts], np.int32))
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.cache = [Cache(cfg, sum(pages_of) + batch * own, device) for _ in range(cfg.layers)]

    def linears(self, layer, names, x, offs):
        todo = [layer[n] for n in names]
        ys = [torch.empty(x.shape[0], w.shape[0], dtype=torch.bfloat16, device=x.device) for w, _ in todo]
        return bd.matmul_grouped([(x, w, y, vs) for (w, vs), y in zip(todo, ys)], offs, self.segv)

    def forward(self, tokens, pos, table, lens, q_offsets, offs, attend):
        """Hidden states of ``tokens`` at ``pos``, the last tokens of the sequences that ``table``, ``lens``
        and ``q_offsets`` describe; their keys go there, and attend(layer number, q, cache) sees them."""
        cfg = self.cfg
        x = self.model.embed[tokens.long()]
        for i, layer in enumerate(self.model.layers):
            q, k, v = (y.unflatten(1, (-1, cfg.head_dim))
                       for y in self.linears(layer, ("q", "k", "v"), norm(x), offs))
            c = self.cache[i]
            bd.cache_write(rotary(k, pos), v, c.k, c.v, table, lens, q_offsets, **c.scales)
            a = attend(i, rotary(q, pos), c)
            x = x + self.linears(layer, ("o",), a.flatten(1), offs)[0]
            gate, up = self.linears(layer, ("gate", "up"), norm(x), offs)
            x = x + self.linears(layer, ("down",), torch.nn.functional.silu(gate) * up, offs)[0]
        return norm(x)

    def prefill(self):
        """Every variant's prompt, all in one ragged batch."""
        cfg = self.cfg
        n = [len(p) for p in self.prompts]
        offs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        pos = torch.cat([torch.arange(m) for m in n]).to(self.device)
        q_offsets = torch.from_numpy(offs).to(self.device)
        everything = self.prefix.shape[1] * cfg.page

        def attend(i, q, c):
            return bd.attend_window(q, c.k, c.v, self.prefix, self.prefix_lens,
                                    cfg.window if i % 2 else everything, cfg.sinks,
                                    q_offsets=q_offsets, max_q_len=max(n), **c.scales)

        tokens = torch.from_numpy(np.concatenate(self.prompts)).to(self.device)
        return self.forward(tokens, pos, self.prefix, self.prefix_lens, q_offsets, offs, attend)

    def decode(self, tokens):
        """float32 logits after one more token per request (in the order of ``perm``)."""
        cfg = self.cfg
        pos = self.first + self.lens
        self.lens += 1
        seen = self.first + self.lens

        def attend(i, q, c):
            if i % 2:
                return bd.attend_window(q, c.k, c.v, self.joined, seen, cfg.window, cfg.sinks, **c.scales)
            return bd.attend_shared(q, c.k, c.v, self.table, self.lens, self.prefix, self.prefix_lens,
                                    self.offs, **c.scales)

        x = self.forward(tokens, pos, self.joined, seen, None, self.offs, attend)
        w, variants = self.model.head
        return bd.matmul(x, w, variants, self.offs, self.segv, out_dtype="f32")


def main():
    device = torch.device("cuda:0")
    cfg = Config(kv=sys.argv[1] if len(sys.argv) > 1 else "bf16")
    rng = np.random.default_rng(7)
    model = Model(cfg, device)
    variant = rng.integers(0, cfg.variants, 20)
    prompts = [rng.integers(0, cfg.vocab, cfg.page * n) for n in (12, 3, 7)]
    steps = 24
    engine = Engine(model, variant, prompts, steps, device)
    engine.prefill()
    tokens = torch.from_numpy(rng.integers(0, cfg.vocab, len(variant))).to(device)
    # every request its own settings
    full = lambda lo, hi: torch.from_numpy(rng.uniform(lo, hi, len(variant)).astype(np.float32)).to(device)  # noqa: E731
    temperature, top_p, min_p = full(0.5, 1.2), full(0.7, 1.0), full(0.0, 0.05)
    top_k = torch.from_numpy(rng.integers(0, 60, len(variant)).astype(np.int32)).to(device)
    gen = torch.Generator(device=device).manual_seed(1)
    lines, logprob = [], torch.zeros(len(variant), device=device)
    for _ in range(steps):
        u = torch.rand(len(variant), generator=gen, device=device)
        tokens, lp = bd.sample(engine.decode(tokens), u, temperature, top_k, top_p, min_p,
                               return_logprob=True)
        lines.append(tokens.cpu().numpy())
        logprob += lp
    out = np.stack(lines, 1)
    for row, request in enumerate(engine.perm):
        print(f"request {request:2d} variant {variant[request]} log-probability "
              f"{logprob[row].item():7.2f}: {' '.join(map(str, out[row][:12]))} ...")


if __name__ == "__main__":
    main()
