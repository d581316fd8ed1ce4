"""Serving operators next to the fused linears: what is timed, and their plain forms.

Three operators take a decode or prefill step from the linears' outputs to the next tokens:

* ``shared``: decode attention (one new token per sequence) where the sequences of a segment of
  the batch share a long prefix kept once in the paged cache, each followed by its own tokens;
* ``window``: causal attention over a paged cache with a sliding window and a few first tokens
  that stay visible, for ragged prefill chunks and for single tokens;
* ``sample``: the next token of each row from given uniform numbers, with temperature, top-k,
  top-p and min-p per row.

``run`` computes them in elementary torch operations, or, with ``own`` set, through the package's
entry points.  ``exact`` holds the definitions in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a chat turn of four users of one variant behind a short system prompt: latency counts
        {"name": "shared_4seq_short", "op": "shared", "batch": 4, "segments": 1, "prefix": 100,
         "own": 60, "heads": 8, "kv_heads": 2, "dim": 64, "page": 16, "kv": "bf16"},
        # the 64-token decode batch over 14 variants, each with its own 2k-token system prompt
        {"name": "shared_64seq_14seg", "op": "shared", "batch": 64, "segments": 14, "prefix": 2048,
         "own": 512, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "kv": "bf16"},
        # the 256-token decode batch, 14 variants with long shared documents
        {"name": "shared_256seq_14seg", "op": "shared", "batch": 256, "segments": 14,
         "prefix": 8192, "own": 768, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "kv": "bf16"},
        # odd sizes: 37 sequences in 3 segments, 3 heads a kv head, 8-bit cache, 24-token pages
        {"name": "shared_37seq_fp8", "op": "shared", "batch": 37, "segments": 3, "prefix": 5001,
         "own": 333, "heads": 12, "kv_heads": 4, "dim": 128, "page": 24, "kv": "fp8"},
        # one user far into a long chat: a single token over window and sinks
        {"name": "window_decode_1seq", "op": "window", "batch": 1, "q_len": 1, "length": 6000,
         "window": 1024, "sinks": 4, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "kv": "bf16"},
        # 64 long chats of uneven length, 8-bit cache
        {"name": "window_decode_64seq_fp8", "op": "window", "batch": 64, "q_len": 1,
         "length": 16384, "window": 8192, "sinks": 16, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "kv": "fp8"},
        # the prefill batch of 4 requests of up to 2048 tokens, none before them
        {"name": "window_prefill_4x2048", "op": "window", "batch": 4, "q_len": 2048,
         "length": 2048, "window": 1024, "sinks": 4, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "kv": "bf16"},
        # an 8192-token chunk of one long document, 8192 tokens already in the cache
        {"name": "window_prefill_8192_of_16384", "op": "window", "batch": 1, "q_len": 8192,
         "length": 16384, "window": 4096, "sinks": 4, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "kv": "bf16"},
        # one chat's next token
        {"name": "sample_1x32000", "op": "sample", "rows": 1, "vocab": 32000, "logits": "f32",
         "mode": "chat", "masked": False},
        # the 64-token decode batch, bf16 logits as the last linear writes them
        {"name": "sample_64x128000_bf16", "op": "sample", "rows": 64, "vocab": 128000,
         "logits": "bf16", "mode": "chat", "masked": False},
        # the 256-token batch with every mix of settings, fp32 logits
        {"name": "sample_256x131072", "op": "sample", "rows": 256, "vocab": 131072,
         "logits": "f32", "mode": "mixed", "masked": False},
        # odd sizes, grammar masks that forbid most of the vocabulary
        {"name": "sample_37x100003_masked", "op": "sample", "rows": 37, "vocab": 100003,
         "logits": "f32", "mode": "mixed", "masked": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "window", "window", "sample"])
    if op == "sample":
        return {"op": op, "rows": _log_int(rng, 1, 256), "vocab": _log_int(rng, 1000, 131072),
                "logits": rng.choice(["f32", "bf16"]), "mode": rng.choice(["chat", "mixed"]),
                "masked": rng.random() < 0.3}
    heads, kv_heads = rng.choice([(64, 8), (32, 8), (16, 16), (12, 4), (40, 8), (8, 1)])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128]),
            "page": rng.choice([16, 24, 64, 128]), "kv": rng.choice(["bf16", "bf16", "fp8"])}
    if op == "shared":
        batch = _log_int(rng, 1, 256)
        case.update(batch=batch, segments=rng.randint(1, min(14, batch)),
                    prefix=_log_int(rng, 1, 8192), own=_log_int(rng, 1, 768))
    elif rng.random() < 0.5:
        case.update(batch=_log_int(rng, 1, 64), q_len=1, length=_log_int(rng, 1, 16384),
                    window=_log_int(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16]))
    else:
        q_len = _log_int(rng, 2, 4096)
        case.update(batch=rng.randint(1, max(1, min(8, 8192 // q_len))), q_len=q_len,
                    length=q_len + rng.choice([0, 0, _log_int(rng, 1, 4096)]),
                    window=_log_int(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 16]))
    return case


def _spread(n, hi):
    """n lengths between hi/8 and hi (the first is hi), the same for every seed: a batch's uneven
    lengths, at golden-ratio steps."""
    return [max(1, int(hi * (1.0 - 0.875 * ((i * 0.6180339887498949) % 1.0)))) for i in range(n)]


def _segment_sizes(batch, segments):
    """Sequences per segment, Zipf(1.1) as the decode batches draw their variants, each >= 1."""
    w = [(i + 1) ** -1.1 for i in range(segments)]
    left = batch - segments
    sizes = [1 + int(left * x / sum(w)) for x in w]
    sizes[0] += batch - sum(sizes)
    return sizes


def _shared_lengths(case):
    return (_segment_sizes(case["batch"], case["segments"]),
            _spread(case["segments"], case["prefix"]), _spread(case["batch"], case["own"]))


def _window_lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    if case["q_len"] == 1:
        return [1] * case["batch"], _spread(case["batch"], case["length"])
    q = _spread(case["batch"], case["q_len"])
    return q, [case["length"] - case["q_len"] + n for n in q]


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        size = 2 if case["logits"] == "bf16" else 4
        # a comparison and an exponential's worth of arithmetic per logit
        return {"bytes": n * size + case["rows"] * 28, "flops": 2 * n}
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    size = 1 if case["kv"] == "fp8" else 2
    if case["op"] == "shared":
        sizes, plen, olen = _shared_lengths(case)
        pairs = sum(n * p for n, p in zip(sizes, plen)) + sum(olen)
        keys, tokens = sum(plen) + sum(olen), case["batch"]
    else:
        pairs = keys = 0
        w, s = case["window"], case["sinks"]
        q, lens = _window_lengths(case)
        for n, length in zip(q, lens):
            pos = np.arange(length - n, length, dtype=np.int64)
            lo = np.maximum(pos - w + 1, 0)
            pairs += int(np.sum(pos + 1 - lo + np.minimum(lo, s)))
            first = int(lo[0])
            keys += length - first + min(first, s)
        tokens = sum(q)
    return {"bytes": keys * hk * d * 2 * size + 2 * tokens * h * d * 2 + 4 * tokens * h,
            "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _cache(case, pages, g):
    """Paged keys and values, [pages, page, kv heads, dim] views of head-major pages; the 8-bit
    form stores value / scale."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    out = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device=_DEV)
        x.normal_(generator=g)
        if case["kv"] == "fp8":
            x = (x * 64.0).to(torch.float8_e4m3fn)
        out.append(x.permute(0, 2, 1, 3))
    return out[0], out[1], (1.0 / 64.0 if case["kv"] == "fp8" else 1.0)


def _tables(lengths, page, perm, at):
    """int32 page table of sequences of these lengths, pages taken from perm[at:]; entries past a
    sequence's end are -1."""
    width = max(1, max(-(-n // page) for n in lengths))
    t = np.full((len(lengths), width), -1, dtype=np.int32)
    for i, n in enumerate(lengths):
        k = -(-n // page)
        t[i, :k] = perm[at:at + k]
        at += k
    return torch.from_numpy(t).to(_DEV), at


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=_DEV)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, seed, g)
    page = case["page"]
    rng = np.random.default_rng(seed)
    st = {"case": case}
    if case["op"] == "shared":
        sizes, plen, olen = _shared_lengths(case)
        pages = sum(-(-n // page) for n in plen + olen)
        perm = rng.permutation(pages).astype(np.int32)
        st["prefix_table"], at = _tables(plen, page, perm, 0)
        st["table"], _ = _tables(olen, page, perm, at)
        st["prefix_lens"], st["lens"] = _ints(plen), _ints(olen)
        st["seg_offsets"] = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        tokens = case["batch"]
    else:
        q, lens = _window_lengths(case)
        pages = sum(-(-n // page) for n in lens)
        st["table"], _ = _tables(lens, page, rng.permutation(pages).astype(np.int32), 0)
        st["lens"] = _ints(lens)
        st["q_offsets"] = _ints([0] + np.cumsum(q).tolist())
        st["q_lens"], st["host_lens"] = q, lens
        tokens = sum(q)
    st["k"], st["v"], st["kv_scale"] = _cache(case, pages, g)
    x = torch.empty((tokens, case["heads"], case["dim"]), dtype=torch.float32, device=_DEV)
    x.normal_(generator=g)
    st["q"] = (1.5 * x).to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(case["dim"])
    return st


def _prepare_sample(case, seed, g):
    rows, vocab = case["rows"], case["vocab"]
    x = torch.empty((rows, vocab), dtype=torch.float32, device=_DEV)
    x.normal_(mean=0.0, std=2.0, generator=g)
    # a few likely tokens well above the rest, as a language model's logits have
    hot = torch.randint(0, vocab, (rows, 24), device=_DEV, generator=g)
    lift = torch.empty((rows, 24), dtype=torch.float32, device=_DEV)
    lift.normal_(mean=13.0, std=2.5, generator=g)
    x.scatter_(1, hot, lift)
    if case["masked"]:
        allowed = torch.empty((rows, vocab), device=_DEV).uniform_(generator=g) < 0.02
        allowed[:, 0] = True
        x.masked_fill_(~allowed, float("-inf"))
    rng = np.random.default_rng(seed)
    if case["mode"] == "chat":
        temp = np.full(rows, 0.7)
        k = np.full(rows, 50)
        p = np.full(rows, 0.9)
        m = np.zeros(rows)
    else:
        temp = rng.choice([0.0, 0.3, 0.7, 1.0, 1.3], size=rows)
        k = rng.choice([0, 0, 1, 20, 50, 200, 1000], size=rows)
        p = rng.choice([1.0, 1.0, 0.5, 0.9, 0.95, 0.99], size=rows)
        m = rng.choice([0.0, 0.0, 0.02, 0.1], size=rows)

    def f32(a):
        return torch.from_numpy(a.astype(np.float32)).to(_DEV)

    return {"case": case, "logits": x.to(_TYPES[case["logits"]]),
            "u": f32(rng.integers(0, 1 << 24, size=rows) / float(1 << 24)),
            "temperature": f32(temp), "top_k": _ints(k.tolist()), "top_p": f32(p), "min_p": f32(m)}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_shared(st):
    import tenant_serving_bitdelta_amd as bd
    return bd.attend_shared(st["q"], st["k"], st["v"], st["table"], st["lens"],
                            st["prefix_table"], st["prefix_lens"], st["seg_offsets"],
                            scale=st["scale"], k_scale=st["kv_scale"], v_scale=st["kv_scale"],
                            return_lse=True)


def _own_window(st):
    import tenant_serving_bitdelta_amd as bd
    c = st["case"]
    one = c["q_len"] == 1
    return bd.attend_window(st["q"], st["k"], st["v"], st["table"], st["lens"],
                            c["window"], c["sinks"],
                            q_offsets=None if one else st["q_offsets"],
                            max_q_len=c["q_len"], scale=st["scale"], k_scale=st["kv_scale"],
                            v_scale=st["kv_scale"], return_lse=True)


def _own_sample(st):
    import tenant_serving_bitdelta_amd as bd
    return bd.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                     top_p=st["top_p"], min_p=st["min_p"], return_logprob=True)


def _gather(pages, table, count, scale):
    """fp32 [sequences, heads, count, dim] rows of a paged cache; absent pages read page 0."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = raw[table.clamp(min=0).long()].flatten(1, 2)[:, :count].contiguous().view(pages.dtype)
    return (x.float() * scale).transpose(1, 2).contiguous()


def _softmax_mix(scores, mixes):
    """Softmax over the last axes of several score blocks together, and its products."""
    top = torch.stack([s.amax(-1) for s in scores]).amax(0)
    base = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weights = [torch.exp(s - base[..., None]) for s in scores]
    total = sum(w.sum(-1) for w in weights)
    out = sum(torch.matmul(w, v) for w, v in zip(weights, mixes))
    safe = torch.where(total > 0, total, torch.ones_like(total))
    return out / safe[..., None], torch.log(total) + base


def _plain_shared(st):
    c, q = st["case"], st["q"].float() * st["scale"]
    h, hk, d, s = c["heads"], c["kv_heads"], c["dim"], st["kv_scale"]
    width, pwidth = st["table"].shape[1] * c["page"], st["prefix_table"].shape[1] * c["page"]
    gone = torch.arange(width, device=_DEV)[None] >= st["lens"][:, None]
    pgone = torch.arange(pwidth, device=_DEV)[None] >= st["prefix_lens"][:, None]
    outs, lses = [], []
    for g in range(c["segments"]):
        a, b = int(st["seg_offsets"][g]), int(st["seg_offsets"][g + 1])
        n = b - a
        qg = q[a:b].view(n, hk, h // hk, d)
        k = _gather(st["k"], st["table"][a:b], width, s)
        v = _gather(st["v"], st["table"][a:b], width, s)
        pk = _gather(st["k"], st["prefix_table"][g:g + 1], pwidth, s)[0]
        pv = _gather(st["v"], st["prefix_table"][g:g + 1], pwidth, s)[0]
        so = torch.matmul(qg, k.transpose(2, 3))
        so = so.masked_fill(gone[a:b, None, None], float("-inf"))
        rows = qg.transpose(0, 1).reshape(hk, n * (h // hk), d)
        sp = torch.matmul(rows, pk.transpose(1, 2)).masked_fill(pgone[g], float("-inf"))
        top = torch.maximum(so.amax(-1), sp.amax(-1).view(hk, n, h // hk).transpose(0, 1))
        base = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        wo = torch.exp(so - base[..., None])
        wp = torch.exp(sp - base.transpose(0, 1).reshape(hk, -1, 1))
        total = wo.sum(-1) + wp.sum(-1).view(hk, n, h // hk).transpose(0, 1)
        out = torch.matmul(wo, v) + torch.matmul(wp, pv).view(hk, n, h // hk, d).transpose(0, 1)
        safe = torch.where(total > 0, total, torch.ones_like(total))
        outs.append((out / safe[..., None]).reshape(n, h, d))
        lses.append((torch.log(total) + base).reshape(n, h))
    return torch.cat(outs).to(torch.bfloat16), torch.cat(lses)


def _plain_window(st):
    c, q = st["case"], st["q"].float() * st["scale"]
    h, hk, d, s = c["heads"], c["kv_heads"], c["dim"], st["kv_scale"]
    w, sinks = c["window"], c["sinks"]
    outs, lses, at = [], [], 0
    for i, (n, length) in enumerate(zip(st["q_lens"], st["host_lens"])):
        k = _gather(st["k"], st["table"][i:i + 1], length, s)[0]
        v = _gather(st["v"], st["table"][i:i + 1], length, s)[0]
        for j in range(0, n, 1024):
            m = min(1024, n - j)
            p0 = length - n + j
            lo = max(0, p0 - w + 1)
            cols = torch.cat([torch.arange(0, min(sinks, lo), device=_DEV),
                              torch.arange(lo, p0 + m, device=_DEV)])
            pos = torch.arange(p0, p0 + m, device=_DEV)[:, None]
            seen = (cols <= pos) & ((cols > pos - w) | (cols < sinks))
            qj = q[at + j:at + j + m].view(m, hk, h // hk, d).permute(1, 2, 0, 3).contiguous()
            kj = k[:, cols].transpose(1, 2).contiguous()[:, None]
            sc = torch.matmul(qj, kj).masked_fill(~seen, float("-inf"))
            out, lse = _softmax_mix([sc], [v[:, cols][:, None]])
            outs.append(out.permute(2, 0, 1, 3).reshape(m, h, d).to(torch.bfloat16))
            lses.append(lse.permute(2, 0, 1).reshape(m, h))
        at += n
    return torch.cat(outs), torch.cat(lses)


def _plain_sample(st):
    x = st["logits"].double()
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    rows, vocab = x.shape
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    temp = st["temperature"].double()
    greedy = ~(temp > 0)
    diff = val - val[:, :1]
    diff = torch.where(val == val[:, :1], torch.zeros_like(diff), diff)
    wt = torch.exp(diff / torch.where(greedy, torch.ones_like(temp), temp)[:, None])
    cum = torch.cumsum(wt, 1)
    k = st["top_k"].long()
    k = torch.where((k <= 0) | (k > vocab), torch.full_like(k, vocab), k)
    zk = cum.gather(1, k[:, None] - 1)
    p = st["top_p"].double()[:, None]
    np_ = torch.where(p[:, 0] < 1, (cum < p * zk).sum(1) + 1, torch.full_like(k, vocab))
    nm = (wt >= st["min_p"].double()[:, None]).sum(1)
    n = torch.minimum(torch.minimum(k, np_), nm).clamp(1, vocab)
    n = torch.where(greedy, torch.ones_like(n), n)
    zn = cum.gather(1, n[:, None] - 1)
    j = (cum <= st["u"].double()[:, None] * zn).sum(1)
    j = torch.minimum(j, n - 1)[:, None]
    dead = torch.isinf(val[:, 0]) & (val[:, 0] < 0)
    token = torch.where(dead, torch.full_like(n, -1), idx.gather(1, j)[:, 0])
    logp = torch.where(dead, torch.full_like(temp, float("-inf")),
                       torch.log(wt.gather(1, j)[:, 0] / zn[:, 0]))
    return token.to(torch.int32), logp.to(torch.float32)


_OWN = {"shared": _own_shared, "window": _own_window, "sample": _own_sample}
_PLAIN = {"shared": _plain_shared, "window": _plain_window, "sample": _plain_sample}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(st)
    return _exact_attention(case, st)


def _rows64(pages, ids, page, count, scale):
    """fp64 [count, heads, dim]: token t of a sequence is row t % page of page ids[t // page]."""
    t = torch.arange(count, device=_DEV)
    flat = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    rows = flat[ids[t // page].long(), t % page].contiguous().view(pages.dtype)
    return rows.to(torch.float32).double() * scale


def _exact_block(q, k, v, seen, scale):
    """One sequence's block: q [m, H, D], k and v [n, Hk, D], seen [m, n]."""
    m, h, d = q.shape
    hk = k.shape[1]
    out = torch.zeros((m, h, d), dtype=torch.float64, device=_DEV)
    lse = torch.full((m, h), float("-inf"), dtype=torch.float64, device=_DEV)
    if k.shape[0] == 0:
        return out, lse
    alive = seen.any(1)
    for g in range(hk):
        for j in range(g * (h // hk), (g + 1) * (h // hk)):
            sc = (q[:, j].double() @ k[:, g].T.contiguous()) * scale
            sc = torch.where(seen, sc, torch.full_like(sc, float("-inf")))
            z = torch.logsumexp(sc, 1)
            wt = torch.exp(sc - torch.where(alive, z, torch.zeros_like(z))[:, None])
            out[:, j] = wt @ v[:, g].contiguous()
            lse[:, j] = z
    return out, lse


def _exact_attention(case, st):
    page, s = case["page"], st["kv_scale"]
    outs, lses = [], []
    if case["op"] == "shared":
        sizes, plen, olen = _shared_lengths(case)
        b = 0
        for g, n in enumerate(sizes):
            pk = _rows64(st["k"], st["prefix_table"][g], page, plen[g], s)
            pv = _rows64(st["v"], st["prefix_table"][g], page, plen[g], s)
            for _ in range(n):
                k = torch.cat([pk, _rows64(st["k"], st["table"][b], page, olen[b], s)])
                v = torch.cat([pv, _rows64(st["v"], st["table"][b], page, olen[b], s)])
                hk, d = k.shape[1], k.shape[2]
                q = st["q"][b].double().view(hk, -1, d)
                sc = torch.bmm(q, k.permute(1, 2, 0).contiguous()) * st["scale"]
                z = torch.logsumexp(sc, 2)
                o = torch.bmm(torch.exp(sc - z[..., None]), v.transpose(0, 1).contiguous())
                outs.append(o.reshape(1, -1, d))
                lses.append(z.reshape(1, -1))
                b += 1
        return torch.cat(outs), torch.cat(lses)
    q_lens, lens = _window_lengths(case)
    at = 0
    for i, (n, length) in enumerate(zip(q_lens, lens)):
        k = _rows64(st["k"], st["table"][i], page, length, s)
        v = _rows64(st["v"], st["table"][i], page, length, s)
        for j in range(0, n, 2048):
            m = min(2048, n - j)
            hi = length - n + j + m
            lo = max(0, length - n + j + 1 - case["window"])
            col = torch.arange(hi, device=_DEV)
            col = col[(col >= lo) | (col < case["sinks"])]
            pos = torch.arange(hi - m, hi, device=_DEV)[:, None]
            seen = (col[None] <= pos) & ((pos - col[None] < case["window"])
                                         | (col[None] < case["sinks"]))
            o, z = _exact_block(st["q"][at + j:at + j + m], k[col], v[col], seen, st["scale"])
            outs.append(o)
            lses.append(z)
        at += n
    return torch.cat(outs), torch.cat(lses)


def _exact_sample(st):
    """Row by row on the host: sort by descending logit, ties by index, and walk the filters."""
    logits = st["logits"].float().cpu().numpy().astype(np.float64)
    u, temp, top_p, min_p = (st[n].cpu().numpy().astype(np.float64)
                             for n in ("u", "temperature", "top_p", "min_p"))
    top_k = st["top_k"].cpu().numpy()
    rows, vocab = logits.shape
    token = np.full(rows, -1, dtype=np.int32)
    logp = np.full(rows, -np.inf)
    for r in range(rows):
        x = logits[r]
        order = np.argsort(-x, kind="stable")
        best = x[order[0]]
        if best == -np.inf:
            continue
        if not temp[r] > 0:
            token[r], logp[r] = order[0], 0.0
            continue
        w = np.exp((x[order] - best) / temp[r])
        n = vocab if top_k[r] <= 0 else min(vocab, int(top_k[r]))
        limit = n
        if top_p[r] < 1:
            run_ = np.cumsum(w[:n])
            limit = min(n, int(np.searchsorted(run_, top_p[r] * run_[-1])) + 1)
        if min_p[r] > 0:
            limit = min(limit, max(1, int(np.count_nonzero(w >= min_p[r]))))
        run_ = np.cumsum(w[:limit])
        j = min(int(np.searchsorted(run_, u[r] * run_[-1], side="right")), limit - 1)
        token[r], logp[r] = order[j], np.log(w[j] / run_[-1])
    return torch.from_numpy(token).to(_DEV), torch.from_numpy(logp).to(_DEV)
