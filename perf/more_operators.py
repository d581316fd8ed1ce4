"""The paged cache in 4 and 8 bits: what is timed, and the plain forms.

Four operators around the cache that decode and prefill steps read:

* ``write``: new keys and values into their pages, quantised on the way (bf16, e4m3 or 4 bits);
* ``read``: the tokens of sequences back from their pages, as bf16 rows;
* ``shared``: decode attention over a 4-bit cache whose prefixes are shared by segment;
* ``window``: causal attention over a 4-bit cache with a sliding window and first tokens that stay
  visible, for ragged chunks and for single tokens.

4 bits: a block of 32 consecutive values y of a row (divided by the cache's scale) holds codes of
{0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign, and a byte e + 127: 2^e is the smallest power of two with
max |y| <= 7 * 2^e, and a code is y / 2^e rounded to nearest, ties to the even code.

``run`` computes them in elementary torch operations, or, with ``own`` set, through the package's
entry points.  ``exact`` holds the definitions in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda"
_BYTES = {"bf16": 2.0, "fp8": 1.0, "fp4": 17.0 / 32.0}  # of a stored value


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # the newest token of four chats: latency counts (written, then read back)
        {"name": "write_4seq_fp4", "op": "write", "batch": 4, "q_len": 1, "length": 160,
         "kv_heads": 2, "dim": 64, "page": 16, "kv": "fp4", "scale": 1.0},
        # the prefill batch of 4 requests of up to 2048 tokens (written, then read back)
        {"name": "write_4x2048_fp4", "op": "write", "batch": 4, "q_len": 2048, "length": 2048,
         "kv_heads": 8, "dim": 128, "page": 64, "kv": "fp4", "scale": 1.0},
        # odd sizes: chunks of 37 requests into 24-token pages of an 8-bit cache
        {"name": "write_37chunks_fp8", "op": "write", "batch": 37, "q_len": 333, "length": 1001,
         "kv_heads": 4, "dim": 128, "page": 24, "kv": "fp8", "scale": 0.0571},
        # 14 variants' system prompts, taken out of the 4-bit cache as a whole
        {"name": "read_14x8192_fp4", "op": "read", "batch": 14, "q_len": 8192, "length": 8192,
         "kv_heads": 8, "dim": 128, "page": 64, "kv": "fp4", "scale": 1.0},
        # the last 100 tokens of three chats, 8-bit cache
        {"name": "read_3x100_fp8", "op": "read", "batch": 3, "q_len": 100, "length": 777,
         "kv_heads": 2, "dim": 64, "page": 16, "kv": "fp8", "scale": 0.0625},
        # a chat turn of four users of one variant behind a short system prompt: latency counts
        {"name": "shared_4seq_short", "op": "shared", "batch": 4, "segments": 1, "prefix": 100,
         "own": 60, "heads": 8, "kv_heads": 2, "dim": 64, "page": 16},
        # the 64-token decode batch over 14 variants, each with its own 2k-token system prompt
        {"name": "shared_64seq_14seg", "op": "shared", "batch": 64, "segments": 14, "prefix": 2048,
         "own": 512, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16},
        # the 256-token decode batch, 14 variants with long shared documents
        {"name": "shared_256seq_14seg", "op": "shared", "batch": 256, "segments": 14,
         "prefix": 8192, "own": 768, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64},
        # one user far into a very long document: a single token that sees all of it
        {"name": "window_decode_1x131072", "op": "window", "batch": 1, "q_len": 1,
         "length": 131072, "window": 131072, "sinks": 0, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64},
        # 64 long chats of uneven length
        {"name": "window_decode_64seq", "op": "window", "batch": 64, "q_len": 1, "length": 16384,
         "window": 8192, "sinks": 16, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64},
        # odd sizes: up to 5 drafted tokens of 37 requests, 3 heads a kv head, 24-token pages
        {"name": "window_37x5_draft", "op": "window", "batch": 37, "q_len": 5, "length": 5001,
         "window": 3001, "sinks": 4, "heads": 12, "kv_heads": 4, "dim": 128, "page": 24},
        # the prefill batch of 4 requests of up to 2048 tokens behind 4096 cached ones
        {"name": "window_prefill_4x2048", "op": "window", "batch": 4, "q_len": 2048,
         "length": 6144, "window": 4096, "sinks": 4, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "shared", "window", "window"])
    heads, kv_heads = rng.choice([(64, 8), (32, 8), (16, 16), (12, 4), (40, 8), (8, 1)])
    case = {"op": op, "kv_heads": kv_heads, "dim": rng.choice([64, 128]),
            "page": rng.choice([16, 24, 64, 128])}
    if op in ("write", "read"):
        q_len = rng.choice([1, _log_int(rng, 2, 8192)])
        case.update(batch=_log_int(rng, 1, max(1, min(256, 65536 // q_len))), q_len=q_len,
                    length=q_len + rng.choice([0, _log_int(rng, 1, 2048)]),
                    kv=rng.choice(["fp4", "fp4", "fp8", "bf16"]))
        case["scale"] = {"fp4": rng.choice([1.0, 0.5]), "fp8": rng.choice([0.0625, 0.0571]),
                         "bf16": 1.0}[case["kv"]]
    elif op == "shared":
        batch = _log_int(rng, 1, 256)
        case.update(heads=heads, batch=batch, segments=rng.randint(1, min(14, batch)),
                    prefix=_log_int(rng, 1, 8192), own=_log_int(rng, 1, 768))
    elif rng.random() < 0.5:
        case.update(heads=heads, batch=_log_int(rng, 1, 64), q_len=1,
                    length=_log_int(rng, 1, 16384), window=_log_int(rng, 16, 8192),
                    sinks=rng.choice([0, 1, 4, 16]))
    else:
        q_len = _log_int(rng, 2, 4096)
        case.update(heads=heads, batch=rng.randint(1, max(1, min(8, 8192 // q_len))), q_len=q_len,
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


def _chunk_lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    if case["q_len"] == 1:
        return [1] * case["batch"], _spread(case["batch"], case["length"])
    q = _spread(case["batch"], case["q_len"])
    return q, [case["length"] - case["q_len"] + n for n in q]


def work(case):
    hk, d = case["kv_heads"], case["dim"]
    if case["op"] in ("write", "read"):
        n = 2 * sum(_chunk_lengths(case)[0]) * hk * d
        rows, stored = 2.0 * n, _BYTES[case["kv"]] * n
        # what is written in 4 bits is also handed back as the values it stands for
        back = rows if case["op"] == "write" and case["kv"] == "fp4" else 0.0
        return {"bytes": rows + stored + back, "flops": 2.0 * n}
    h = case["heads"]
    if case["op"] == "shared":
        sizes, plen, olen = _shared_lengths(case)
        pairs = sum(n * p for n, p in zip(sizes, plen)) + sum(olen)
        keys, tokens = sum(plen) + sum(olen), case["batch"]
    else:
        pairs = keys = 0
        w, s = case["window"], case["sinks"]
        q, lens = _chunk_lengths(case)
        for n, length in zip(q, lens):
            pos = np.arange(length - n, length, dtype=np.int64)
            lo = np.maximum(pos - w + 1, 0)
            pairs += int(np.sum(pos + 1 - lo + np.minimum(lo, s)))
            first = int(lo[0])
            keys += length - first + min(first, s)
        tokens = sum(q)
    return {"bytes": keys * hk * d * 2 * _BYTES["fp4"] + 2 * tokens * h * d * 2 + 4 * tokens * h,
            "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _values(shape, g, lift):
    """bf16 keys or values: normal, with ``lift`` some channels well above the rest, as keys have."""
    x = torch.empty(shape, dtype=torch.float32, device=_DEV)
    x.normal_(generator=g)
    if lift:
        x[..., 5::32] *= 6.0
    return x.to(torch.bfloat16)


def _encode(y):
    """(codes [..., n / 2], scale bytes [..., n / 32]) of fp32 values [..., n]."""
    b = y.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    part, power = torch.frexp(amax)  # amax = part * 2^power, part in [0.5, 1)
    byte = (power + torch.where(part > 0.875, 1, 0) + 124).clamp(2, 252)
    # a finite quotient of two fp32 powers of two, both in range
    a = b.abs() / torch.ldexp(torch.ones_like(amax), byte - 127)[..., None]
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + torch.where(torch.signbit(b), 8, 0)).flatten(-2).unflatten(-1, (-1, 2))
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), byte.to(torch.uint8)


def _decode(codes, bytes_):
    """fp32 values of codes and scale bytes."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=_DEV)
    grid = torch.cat([grid, -grid])
    c = codes.long()
    x = torch.stack([grid[c % 16], grid[c // 16]], -1).flatten(-2).unflatten(-1, (-1, 32))
    scale = torch.ldexp(torch.ones_like(bytes_, dtype=torch.float32), bytes_.int() - 127)
    return (x * scale[..., None]).flatten(-2)


def _empty_cache(case, kv, pages):
    """Cleared pages of keys and values, [pages, page, kv heads, ...] views of head-major pages: in
    4 bits, each with its scale bytes."""
    out = {}
    for name in "kv":
        for what, width, dtype in {
                "bf16": [("", case["dim"], torch.bfloat16)],
                "fp8": [("", case["dim"], torch.float8_e4m3fn)],
                "fp4": [("", case["dim"] // 2, torch.uint8),
                        ("_bytes", case["dim"] // 32, torch.uint8)]}[kv]:
            raw = torch.zeros((pages, case["kv_heads"], case["page"], width), device=_DEV,
                              dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype)
            out[name + what] = raw.view(dtype).permute(0, 2, 1, 3)
    return out


def _filled_cache(case, kv, pages, g):
    """The same with earlier tokens in all places."""
    cache = _empty_cache(case, kv, pages)
    step = max(1, (1 << 24) // (case["kv_heads"] * case["page"] * case["dim"]))
    for name in "kv":
        for i in range(0, pages, step):
            n = min(step, pages - i)
            x = _values((n, case["kv_heads"], case["page"], case["dim"]), g, name == "k")
            x = x.float().permute(0, 2, 1, 3)
            if kv == "fp4":
                codes, bytes_ = _encode(x)
                cache[name][i:i + n] = codes
                cache[name + "_bytes"][i:i + n] = bytes_
            elif kv == "fp8":
                y = (x / case["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
                cache[name].view(torch.uint8)[i:i + n] = y.view(torch.uint8)
            else:
                cache[name][i:i + n] = x.to(torch.bfloat16)
    return cache


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
    rng = np.random.default_rng(seed)
    page = case["page"]
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
        q, lens = _chunk_lengths(case)
        pages = sum(-(-n // page) for n in lens)
        st["table"], _ = _tables(lens, page, rng.permutation(pages).astype(np.int32), 0)
        st["lens"] = _ints(lens)
        st["q_offsets"] = _ints([0] + np.cumsum(q).tolist())
        st["q_lens"], st["host_lens"] = q, lens
        tokens = sum(q)
    kv = case.get("kv", "fp4")
    if case["op"] == "write":
        st.update(_empty_cache(case, kv, pages))
        for name in "kv":
            st["new_" + name] = _values((tokens, case["kv_heads"], case["dim"]), g, name == "k")
    else:
        st.update(_filled_cache(case, kv, pages, g))
    if "scale" in case:
        st["divisor"] = torch.tensor(case["scale"], device=_DEV)
    if "heads" in case:
        x = torch.empty((tokens, case["heads"], case["dim"]), dtype=torch.float32, device=_DEV)
        x.normal_(generator=g)
        st["q"] = (1.5 * x).to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(case["dim"])
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_blocks(st):
    if "k_bytes" not in st:
        return {}
    return {"k_block_scales": st["k_bytes"], "v_block_scales": st["v_bytes"]}


def _own_places(st):
    c = st["case"]
    return {"q_offsets": None if c["q_len"] == 1 else st["q_offsets"], "k_scale": c["scale"],
            "v_scale": c["scale"], **_own_blocks(st)}


def _own_write(st):
    import tenant_serving_bitdelta_amd as bd
    at = _own_places(st)
    bd.cache_write(st["new_k"], st["new_v"], st["k"], st["v"], st["table"], st["lens"], **at)
    if st["case"]["kv"] != "fp4":
        return st["k"], st["v"]
    return bd.cache_read(st["k"], st["v"], st["table"], st["lens"], tokens=st["new_k"].shape[0],
                         **at)


def _own_read(st):
    import tenant_serving_bitdelta_amd as bd
    return bd.cache_read(st["k"], st["v"], st["table"], st["lens"], tokens=sum(st["q_lens"]),
                         **_own_places(st))


def _own_shared(st):
    import tenant_serving_bitdelta_amd as bd
    return bd.attend_shared(st["q"], st["k"], st["v"], st["table"], st["lens"],
                            st["prefix_table"], st["prefix_lens"], st["seg_offsets"],
                            scale=st["scale"], return_lse=True, **_own_blocks(st))


def _own_window(st):
    import tenant_serving_bitdelta_amd as bd
    c = st["case"]
    one = c["q_len"] == 1
    return bd.attend_window(st["q"], st["k"], st["v"], st["table"], st["lens"],
                            c["window"], c["sinks"], q_offsets=None if one else st["q_offsets"],
                            max_q_len=c["q_len"], scale=st["scale"], return_lse=True,
                            **_own_blocks(st))


def _plain_places(st):
    """(page, slot) of each row: the last tokens of each sequence."""
    n, lens = torch.diff(st["q_offsets"]).long(), st["lens"].long()
    seq = torch.repeat_interleave(torch.arange(len(n), device=_DEV), n,
                                  output_size=sum(st["q_lens"]))
    row = torch.arange(len(seq), device=_DEV)
    pos = row - st["q_offsets"][1:].long()[seq] + lens[seq]
    page = st["case"]["page"]
    return st["table"][seq, pos // page].long(), pos % page


def _plain_rows(st, page, slot):
    """bf16 rows of the cache."""
    out = []
    for name in "kv":
        if name + "_bytes" in st:
            x = _decode(st[name][page, slot], st[name + "_bytes"][page, slot])
        elif st[name].dtype == torch.float8_e4m3fn:
            x = st[name].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
        else:
            x = st[name][page, slot].float()
        out.append((x * st["divisor"]).to(torch.bfloat16))
    return out


def _plain_write(st):
    page, slot = _plain_places(st)
    for name in "kv":
        y = st["new_" + name].float() / st["divisor"]
        if name + "_bytes" in st:
            st[name][page, slot], st[name + "_bytes"][page, slot] = _encode(y)
        elif st[name].dtype == torch.float8_e4m3fn:
            y = y.clamp(-448, 448).to(torch.float8_e4m3fn)
            st[name].view(torch.uint8)[page, slot] = y.view(torch.uint8)
        else:
            st[name][page, slot] = y.to(torch.bfloat16)
    return _plain_rows(st, page, slot) if "k_bytes" in st else [st["k"], st["v"]]


def _plain_read(st):
    return _plain_rows(st, *_plain_places(st))


def _gather(st, name, table, count):
    """fp32 [sequences, heads, count, dim] rows of the cache; absent pages read page 0."""
    at = table.clamp(min=0).long()
    x = _decode(st[name][at].flatten(1, 2)[:, :count],
                st[name + "_bytes"][at].flatten(1, 2)[:, :count])
    return x.transpose(1, 2).contiguous()


def _softmax_mix(scores, v):
    """Softmax over the last axis, its product with v, and the log-sum."""
    top = scores.amax(-1)
    base = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weights = torch.exp(scores - base[..., None])
    total = weights.sum(-1)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    return torch.matmul(weights, v) / safe[..., None], torch.log(total) + base


def _plain_shared(st):
    c, q = st["case"], st["q"].float() * st["scale"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    width, pwidth = st["table"].shape[1] * c["page"], st["prefix_table"].shape[1] * c["page"]
    gone = torch.arange(width, device=_DEV)[None] >= st["lens"][:, None]
    pgone = torch.arange(pwidth, device=_DEV)[None] >= st["prefix_lens"][:, None]
    outs, lses = [], []
    for g in range(c["segments"]):
        a, b = int(st["seg_offsets"][g]), int(st["seg_offsets"][g + 1])
        n = b - a
        qg = q[a:b].view(n, hk, h // hk, d)
        k, v = (_gather(st, name, st["table"][a:b], width) for name in "kv")
        pk, pv = (_gather(st, name, st["prefix_table"][g:g + 1], pwidth)[0] for name in "kv")
        so = torch.matmul(qg, k.transpose(2, 3).contiguous())
        so = so.masked_fill(gone[a:b, None, None], float("-inf"))
        rows = qg.transpose(0, 1).reshape(hk, n * (h // hk), d)
        sp = torch.matmul(rows, pk.transpose(1, 2).contiguous())
        sp = sp.masked_fill(pgone[g], float("-inf"))
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


def _plain_single(st):
    """One token of each sequence: a few sequences at a time, all their keys, masked."""
    c, q = st["case"], st["q"].float() * st["scale"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    width = st["table"].shape[1] * c["page"]
    key = torch.arange(width, device=_DEV)[None]
    outs, lses = [], []
    step = max(1, (1 << 28) // (width * hk * d))
    for i in range(0, c["batch"], step):
        n = min(step, c["batch"] - i)
        last = st["lens"][i:i + n, None] - 1
        seen = (key <= last) & ((last - key < c["window"]) | (key < c["sinks"]))
        k, v = (_gather(st, name, st["table"][i:i + n], width) for name in "kv")
        sc = torch.matmul(q[i:i + n].view(n, hk, h // hk, d), k.transpose(2, 3).contiguous())
        out, lse = _softmax_mix(sc.masked_fill(~seen[:, None, None], float("-inf")), v)
        outs.append(out.reshape(n, h, d).to(torch.bfloat16))
        lses.append(lse.reshape(n, h))
    return torch.cat(outs), torch.cat(lses)


def _plain_window(st):
    c, q = st["case"], st["q"].float() * st["scale"]
    if c["q_len"] == 1:
        return _plain_single(st)
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    w, sinks = c["window"], c["sinks"]
    outs, lses, at = [], [], 0
    for i, (n, length) in enumerate(zip(st["q_lens"], st["host_lens"])):
        k, v = (_gather(st, name, st["table"][i:i + 1], length)[0] for name in "kv")
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
            out, lse = _softmax_mix(sc, v[:, cols][:, None])
            outs.append(out.permute(2, 0, 1, 3).reshape(m, h, d).to(torch.bfloat16))
            lses.append(lse.permute(2, 0, 1).reshape(m, h))
        at += n
    return torch.cat(outs), torch.cat(lses)


_OWN = {"write": _own_write, "read": _own_read, "shared": _own_shared, "window": _own_window}
_PLAIN = {"write": _plain_write, "read": _plain_read, "shared": _plain_shared,
          "window": _plain_window}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, st)
    if case["op"] == "read":
        return [_exact_tokens(case, st, name) for name in "kv"]
    return _exact_attention(case, st)


def _exact_e4m3(y):
    """fp64 values on the grid of e4m3: 3 bits behind the leading one, steps of 2^-9 at least."""
    _, power = torch.frexp(y)
    step = torch.exp2((power - 4).clamp(min=-9).double())
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_4bit(y):
    """fp64 values on the grid of their blocks: steps of 1/2, 1 and 2 in units of 2^e."""
    b = y.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 7.0))
    e = torch.where(top > 7.0 * torch.exp2(e), e + 1, e)       # (the logarithm's own rounding)
    e = torch.where(top <= 7.0 * torch.exp2(e - 1), e - 1, e).clamp(-125.0, 125.0)
    u = b / torch.exp2(e)
    step = torch.where(u.abs() < 2.0, 0.5, torch.where(u.abs() < 4.0, 1.0, 2.0)).double()
    return ((torch.round(u / step) * step).clamp(-6.0, 6.0) * torch.exp2(e)).flatten(-2)


def _exact_write(case, st):
    s = float(np.float32(case["scale"]))
    out = []
    for name in "kv":
        y = st["new_" + name].double() / s
        if case["kv"] == "fp4":
            out.append(_exact_4bit(y) * s)
            continue
        y = _exact_e4m3(y) if case["kv"] == "fp8" else y
        full = torch.zeros(st[name].shape, dtype=torch.float64, device=_DEV)
        at = 0
        for i, (n, length) in enumerate(zip(st["q_lens"], st["host_lens"])):
            t = torch.arange(length - n, length, device=_DEV)
            full[st["table"][i][t // case["page"]].long(), t % case["page"]] = y[at:at + n]
            at += n
        out.append(full)
    return out


def _rows64(st, name, ids, page, first, last):
    """fp64 [last - first, heads, dim]: token t of a sequence is row t % page of page ids[t // page]."""
    t = torch.arange(first, last, device=_DEV)
    at = ids[t // page].long(), t % page
    pages = st[name]
    if name + "_bytes" not in st:
        if pages.dtype == torch.float8_e4m3fn:
            return pages.view(torch.uint8)[at].contiguous().view(torch.float8_e4m3fn).double()
        return pages[at].double()
    c = pages[at]
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).long()
    m, p = c & 1, (c >> 1) & 3  # one bit behind the leading one, exponent (0: no leading one)
    size = torch.where(p > 0, (2 + m) * torch.exp2(p.double() - 2), 0.5 * m)
    x = torch.where(c > 7, -size, size).unflatten(-1, (-1, 32))
    return (x * torch.exp2(st[name + "_bytes"][at].double() - 127.0)[..., None]).flatten(-2)


def _exact_tokens(case, st, name):
    s = float(np.float32(case["scale"]))
    return torch.cat([_rows64(st, name, st["table"][i], case["page"], length - n, length) * s
                      for i, (n, length) in enumerate(zip(st["q_lens"], st["host_lens"]))])


def _exact_block(q, k, v, seen, scale):
    """One sequence's block: q [m, H, D], k and v [n, Hk, D], seen [m, n]."""
    m, h, d = q.shape
    hk = k.shape[1]
    out = torch.zeros((m, h, d), dtype=torch.float64, device=_DEV)
    lse = torch.full((m, h), float("-inf"), dtype=torch.float64, device=_DEV)
    alive = seen.any(1)
    for g in range(hk):
        vg = v[:, g].contiguous()
        for j in range(g * (h // hk), (g + 1) * (h // hk)):
            sc = (q[:, j].double() @ k[:, g].T.contiguous()) * scale
            sc = torch.where(seen, sc, torch.full_like(sc, float("-inf")))
            z = torch.logsumexp(sc, 1)
            wt = torch.exp(sc - torch.where(alive, z, torch.zeros_like(z))[:, None])
            out[:, j] = wt @ vg
            lse[:, j] = z
    return out, lse


def _exact_attention(case, st):
    page = case["page"]
    outs, lses = [], []
    if case["op"] == "shared":
        sizes, plen, olen = _shared_lengths(case)
        b = 0
        for g, n in enumerate(sizes):
            pre = [_rows64(st, name, st["prefix_table"][g], page, 0, plen[g]) for name in "kv"]
            for _ in range(n):
                k, v = (torch.cat([p, _rows64(st, name, st["table"][b], page, 0, olen[b])])
                        for p, name in zip(pre, "kv"))
                hk, d = k.shape[1], k.shape[2]
                q = st["q"][b].double().view(hk, -1, d)
                sc = torch.bmm(q, k.permute(1, 2, 0).contiguous()) * st["scale"]
                z = torch.logsumexp(sc, 2)
                o = torch.bmm(torch.exp(sc - z[..., None]), v.transpose(0, 1).contiguous())
                outs.append(o.reshape(1, -1, d))
                lses.append(z.reshape(1, -1))
                b += 1
        return torch.cat(outs), torch.cat(lses)
    q_lens, lens = _chunk_lengths(case)
    at = 0
    for i, (n, length) in enumerate(zip(q_lens, lens)):
        k, v = (_rows64(st, name, st["table"][i], page, 0, length) for name in "kv")
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
