"""Plain forms of the paged cache's stored types, for the tests: numpy, value by value.  y = x / scale is
one fp32 division, as the interface has it; all that follows is exact in float64."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quotient(x, scale):
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        return (np.asarray(x, np.float32) / np.float32(scale)).astype(np.float64)


def encode4(x, scale=1.0):
    """(codes uint8 [..., n], scale bytes uint8 [..., n / 32]) of values [..., n]; a block that is not
    finite: byte 255, codes 0."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)).all(-1)
    y = quotient(x, scale).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    y = np.clip(np.where(bad[..., None], 0.0, y), -3.4028234663852886e38, 3.4028234663852886e38)
    top = np.abs(y).max(-1)
    e = np.full(top.shape, -125)
    for k in range(-125, 125):  # the smallest e with top <= 7 * 2^e
        e = np.where(top > 7.0 * 2.0 ** k, k + 1, e)
    u = np.abs(y) / 2.0 ** e[..., None]
    d = np.abs(u[..., None] - GRID)
    near = d.min(-1)
    # of two as near the even code
    code = np.full(u.shape, -1)
    for c in (1, 3, 5, 7, 0, 2, 4, 6):
        code = np.where(d[..., c] == near, c, code)
    code = np.where(np.signbit(y), code + 8, code)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def decode4(codes, byte):
    v = np.concatenate([GRID, -GRID])[codes].reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(codes.shape)


def pack4(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack4(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def encode8(x, scale=1.0):
    """float64 values of e4m3: 3 bits behind the leading one, steps of 2^-9 at least, 448 at most."""
    x = np.asarray(x, np.float64)
    y = np.clip(quotient(x, scale), -448.0, 448.0)
    _, p = np.frexp(np.where(np.isfinite(y), y, 0.0))
    step = 2.0 ** np.maximum(p - 4, -9)
    r = np.clip(np.rint(y / step) * step, -448.0, 448.0)
    return np.where(np.isfinite(x), r, np.nan)


def bf16(x):
    """float64 values rounded to bf16 from fp32 (all that is stored comes from there)."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().bfloat16().double().numpy()


def places(q_lens, lens, table, page, pages):
    """(row, sequence, page id, slot) of every row, id -1 where its token has no place."""
    out, row = [], 0
    for b, n in enumerate(q_lens):
        for i in range(n):
            pos = lens[b] - n + i
            at = pos // page if pos >= 0 else -1
            pid = int(table[b][at]) if 0 <= at < table.shape[1] else -1
            out.append((row, b, pid if 0 <= pid < pages else -1, pos % page))
            row += 1
    return out
