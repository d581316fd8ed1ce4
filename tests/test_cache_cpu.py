"""Writing and reading the paged cache without a GPU: every refusal of the two entry points, which come
before any device memory is touched (the addresses are fake), and the tests' own plain forms by hand."""
import ctypes
import os

import numpy as np
import pytest
import torch

import cache_ref as R

bd = pytest.importorskip("tenant_serving_bitdelta_amd")
if not os.path.exists(bd.LIB_PATH):
    pytest.skip("libbitdelta.so not built", allow_module_level=True)

L = bd.lib()
OK, INVALID, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5
FAKE = 0x7F0000000000


def _cache(**kw):
    c = bd._KvCache()
    d = dict(k=FAKE, v=FAKE, dtype=2, num_pages=64, page_size=16, kv_heads=2, head_dim=128,
             k_stride_page=4096, k_stride_token=256, k_stride_head=128, v_stride_page=4096,
             v_stride_token=256, v_stride_head=128, k_scale=1.0, v_scale=1.0, k_block_scales=FAKE,
             v_block_scales=FAKE)
    d.update(kw)
    for n, v in d.items():
        setattr(c, n, v)
    return c


def _rows(**kw):
    r = bd._KvRows()
    d = dict(k=FAKE, v=FAKE, tokens=4, k_stride_token=256, k_stride_head=128, v_stride_token=256,
             v_stride_head=128)
    d.update(kw)
    for n, v in d.items():
        setattr(r, n, v)
    return r


def _call(f, rows=None, cache=None, batch=4, table=FAKE, width=200, lens=FAKE, qo=FAKE):
    rows, cache = rows or _rows(), cache or _cache()
    return f(ctypes.byref(rows), ctypes.byref(cache), batch, table, width, lens, qo, None)


BOTH = [L.bitdelta_cache_write, L.bitdelta_cache_read]


@pytest.mark.parametrize("f", BOTH)
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
    (dict(k_block_scales=None), INVALID), (dict(v_block_scales=None), INVALID),
    (dict(k_block_scales=FAKE + 2), ALIGN), (dict(v_block_scales=FAKE + 1), ALIGN),
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(k_stride_token=64), ALIGN), (dict(v_stride_page=4096 + 64), ALIGN),
    (dict(k_stride_head=-128), INVALID), (dict(k_stride_page=128 << 36), UNSUPPORTED), (dict(k=FAKE + 8), ALIGN),
    (dict(k_scale=0.0), INVALID), (dict(k_scale=float("nan")), INVALID), (dict(v_scale=float("inf")), INVALID),
    (dict(kv_heads=(1 << 16) + 1), UNSUPPORTED),
])
def test_refuses_bad_cache(f, kw, status):
    assert _call(f, cache=_cache(**kw)) == status


@pytest.mark.parametrize("f", BOTH)
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(tokens=-1), INVALID),
    (dict(k_stride_token=252), ALIGN), (dict(v_stride_head=4), ALIGN), (dict(k_stride_head=-8), INVALID),
    (dict(v_stride_token=-256), INVALID), (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN),
    (dict(tokens=(1 << 29) + 1), UNSUPPORTED),
])
def test_refuses_bad_rows(f, kw, status):
    assert _call(f, rows=_rows(**kw)) == status


@pytest.mark.parametrize("f", BOTH)
@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(width=-1), INVALID), (dict(table=FAKE + 2), ALIGN), (dict(lens=FAKE + 3), ALIGN),
    (dict(qo=FAKE + 2), ALIGN), (dict(batch=1025), UNSUPPORTED), (dict(width=1 << 27), UNSUPPORTED),
    (dict(qo=None, batch=3), SHAPE), (dict(qo=None, batch=5), SHAPE),
])
def test_refuses_bad_tables(f, kw, status):
    assert _call(f, **kw) == status


@pytest.mark.parametrize("f", BOTH)
def test_null_structures_and_empty_calls(f):
    assert f(None, ctypes.byref(_cache()), 4, FAKE, 200, FAKE, FAKE, None) == INVALID
    assert f(ctypes.byref(_rows()), None, 4, FAKE, 200, FAKE, FAKE, None) == INVALID
    assert _call(f, rows=_rows(tokens=0, k=None, v=None)) == OK
    assert _call(f, batch=0) == OK


def test_reference_by_hand():
    x = np.zeros(64)
    x[:12] = [7.0, 6.9, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -5.01, -0.0]
    x[32:34] = [7.01, 1.0]  # twice the step
    codes, byte = R.encode4(x)
    assert list(byte) == [127, 128]
    assert list(codes[:12]) == [7, 7, 6, 6, 4, 4, 2, 2, 0, 8, 15, 8]
    assert list(codes[32:34]) == [6, 1]  # 3.505 -> 4, 0.5 -> 0.5
    v = R.decode4(codes, byte)
    assert list(v[:4]) == [6, 6, 4, 4] and list(v[32:34]) == [8, 1]
    assert np.array_equal(R.unpack4(R.pack4(codes)), codes)
    x[40] = np.inf
    assert list(R.encode4(x)[1]) == [127, 255] and np.isnan(R.decode4(*R.encode4(x))[32:]).all()
    assert list(R.encode4(np.full(32, 1e-40))[1]) == [2] and list(R.encode4(np.full(32, 3e38))[1]) == [252]
    y = np.concatenate([np.linspace(-500, 500, 3001), np.linspace(-0.1, 0.1, 777)]).astype(np.float32)
    y = y[np.abs(y) < 464]  # beyond, torch's conversion gives NaN
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.encode8(y), want)
    assert np.isnan(R.encode8([np.inf, np.nan])).all() and list(R.encode8([1e9, -500.0])) == [448, -448]


@pytest.mark.parametrize("dim", [64, 128])
def test_error_is_at_most_half_a_step(dim):
    x = np.random.default_rng(dim).normal(size=(500, dim)) * np.exp2(np.random.default_rng(1).integers(-20, 20, (500, 1)))
    x = R.bf16(x)
    codes, byte = R.encode4(x)
    unit = np.repeat(2.0 ** (byte.astype(float) - 127), 32, -1)
    v = R.decode4(codes, byte)
    top = np.abs(x) / unit
    half = np.where(top <= 2, 0.25, np.where(top <= 4, 0.5, 1.0)) * unit
    assert (np.abs(v - x) <= half).all() and top.max() <= 7
