"""Paged attention without a GPU: the index arithmetic the kernels share with the host (page
quotients, key lists, bad tables, the split over workgroups) and every refusal of the two entry
points, which come before any device memory is touched (the addresses are fake)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

bd = pytest.importorskip("tenant_serving_bitdelta_amd")
if not os.path.exists(bd.LIB_PATH):
    pytest.skip("libbitdelta.so not built", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = bd.lib()
OK, INVALID, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5
FAKE = 0x7F0000000000
BIG = 1 << 40


def _build_and_run(tmp_path, flags):
    hipcc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc"))
                  if c and os.path.exists(c)), None)
    if hipcc is None:
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "attend_index_check")
    r = subprocess.run([hipcc, "-O1", "-std=c++17", *flags,
                        os.path.join(ROOT, "tests", "attend_index_check.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=600)
    if r.returncode != 0 and "sanitizer" in r.stderr.lower() and "not found" in r.stderr:
        pytest.skip("sanitizer runtime not available")
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout + r.stderr)[-4000:]


def test_index_arithmetic(tmp_path):
    _build_and_run(tmp_path, [])


def test_index_arithmetic_under_host_sanitizers(tmp_path):
    _build_and_run(tmp_path, ["-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
                              "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"])


def _cache(**kw):
    c = bd._KvCache()
    d = dict(k=FAKE, v=FAKE, dtype=0, num_pages=64, page_size=16, kv_heads=2, head_dim=128,
             k_stride_page=4096, k_stride_token=256, k_stride_head=128, v_stride_page=4096,
             v_stride_token=256, v_stride_head=128, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    for n, v in d.items():
        setattr(c, n, v)
    return c


def _rows(**kw):
    r = bd._AttendRows()
    d = dict(q=FAKE, out=FAKE, lse=None, tokens=4, heads=8, q_stride_token=1024, q_stride_head=128,
             out_stride_token=1024, out_stride_head=128, scale=0.1)
    d.update(kw)
    for n, v in d.items():
        setattr(r, n, v)
    return r


def _shared(rows=None, cache=None, table=FAKE, width=200, lens=FAKE, pt=FAKE, pw=300, pl=FAKE,
            offs=(0, 4), ws=FAKE, ws_bytes=BIG):
    rows, cache = rows or _rows(), cache or _cache()
    o = np.asarray(offs, dtype=np.int32)
    return L.bitdelta_attend_shared(ctypes.byref(rows), ctypes.byref(cache), table, width, lens, pt,
                                    pw, pl, o.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                    len(offs) - 1, ws, ws_bytes, None)


def _window(rows=None, cache=None, batch=4, table=FAKE, width=200, lens=FAKE, qo=None, mq=1,
            window=3000, sinks=4, ws=FAKE, ws_bytes=BIG):
    rows, cache = rows or _rows(), cache or _cache()
    return L.bitdelta_attend_window(ctypes.byref(rows), ctypes.byref(cache), batch, table, width,
                                    lens, qo, mq, window, sinks, ws, ws_bytes, None)


BAD_CACHE = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_heads=3), SHAPE), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(k_stride_token=4), ALIGN),
    (dict(v_stride_page=4097), ALIGN), (dict(k_stride_head=-128), INVALID),
    (dict(dtype=1, k_stride_head=136), ALIGN), (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN),
    (dict(k_scale=0.0), INVALID), (dict(k_scale=float("nan")), INVALID),
    (dict(v_scale=float("inf")), INVALID), (dict(v_scale=-1.0), INVALID),
]
BAD_ROWS = [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(tokens=-1), INVALID),
    (dict(heads=0), INVALID), (dict(heads=7), SHAPE), (dict(heads=256), UNSUPPORTED),
    (dict(q_stride_token=1020), ALIGN), (dict(q_stride_head=-8), INVALID),
    (dict(out_stride_head=2), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(out=FAKE + 4), ALIGN),
    (dict(lse=FAKE + 2), ALIGN), (dict(scale=0.0), INVALID), (dict(scale=-0.5), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
]


@pytest.mark.parametrize("call", [_shared, _window])
@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_refuses_bad_cache(call, kw, status):
    assert call(cache=_cache(**kw)) == status


@pytest.mark.parametrize("call", [_shared, _window])
@pytest.mark.parametrize("kw,status", BAD_ROWS)
def test_refuses_bad_rows(call, kw, status):
    assert call(rows=_rows(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(width=-1), INVALID),
    (dict(pt=None), INVALID), (dict(pl=None), INVALID), (dict(pw=-1), INVALID),
    (dict(table=FAKE + 2), ALIGN), (dict(pl=FAKE + 1), ALIGN), (dict(width=1 << 27), UNSUPPORTED),
    (dict(pw=(1 << 26), width=8), UNSUPPORTED),
    (dict(offs=(0, 3)), SHAPE), (dict(offs=(1, 4)), SHAPE), (dict(offs=(0, 3, 2, 4)), SHAPE),
    (dict(offs=tuple([0] * 66) + (4,)), INVALID), (dict(rows=_rows(tokens=1025), offs=(0, 1025)), UNSUPPORTED),
    (dict(ws=None, ws_bytes=0), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
    (dict(ws=FAKE + 8), ALIGN),
])
def test_shared_refusals(kw, status):
    assert _shared(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(window=0), INVALID), (dict(sinks=-1), INVALID),
    (dict(mq=0), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(lens=FAKE + 3), ALIGN), (dict(qo=FAKE + 2), ALIGN), (dict(batch=1025), UNSUPPORTED),
    (dict(mq=2), SHAPE), (dict(batch=3), SHAPE), (dict(width=1 << 27), UNSUPPORTED),
    (dict(ws=None, ws_bytes=0), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
])
def test_window_refusals(kw, status):
    assert _window(**kw) == status


def test_empty_calls_do_nothing():
    assert _shared(rows=_rows(tokens=0, q=None, out=None), offs=(0,)) == OK
    assert _window(rows=_rows(tokens=0, q=None, out=None)) == OK
    assert _window(batch=0) == OK


def test_workspace_queries():
    o = np.asarray([0, 4], dtype=np.int32)
    op = o.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    c = _cache()
    need = L.bitdelta_attend_shared_workspace_bytes(4, 8, ctypes.byref(c), 200, 300, op, 1)
    assert need > 0 and _shared(ws_bytes=need - 1) == WORKSPACE
    # short key lists need none, nor do refused arguments
    assert L.bitdelta_attend_shared_workspace_bytes(4, 8, ctypes.byref(c), 2, 3, op, 1) == 0
    assert L.bitdelta_attend_shared_workspace_bytes(4, 7, ctypes.byref(c), 200, 300, op, 1) == 0
    need = L.bitdelta_attend_window_workspace_bytes(4, 8, ctypes.byref(c), 4, 200, 1, 3000, 4)
    assert need > 0 and _window(ws_bytes=need - 1) == WORKSPACE
    assert L.bitdelta_attend_window_workspace_bytes(4, 8, ctypes.byref(c), 4, 200, 1, 100, 4) == 0
    assert L.bitdelta_attend_window_workspace_bytes(4, 8, ctypes.byref(c), 4, 200, 512, 100, 4) == 0
