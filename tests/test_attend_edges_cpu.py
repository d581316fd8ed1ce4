"""Paged attention without a GPU, at the ends of its arguments: the rows of a chunk that are computed,
and refusals (the addresses are fake)."""
import os
import shutil
import subprocess

import pytest

import test_attend_cpu as C

bd = pytest.importorskip("tenant_serving_bitdelta_amd")
if not os.path.exists(bd.LIB_PATH):
    pytest.skip("libbitdelta.so not built", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rows_of_a_chunk(tmp_path):
    hipcc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc"))
                  if c and os.path.exists(c)), None)
    if hipcc is None:
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "attend_chunk_check")
    r = subprocess.run([hipcc, "-O1", "-std=c++17", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
                        "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "attend_chunk_check.cpp"),
                        "-o", exe], capture_output=True, text=True, timeout=600)
    if r.returncode != 0 and "sanitizer" in r.stderr.lower() and "not found" in r.stderr:
        pytest.skip("sanitizer runtime not available")
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout + r.stderr)[-4000:]


@pytest.mark.parametrize("call", [C._shared, C._window])
@pytest.mark.parametrize("tokens,heads,kv_heads", [(1024, 1 << 14, 1 << 14), (1, (1 << 30) + 64, (1 << 24) + 1),
                                                   (1024, 1 << 21, 1 << 15), (700, 2997, 2997)])
def test_refuses_more_than_a_launch_holds(call, tokens, heads, kv_heads):
    kw = {"offs": (0, tokens)} if call is C._shared else {"batch": tokens}
    assert call(rows=C._rows(tokens=tokens, heads=heads), cache=C._cache(kv_heads=kv_heads), **kw) \
        == C.UNSUPPORTED


@pytest.mark.parametrize("call", [C._shared, C._window])
@pytest.mark.parametrize("scale,k_scale,status", [
    (1e30, 1e30, C.INVALID), (1e-30, 1e-30, C.INVALID), (3e38, 2.0, C.INVALID), (1e-38, 0.5, C.INVALID),
    (1e30, 1e-30, C.WORKSPACE), (1e-20, 1e-10, C.WORKSPACE), (1e20, 1e18, C.WORKSPACE)])
def test_refuses_scales_whose_product_is_no_number(call, scale, k_scale, status):
    """(a workspace too small is refused after them)"""
    assert call(rows=C._rows(scale=scale), cache=C._cache(k_scale=k_scale), ws_bytes=1000) == status


@pytest.mark.parametrize("offs,status", [
    ((0, 4), C.WORKSPACE), ((0, 2, 4), C.WORKSPACE), ((0, 3), C.SHAPE), ((1, 4), C.SHAPE),
    ((0, 3, 2, 4), C.SHAPE), (tuple([0] * 66) + (4,), C.INVALID)])
def test_segments_are_checked_without_prefixes(offs, status):
    assert C._shared(pt=None, pw=0, pl=None, offs=offs, ws_bytes=1000) == status


ONE = [(dict(heads=2), dict(kv_heads=1, k_stride_head=3, v_stride_head=1)),
       (dict(heads=1, q_stride_head=-1, out_stride_head=1), dict(kv_heads=1, k_stride_head=-3, v_stride_head=1)),
       (dict(), dict(num_pages=1, k_stride_page=1, v_stride_page=-1)),
       (dict(), dict(page_size=1, k_stride_token=1, v_stride_token=5)),
       (dict(tokens=1, q_stride_token=1, out_stride_token=-1), dict())]


@pytest.mark.parametrize("call", [C._shared, C._window])
@pytest.mark.parametrize("case", range(len(ONE)))
def test_strides_of_single_elements_may_be_anything(call, case):
    """(a workspace too small is refused after them)"""
    r, c = ONE[case]
    n = r.get("tokens", 4)
    kw = {"offs": (0, n), "pw": 4000} if call is C._shared else {"batch": n}
    assert call(rows=C._rows(**r), cache=C._cache(**c), width=4000, ws_bytes=1000, **kw) == C.WORKSPACE


@pytest.mark.parametrize("call,kw,status", [
    (C._shared, dict(width=1 << 29, pw=4), C.UNSUPPORTED), (C._shared, dict(width=1 << 27, pw=4), C.WORKSPACE),
    (C._shared, dict(width=4, pw=1 << 29), C.UNSUPPORTED), (C._shared, dict(width=4, pw=1 << 27), C.WORKSPACE),
    (C._window, dict(width=1 << 29, window=1 << 30), C.UNSUPPORTED),
    (C._window, dict(width=1 << 27, window=1 << 30), C.WORKSPACE),
    (C._window, dict(width=1 << 29, window=1 << 20), C.WORKSPACE)])
def test_refuses_tables_whose_steps_pass_32_bits(call, kw, status):
    """1024 sequences of up to 2^29 tokens (a workspace too small is refused after them)"""
    kw = dict(kw, **({"offs": (0, 1024)} if call is C._shared else {"batch": 1024}))
    assert call(rows=C._rows(tokens=1024), cache=C._cache(page_size=1), ws_bytes=1000, **kw) == status
