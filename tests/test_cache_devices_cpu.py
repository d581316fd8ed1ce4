"""Caches whose tensors are on several devices are refused before anything is launched.  (Fake tensors: they
have a device and a shape, and no memory.)"""
import os

import pytest

torch = pytest.importorskip("torch")
bd = pytest.importorskip("tenant_serving_bitdelta_amd")
fake = pytest.importorskip("torch._subclasses.fake_tensor")
if not os.path.exists(bd.LIB_PATH):
    pytest.skip("libbitdelta.so not built", allow_module_level=True)

DTYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "fp4": torch.uint8}


@pytest.fixture
def empty():
    """make(shape, dtype, index): on device `index`"""
    with fake.FakeTensorMode():
        yield lambda shape, dtype, index=0: torch.empty(shape, dtype=dtype, device=f"cuda:{index}")


def _pages(empty, kv, index):
    shape = (4, 16, 2, 32 if kv == "fp4" else 64)
    return empty(shape, DTYPES[kv], index), empty((*shape[:3], 2), torch.uint8, index)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("call", ["write", "read", "shared", "window"])
def test_values_on_another_device_than_keys(empty, kv, call):
    (k, kb), (v, vb) = _pages(empty, kv, 0), _pages(empty, kv, 1)
    x = empty((2, 2, 64), torch.bfloat16)
    table, lens = empty((2, 3), torch.int32), empty((2,), torch.int32)
    blocks = dict(k_block_scales=kb, v_block_scales=vb) if kv == "fp4" else {}
    with pytest.raises(ValueError, match="v_pages are on cuda:1, k_pages on cuda:0"):
        if call == "write":
            bd.cache_write(x, x, k, v, table, lens, **blocks)
        elif call == "read":
            bd.cache_read(k, v, table, lens, **blocks)
        elif call == "shared":
            bd.attend_shared(x, k, v, table, lens, None, None, [0, 2], **blocks)
        else:
            bd.attend_window(x, k, v, table, lens, 8, **blocks)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("what", ["k", "v", "table", "lens"])
def test_rows_and_tables_on_another_device_than_the_pages(empty, kv, what, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)  # (asked for between the checks)
    (k, kb), (v, vb) = _pages(empty, kv, 0), _pages(empty, kv, 0)
    blocks = dict(k_block_scales=kb, v_block_scales=vb) if kv == "fp4" else {}
    on = {name: int(name == what) for name in ("k", "v", "table", "lens")}
    rows = [empty((2, 2, 64), torch.bfloat16, on[name]) for name in "kv"]
    table, lens = empty((2, 3), torch.int32, on["table"]), empty((2,), torch.int32, on["lens"])
    q_offsets = empty((3,), torch.int32)
    with pytest.raises(ValueError, match="on cuda:"):
        bd.cache_write(*rows, k, v, table, lens, q_offsets, **blocks)
    with pytest.raises(ValueError, match="on cuda:"):
        bd.cache_read(k, v, table, lens, q_offsets, k_out=rows[0], v_out=rows[1], **blocks)
