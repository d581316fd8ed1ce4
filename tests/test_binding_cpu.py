"""The Python binding without a GPU: a library that does not fit it."""
import shutil
import subprocess

import pytest

bd = pytest.importorskip("tenant_serving_bitdelta_amd")


def test_an_older_library_is_named_with_what_to_do(tmp_path, monkeypatch):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, lib = tmp_path / "old.c", tmp_path / "libold.so"
    src.write_text("int bitdelta_abi_version(void) { return %d; }\n" % bd.ABI_VERSION)
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(lib)], check=True, timeout=60)
    monkeypatch.setattr(bd, "LIB_PATH", str(lib))
    monkeypatch.setattr(bd, "_LIB", None)
    with pytest.raises(RuntimeError, match="build"):
        bd.lib()
    with pytest.raises(RuntimeError, match="bitdelta_attend_shared"):
        bd.abi_version()
