"""A library built from older sources says so when it is loaded (CPU)."""
import os
import shutil
import subprocess

import pytest

from fft_long_convolution_amd import lconv


def test_a_library_without_an_entry_point(tmp_path, monkeypatch):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    src, so = tmp_path / "old.c", str(tmp_path / "old.so")
    src.write_text("int lconv_abi_version(void) { return 8; }\n")
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", so], check=True)
    monkeypatch.setattr(lconv, "_lib", None)
    with pytest.raises(RuntimeError, match="older sources"):
        lconv.load(so)
    with pytest.raises(RuntimeError, match="missing"):
        lconv.load(os.path.join(str(tmp_path), "none.so"))
    assert lconv._lib is None
