"""Host code of the recurrence, the q/k norms and the short convolution (argument checks, plans, workspaces, dispatch) under the
address and undefined-behaviour sanitizers (CPU only; the device launchers replaced by ones that check what they are given)."""
import os

from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _run, _tool, outdir  # noqa: F401


def test_block_host_code_under_sanitizers(outdir):  # noqa: F811
    cxx, rocm = _tool("clang++"), "/opt/rocm"
    exe = os.path.join(outdir, "block_san")
    _run([cxx, *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-Wno-unused-result", "-Wno-unused-value",
          os.path.join(CSRC, "block_api.cpp"), os.path.join(HERE, "block_main.cpp"), "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    assert "BLOCK_SANITIZED_OK" in _run([exe], env=env).stdout
