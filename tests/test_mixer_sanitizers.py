"""The mixer operators' host code (argument checks, plans, workspace layouts, dispatch) under the address and
undefined-behaviour sanitizers (CPU only; the device launchers replaced by stand-ins that fail)."""
import os

from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _run, _tool, outdir  # noqa: F401


def test_mixer_host_code_under_sanitizers(outdir):  # noqa: F811
    cxx, rocm = _tool("clang++"), "/opt/rocm"
    exe = os.path.join(outdir, "mixer_san")
    srcs = [os.path.join(CSRC, "mixer_api.cpp"), os.path.join(HERE, "mixer_stubs.cpp"), os.path.join(HERE, "mixer_main.cpp")]
    _run([cxx, *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-Wno-unused-result", "-Wno-unused-value", *srcs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = _run([exe], env=env)
    assert "MIXER_SANITIZED_OK" in r.stdout
