"""Calls whose launches would pass a grid's reach are refused before the first launch (CPU, under the sanitizers)."""
import os

from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _run, _tool, outdir  # noqa: F401


def test_launches_stay_within_a_grid(outdir):  # noqa: F811
    cxx, rocm = _tool("clang++"), "/opt/rocm"
    exe = os.path.join(outdir, "mixer_limits")
    srcs = [os.path.join(CSRC, "mixer_api.cpp"), os.path.join(HERE, "mixer_limits_main.cpp")]
    _run([cxx, *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-Wno-unused-result", "-Wno-unused-value", *srcs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    assert "MIXER_LIMITS_OK" in _run([exe], env=env).stdout
