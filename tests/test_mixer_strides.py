"""Strides over dimensions of length one: what the C entries hand to the launchers (CPU, under the sanitizers), and
single-token gradients on such strides (GPU)."""
import os

import numpy as np
import pytest

from tests.mixer_util import host, say
from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _run, _tool, outdir  # noqa: F401


def test_strides_of_single_tokens_reach_no_address(outdir):  # noqa: F811
    cxx, rocm = _tool("clang++"), "/opt/rocm"
    exe = os.path.join(outdir, "mixer_strides")
    srcs = [os.path.join(CSRC, "mixer_api.cpp"), os.path.join(HERE, "mixer_strides_main.cpp")]
    _run([cxx, *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-Wno-unused-result", "-Wno-unused-value", *srcs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    assert "MIXER_STRIDES_OK" in _run([exe], env=env).stdout


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G", [2, 4])
def test_single_token_gradients_on_strides_that_no_token_uses(dtype, G):
    """A token stride of 2^29 bytes that one token never steps over: bit for bit the dense call's gradients, on operands
    and on outputs."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    say(f"[linattn one token, unused strides] {dtype} G={G}")
    rng = np.random.default_rng(90 + G)
    B, H, Dk, Dv = 3, 4, 64, 40
    t = {"q": host(rng, (B, H, 1, Dk), dtype).cuda(), "k": host(rng, (B, G, 1, Dk), dtype).cuda(),
         "v": host(rng, (B, G, 1, Dv), dtype).cuda(), "dy": host(rng, (B, H, 1, Dv), dtype).cuda()}
    ld = torch.full((H,), -0.1, device="cuda")
    S, dS = host(rng, (B, H, Dk, Dv), "f32").cuda(), host(rng, (B, H, Dk, Dv), "f32").cuda()
    code = lconv.dtype_code(t["q"].dtype)
    need = lconv.lconv_linattn_bwd_workspace_bytes(B, H, G, 1, Dk, Dv, code)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    unused = 2 ** 29 // t["q"].element_size()
    runs = []
    for n in (None, unused):
        st = lambda heads, D: None if n is None else lconv.Strides(heads * D, D, n)  # noqa: E731,B023
        out = {"dq": torch.empty_like(t["q"]), "dk": torch.empty_like(t["k"]), "dv": torch.empty_like(t["v"]),
               "ds": torch.empty_like(S), "dl": torch.empty_like(ld)}
        status = lconv.lconv_linattn_bwd(
            t["dy"].data_ptr(), st(H, Dv), t["q"].data_ptr(), st(H, Dk), t["k"].data_ptr(), st(G, Dk), t["v"].data_ptr(), st(G, Dv),
            ld.data_ptr(), 0.3, S.data_ptr(), dS.data_ptr(), None, out["dq"].data_ptr(), st(H, Dk), out["dk"].data_ptr(), st(G, Dk),
            out["dv"].data_ptr(), st(G, Dv), out["ds"].data_ptr(), out["dl"].data_ptr(), B, H, G, 1, Dk, Dv, code, ws.data_ptr(),
            need, torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        runs.append(out)
    for name in runs[0]:
        assert bool((runs[0][name] == runs[1][name]).all()), name
