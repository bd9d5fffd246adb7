// The marks of the gated recurrence, which the caller allocates by the size query, near the limit of a grid: a call that
// launches has a query that gives the room that its kernels write, for every type, and its marks' whole range is kept apart
// from the other operands.  Launchers record; addresses are never dereferenced.  Exit status 0 when all holds.
#include <cstdint>
#include <cstdio>

#include "block_kernels.h"
#include "lconv.h"

static int failures = 0, launches = 0;

static void need(bool ok, const char* what, int64_t B, int64_t N, int64_t C, int dt) {
    if (ok) return;
    std::fprintf(stderr, "%s: %lld x %lld x %lld, type %d\n", what, (long long)B, (long long)N, (long long)C, dt);
    ++failures;
}

namespace lcv {
hipError_t launch_scan_fwd(int, const ScanArgs&, hipStream_t) { return ++launches, hipSuccess; }
hipError_t launch_scan_bwd(int, const ScanArgs&, hipStream_t) { return ++launches, hipSuccess; }
hipError_t launch_scan_step(int, const ScanStepArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_row_state(const float*, float*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_qknorm_fwd(int, const QkArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_qknorm_bwd(int, const QkArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_conv_fwd(int, const ConvArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_conv_bwd(int, const ConvArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_conv_step(int, const ConvStepArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_conv_state(int, const void*, void*, int64_t, hipStream_t) { return hipSuccess; }
}  // namespace lcv

static void* at(uint64_t a) { return (void*)(uintptr_t)(a << 57); }
static float* fat(uint64_t a) { return (float*)at(a); }

int main() {
    const size_t much = (size_t)1 << 60;
    int taken = 0, refused = 0;
    for (int64_t B : {(int64_t)1, (int64_t)65536, (int64_t)131072, (int64_t)1 << 20, (int64_t)3000000, ((int64_t)1 << 22) - 1, (int64_t)1 << 24})
        for (int64_t N : {1, 8, 16, 64, 65, 1000})
            for (int64_t C : {1, 64, 66, 128, 130, 2560, 5120, 1 << 17})
                for (lconv_dtype_t dt : {LCONV_F32, LCONV_F16, LCONV_BF16}) {
                    const size_t marks = (size_t)B * (size_t)((N + 63) / 64) * (size_t)C * 4;
                    const auto fwd = [&](float* state_out) {
                        return lconv_gated_scan_fwd(at(1), nullptr, at(2), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, at(6), nullptr,
                                                    state_out, fat(7), B, N, C, LCONV_GATE_SIGMOID, dt, at(8), much, nullptr);
                    };
                    const auto bwd = [&](void* dx) {
                        return lconv_gated_scan_bwd(at(1), nullptr, at(2), nullptr, at(3), nullptr, nullptr, nullptr, nullptr, fat(7), nullptr,
                                                    nullptr, dx, nullptr, at(9), nullptr, nullptr, nullptr, nullptr, nullptr, B, N, C,
                                                    LCONV_GATE_SIGMOID, dt, at(12), much, nullptr);
                    };
                    launches = 0;
                    const int f = fwd(nullptr), b = bwd(at(8));
                    need((f == LCONV_SUCCESS) == (b == LCONV_SUCCESS) && launches == (f == LCONV_SUCCESS ? 2 : 0), "one pass alone", B, N, C, dt);
                    if (f != LCONV_SUCCESS) {
                        ++refused;
                        need(f == LCONV_ERR_UNSUPPORTED, "status", B, N, C, dt);
                        continue;
                    }
                    ++taken;
                    need(lconv_gated_scan_marks_bytes(B, N, C) == marks, "room for marks", B, N, C, dt);
                    // outputs in the marks' last bytes
                    char* const end = (char*)fat(7) + (marks - 1) / 16 * 16;
                    need(fwd((float*)end) == LCONV_ERR_ALIASING, "state in the marks", B, N, C, dt);
                    need(bwd(end) == LCONV_ERR_ALIASING, "gradient in the marks", B, N, C, dt);
                }
    if (taken == 0 || refused == 0) ++failures;
    if (failures) return 1;
    std::printf("BLOCK_SIZES_OK\n");
    return 0;
}
