// Launches of the mixer operators' calls against a grid's reach, seen by launchers that record it: threads along a grid
// stay below 2^32, and a call past that is refused before its first launch.
#include <cstdint>
#include <cstdio>

#include "lconv.h"
#include "mixer_kernels.h"
#include "mixer_plan.h"

static int failures = 0, launches = 0;

static hipError_t grid(const char* what, int64_t workgroups) {
    ++launches;
    if (workgroups * 256 >= (int64_t)1 << 32) {
        std::fprintf(stderr, "%s: %lld workgroups of 256\n", what, (long long)workgroups);
        ++failures;
    }
    return hipSuccess;
}

namespace lcv {
hipError_t launch_linattn(int, const LinJob& a, hipStream_t) {
    return grid("chunks", (a.B * a.H * a.nseg + 7) / 8 * 8 * a.nroles * a.ncb);
}
hipError_t launch_linattn_step(int, const LinStepArgs& a, hipStream_t) {
    const int cb = linattn_step_columns(a.B * a.H, a.DV);
    return grid("tokens", a.B * a.H * ((a.DV + cb - 1) / cb));
}
hipError_t launch_linattn_tan(int, const LinTanArgs& a, float*, hipStream_t) {
    return grid("decay", a.B * a.H * a.nseg * linattn_tan_blocks(a.DV));
}
hipError_t launch_rotary(int, const RotaryArgs& a, hipStream_t) {
    const RotaryPlan p = rotary_plan(a.B * a.N, a.D, a.rot, a.H + a.G);
    return grid("rotary", (p.threads + 255) / 256);
}
hipError_t launch_head_sum(int, const HeadSumArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_copy_state(const float*, float*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_layernorm_fwd(int, const NormArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_layernorm_bwd(int, const NormArgs&, hipStream_t) { return hipSuccess; }
}  // namespace lcv

// a call launches everything or is refused and launches nothing
template <typename F> static bool taken(F&& call, int n) {
    launches = 0;
    const int st = call();
    if (!(st == LCONV_SUCCESS && launches == n) && !(st == LCONV_ERR_UNSUPPORTED && launches == 0)) {
        std::fprintf(stderr, "status %d after %d launches of %d\n", st, launches, n);
        ++failures;
    }
    return st == LCONV_SUCCESS;
}

static void* at(uint64_t a) { return (void*)(uintptr_t)(a << 56); }     // 2^56 bytes apart: the largest operand here
static float* fat(uint64_t a) { return (float*)at(a); }

int main() {
    const size_t much = (size_t)1 << 60;
    for (int64_t rows : {(int64_t)1, (int64_t)300, (int64_t)1 << 20, (int64_t)1 << 22, (int64_t)1 << 23, ((int64_t)1 << 24) - 8,
                         ((int64_t)1 << 24) - 1, (int64_t)1 << 24, ((int64_t)1 << 26) - 1, (int64_t)1 << 26})
        for (int64_t N : {(int64_t)1, (int64_t)70, (int64_t)5000})
            for (int64_t Dk : {8, 128, 256})
                for (int64_t Dv : {8, 128, 200, 256})
                    for (lconv_dtype_t dt : {LCONV_F32, LCONV_BF16}) {
                        const bool f = taken([&] {
                            return lconv_linattn_fwd(at(1), nullptr, at(2), nullptr, at(3), nullptr, fat(4), 1.f, nullptr, nullptr, at(5),
                                                     nullptr, nullptr, rows, 1, 1, N, Dk, Dv, dt, at(9), much, nullptr);
                        }, 1);
                        const bool alike = lcv::linattn_kt(Dk) == lcv::linattn_kt(Dv);
                        const bool b = taken([&] {
                            return lconv_linattn_bwd(at(1), nullptr, at(2), nullptr, at(3), nullptr, at(4), nullptr, fat(5), 1.f, nullptr,
                                                     nullptr, nullptr, at(6), nullptr, at(7), nullptr, at(8), nullptr, nullptr, fat(10),
                                                     rows, 1, 1, N, Dk, Dv, dt, at(9), much, nullptr);
                        }, alike ? 2 : 3);
                        const bool s = taken([&] {
                            return lconv_linattn_step(at(1), nullptr, at(2), nullptr, at(3), nullptr, fat(4), 1.f, fat(5), nullptr, at(6),
                                                      nullptr, rows, 1, 1, Dk, Dv, rows, dt, nullptr);
                        }, 1);
                        // what the header promises is taken
                        if (rows <= (1 << 20) && !(f && b)) ++failures;
                        if (rows <= (1 << 22) && !s) ++failures;
                        if (!f && lconv_linattn_workspace_bytes(rows, 1, 1, N, Dk, Dv, dt) != 0) ++failures;
                        if (!b && lconv_linattn_bwd_workspace_bytes(rows, 1, 1, N, Dk, Dv, dt) != 0) ++failures;
                    }
    for (int64_t tokens : {(int64_t)1, (int64_t)1 << 20, (int64_t)1 << 28, (int64_t)1 << 30, (int64_t)1 << 31, (int64_t)1 << 33, (int64_t)1 << 35})
        for (int64_t H : {1, 4, 33})
            for (int64_t D : {8, 24, 128})
                for (int64_t rot : {(int64_t)2, D}) {
                    const bool r = taken([&] {
                        return lconv_rotary(at(1), nullptr, nullptr, nullptr, nullptr, 0, fat(2), 1.f, at(3), nullptr, nullptr, nullptr, 1,
                                            H, 0, tokens, D, rot, 0, LCONV_BF16, nullptr);
                    }, 1);
                    if (tokens <= (1 << 20) && !r) ++failures;
                }
    if (failures) return 1;
    std::printf("MIXER_LIMITS_OK\n");
    return 0;
}
