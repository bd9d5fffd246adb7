// What the mixer operators' C entries hand to their launchers, seen by launchers that record it: strides over dimensions
// of length one never reach address arithmetic.  Addresses are computed as the chunk kernel does and never dereferenced.
#include <cstdint>
#include <cstdio>

#include "lconv.h"
#include "mixer_kernels.h"

static lcv::LinJob job;
static lcv::RotaryArgs turn;
static int failures = 0, jobs = 0, turns = 0;

namespace lcv {
hipError_t launch_linattn(int, const LinJob& a, hipStream_t) {
    job = a;
    ++jobs;
    // the first token of each operand of a single-token call, by the kernel's own steps: a 64-bit scalar at the chunk's
    // lowest token and a 32-bit offset from there
    for (int i = 0; i < a.nroles && a.N == 1; ++i) {
        const LinRole& r = a.r[i];
        const int64_t low = r.reverse ? 1 - 32 : 0;
        const auto first = [&](const char* what, const void* p, int64_t stride, int size, int tokens) {
            const uint64_t got = (uint64_t)(uintptr_t)p + (uint64_t)(low * stride * size) + (r.reverse ? 32 - tokens : 0) * (uint64_t)(stride * size) +
                                 (uint64_t)((uint32_t)(r.reverse ? tokens - 1 : 0) * (uint32_t)(stride * size));
            if (got != (uint64_t)(uintptr_t)p) {
                std::fprintf(stderr, "role %d: %s is read at %llx, stands at %llx\n", i, what, (unsigned long long)got,
                             (unsigned long long)(uintptr_t)p);
                ++failures;
            }
        };
        first("Q", r.Q.p, r.Q.s.n, 2, 32);
        first("K", r.K.p, r.K.s.n, 2, 32);
        first("V", r.V.p, r.V.s.n, 2, 32);
        first("O", r.O, r.o.n, r.wide ? 4 : 2, 16);     // stores go by 16 tokens
    }
    return hipSuccess;
}
hipError_t launch_rotary(int, const RotaryArgs& a, hipStream_t) {
    turn = a;
    ++turns;
    return hipSuccess;
}
hipError_t launch_linattn_step(int, const LinStepArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_linattn_tan(int, const LinTanArgs&, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_head_sum(int, const HeadSumArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_copy_state(const float*, float*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_layernorm_fwd(int, const NormArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_layernorm_bwd(int, const NormArgs&, hipStream_t) { return hipSuccess; }
}  // namespace lcv

#define EXPECT(ok)                                                            \
    do {                                                                      \
        if (!(ok)) {                                                          \
            std::fprintf(stderr, "line %d: %s\n", __LINE__, #ok);             \
            ++failures;                                                       \
        }                                                                     \
    } while (0)

static void* at(uint64_t a) { return (void*)(uintptr_t)(a << 44); }
static float* fat(uint64_t a) { return (float*)at(a); }

int main() {
    const int64_t D = 64;
    const size_t much = (size_t)1 << 60;
    for (int64_t wild : {D, (int64_t)1 << 27, (int64_t)1 << 28, (int64_t)1 << 40, INT64_MAX / 128, (int64_t)-64, (int64_t)3})
        for (int64_t G : {2, 4}) {
            const lconv_strides_t h4{4 * D, D, wild}, hg{G * D, D, wild};
            EXPECT(lconv_linattn_fwd(at(1), &h4, at(2), &hg, at(3), &hg, fat(4), 1.f, nullptr, nullptr, at(5), &h4, nullptr,
                                     2, 4, G, 1, D, D, LCONV_BF16, at(9), much, nullptr) == LCONV_SUCCESS);
            EXPECT(lconv_linattn_bwd(at(1), &h4, at(2), &h4, at(3), &hg, at(4), &hg, fat(5), 1.f, nullptr, nullptr, nullptr,
                                     at(6), &h4, at(7), &hg, at(8), &hg, nullptr, nullptr, 2, 4, G, 1, D, D, LCONV_BF16, at(9),
                                     much, nullptr) == LCONV_SUCCESS);
        }
    EXPECT(jobs == 28);
    // one batch row and one head of many tokens: their strides are not used either
    const lconv_strides_t one{INT64_MIN, INT64_MAX, D};
    EXPECT(lconv_linattn_fwd(at(1), &one, at(2), &one, at(3), &one, fat(4), 1.f, nullptr, nullptr, at(5), &one, nullptr, 1, 1, 1,
                             40, D, D, LCONV_BF16, at(9), much, nullptr) == LCONV_SUCCESS);
    EXPECT(job.r[0].Q.s.b == 0 && job.r[0].Q.s.h == 0 && job.r[0].Q.s.n == D && job.r[0].o.b == 0);
    // in place is in place whatever the strides that no address depends on
    const lconv_strides_t x{4 * D, D, 7}, y{4 * D, D, 16};
    EXPECT(lconv_rotary(at(1), &x, nullptr, nullptr, nullptr, 0, fat(2), 1.f, at(1), &y, nullptr, nullptr, 2, 4, 0, 1, D, D, 0,
                        LCONV_BF16, nullptr) == LCONV_SUCCESS);
    EXPECT(turns == 1 && turn.q.s.n == turn.yqs.n);
    if (failures) return 1;
    std::printf("MIXER_STRIDES_OK\n");
    return 0;
}
