// The mixer operators' host code under the address and undefined-behaviour sanitizers: size queries over many shapes,
// the plans behind them, the refusals, and valid calls that end at a launcher's stand-in (LCONV_ERR_HIP).  Addresses are
// never dereferenced.  Exit status 0 when every status is the documented one.
#include <cstdint>
#include <cstdio>

#include "lconv.h"
#include "mixer_plan.h"

static int failures = 0;
#define EXPECT(call, want)                                                                                  \
    do {                                                                                                    \
        const int got_ = (int)(call);                                                                       \
        if (got_ != (int)(want)) {                                                                          \
            std::fprintf(stderr, "line %d: %s = %d, expected %d\n", __LINE__, #call, got_, (int)(want));     \
            ++failures;                                                                                     \
        }                                                                                                   \
    } while (0)

static void* at(uint64_t a) { return (void*)(uintptr_t)(a << 44); }
static float* fat(uint64_t a) { return (float*)at(a); }
static int32_t* iat(uint64_t a) { return (int32_t*)at(a); }

// a plan covers the row, no segment is empty, and the launch stays within a grid's reach
static void plans() {
    for (int64_t rows : {(int64_t)1, (int64_t)3, (int64_t)30, (int64_t)256, (int64_t)4096, ((int64_t)1 << 26) - 1})
        for (int roles : {1, 2, 3})
            for (int64_t N : {(int64_t)1, (int64_t)31, (int64_t)33, (int64_t)1001, (int64_t)65536, (int64_t)1 << 20, ((int64_t)1 << 31) - 1})
                for (int64_t DK : {8, 64, 88, 128, 136, 192, 256})
                    for (int64_t DV : {8, 64, 72, 128, 200, 256})
                        for (lconv_dtype_t dt : {LCONV_F32, LCONV_F16, LCONV_BF16}) {
                            const lcv::LinPlan p = lcv::linattn_plan(rows, roles, N, DK, DV, dt);
                            const bool ok = p.nseg >= 1 && p.seg_len % 32 == 0 && (int64_t)p.nseg * p.seg_len >= N &&
                                            (int64_t)(p.nseg - 1) * p.seg_len < N && (int64_t)p.ncb * 64 * p.nw >= DV &&
                                            16 * p.kt >= DK && (double)rows * roles * p.ncb * p.nseg < 2147483648.0;
                            const lcv::LinTanPlan t = lcv::linattn_tan_plan(rows, N, DV);
                            const bool tok = t.nseg >= 1 && t.seg_len % 32 == 0 && (int64_t)t.nseg * t.seg_len >= N &&
                                             (int64_t)(t.nseg - 1) * t.seg_len < N;
                            if (!ok || !tok) {
                                std::fprintf(stderr, "plan: rows %lld roles %d N %lld DK %lld DV %lld dtype %d\n", (long long)rows,
                                             roles, (long long)N, (long long)DK, (long long)DV, (int)dt);
                                ++failures;
                            }
                        }
    for (int64_t rows : {(int64_t)1, (int64_t)333, ((int64_t)1 << 31) - 1})
        for (int64_t C : {1, 7, 128, 129, 1001, 4096, 8192, 8193, 65536})
            if (lcv::layernorm_parts(rows, C) < 1 || lcv::layernorm_parts(rows, C) > rows) ++failures;
    for (int64_t C : {1, 128, 1001, 8192, 8193})
        if (lcv::layernorm_parts(0, C) != 0) {      // no rows leave no partial sum to be read
            std::fprintf(stderr, "layernorm_parts(0, %lld) = %lld\n", (long long)C, (long long)lcv::layernorm_parts(0, C));
            ++failures;
        }
}

int main() {
    plans();
    const lconv_dtype_t BF = LCONV_BF16;
    const size_t MUCH = (size_t)1 << 60;
    void *q = at(1), *k = at(2), *v = at(3), *y = at(4), *ws = at(9);
    float* ld = fat(5);
    lconv_strides_t far{((int64_t)1 << 40), (int64_t)1 << 36, (int64_t)1 << 30};
    // size queries: no shape outside the limits has a size, none overflows
    EXPECT(lconv_linattn_workspace_bytes(INT64_MAX, 2, 2, 64, 64, 64, BF), 0);
    EXPECT(lconv_linattn_workspace_bytes(2, INT64_MAX, INT64_MAX, INT64_MAX, 64, 64, BF), 0);
    EXPECT(lconv_linattn_workspace_bytes(1, 1, 1, 64, 12, 64, BF), 0);
    EXPECT(lconv_linattn_bwd_workspace_bytes(INT64_MAX, 1, 1, 64, 64, 64, BF), 0);
    EXPECT(lconv_linattn_bwd_workspace_bytes(1, 4, 3, 64, 64, 64, BF), 0);
    EXPECT(lconv_layernorm_bwd_workspace_bytes(INT64_MAX, 64), 0);
    EXPECT(lconv_linattn_workspace_bytes(1, 8, 8, 65536, 128, 128, BF) > 0, 1);
    // forward
    const auto fwd = [&](int64_t B, int64_t H, int64_t G, int64_t N, int64_t Dk, int64_t Dv, const lconv_strides_t* qs, size_t wsb) {
        return lconv_linattn_fwd(q, qs, k, nullptr, v, nullptr, ld, 1.f, nullptr, nullptr, y, nullptr, nullptr, B, H, G, N, Dk,
                                 Dv, BF, ws, wsb, nullptr);
    };
    EXPECT(fwd(2, 4, 2, 100, 64, 64, nullptr, MUCH), LCONV_ERR_HIP);
    EXPECT(fwd(1, 8, 8, 65536, 128, 128, nullptr, MUCH), LCONV_ERR_HIP);
    EXPECT(fwd(1, 8, 8, 65536, 128, 128, nullptr, 16), LCONV_ERR_WORKSPACE);
    EXPECT(fwd(0, 4, 2, 100, 64, 64, nullptr, 0), LCONV_SUCCESS);
    EXPECT(fwd(-1, 4, 2, 100, 64, 64, nullptr, 0), LCONV_ERR_INVALID_SHAPE);
    EXPECT(fwd(2, 4, 3, 100, 64, 64, nullptr, 0), LCONV_ERR_UNSUPPORTED);
    EXPECT(fwd(INT64_MAX, 4, 2, 100, 64, 64, nullptr, 0), LCONV_ERR_UNSUPPORTED);
    EXPECT(fwd(2, 4, 2, 4, 64, 64, &far, MUCH), LCONV_ERR_UNSUPPORTED);
    far.n = INT64_MAX / 2 / 16 * 16;
    EXPECT(fwd(2, 4, 2, 100, 64, 64, &far, MUCH), LCONV_ERR_INVALID_SHAPE);
    // gradients, with every optional operand
    const auto bwd = [&](int64_t H, int64_t G, int64_t N, int64_t Dk, int64_t Dv, size_t wsb) {
        return lconv_linattn_bwd(q, nullptr, k, nullptr, v, nullptr, y, nullptr, ld, 1.f, fat(10), fat(11), iat(12), at(13),
                                 nullptr, at(14), nullptr, at(15), nullptr, fat(16), fat(17), 2, H, G, N, Dk, Dv, BF, ws, wsb,
                                 nullptr);
    };
    for (int64_t G : {8, 2})
        for (int64_t N : {1, 100, 5000})
            for (int64_t Dk : {64, 256})
                for (int64_t Dv : {64, 128}) EXPECT(bwd(8, G, N, Dk, Dv, MUCH), LCONV_ERR_HIP);
    EXPECT(bwd(8, 2, 100, 64, 64, 0), LCONV_ERR_WORKSPACE);
    EXPECT(bwd(8, 2, -1, 64, 64, MUCH), LCONV_ERR_INVALID_SHAPE);
    // single tokens
    const auto step = [&](int64_t B, int64_t slots, const int32_t* s) {
        return lconv_linattn_step(q, nullptr, k, nullptr, v, nullptr, ld, 1.f, fat(10), s, y, nullptr, B, 4, 2, 64, 64, slots, BF, nullptr);
    };
    EXPECT(step(3, 3, nullptr), LCONV_ERR_HIP);
    EXPECT(step(3, 2, nullptr), LCONV_ERR_INVALID_SHAPE);
    EXPECT(step(3, 2, iat(11)), LCONV_ERR_HIP);
    EXPECT(step(3, INT64_MAX / 2, iat(11)), LCONV_ERR_INVALID_SHAPE);
    // rotary
    const auto rot = [&](int64_t N, int64_t D, int64_t r, int64_t ps, int flags) {
        return lconv_rotary(q, nullptr, k, nullptr, iat(5), ps, fat(6), 1.f, y, nullptr, at(7), nullptr, 2, 4, 2, N, D, r, flags, BF, nullptr);
    };
    EXPECT(rot(100, 64, 32, 100, 0), LCONV_ERR_HIP);
    EXPECT(rot(100, 64, 31, 100, 0), LCONV_ERR_UNSUPPORTED);
    EXPECT(rot(100, 64, 32, 100, 4), LCONV_ERR_UNSUPPORTED);
    EXPECT(rot(100, 64, 32, INT64_MAX, 0), LCONV_ERR_INVALID_SHAPE);
    EXPECT(rot(INT64_MAX, 64, 32, 0, 0), LCONV_ERR_UNSUPPORTED);
    // layer norm
    const auto nf = [&](int64_t rows, int64_t C, int64_t xs) {
        return lconv_layernorm_fwd(q, xs, k, v, y, C, fat(5), fat(6), rows, C, 1e-5f, BF, nullptr);
    };
    EXPECT(nf(100, 1001, 1001), LCONV_ERR_HIP);
    EXPECT(nf(100, 1001, 1000), LCONV_ERR_INVALID_SHAPE);
    EXPECT(nf(100, 1001, INT64_MAX), LCONV_ERR_INVALID_SHAPE);
    EXPECT(nf(100, 65537, 65537), LCONV_ERR_UNSUPPORTED);
    EXPECT(nf(0, 64, 64), LCONV_SUCCESS);
    const auto nb = [&](int64_t rows, int64_t C, size_t wsb) {
        return lconv_layernorm_bwd(q, C, k, C, v, fat(5), fat(6), y, C, fat(7), fat(8), rows, C, BF, ws, wsb, nullptr);
    };
    EXPECT(nb(100, 1001, MUCH), LCONV_ERR_HIP);
    EXPECT(nb(100, 1001, 8), LCONV_ERR_WORKSPACE);
    EXPECT(nb(100, 20000, MUCH), LCONV_ERR_HIP);
    if (failures) return 1;
    std::printf("MIXER_SANITIZED_OK\n");
    return 0;
}
