// rotary_turn.h -- what the rotary kernels share: elements as they are stored, the sines of an angle, a unit of a head.
#pragma once
#include "mixer_io.h"

namespace lcv {
namespace {

// 8 elements as they are stored; the first n of them, the others zero
template <int IO> struct Raw8 { uint4 w[IO == CT_F32 ? 2 : 1]; };
template <int IO> __device__ __forceinline__ Raw8<IO> raw8_part(const void* base, int64_t i, int n) {
    Raw8<IO> r;
    const typename Elem<IO>::T* p = (const typename Elem<IO>::T*)base + i;
    if (n >= 8) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
        typename Elem<IO>::T e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = j < n ? p[j] : 0;
        __builtin_memcpy(&r, e, sizeof(r));
    }
    return r;
}

// The angle is formed and reduced to a quarter turn in fp64: position * inv_freq is off by at most 2^-53 of itself there,
// 2.4e-7 of a radian at the largest int32 position, while fp32 would be off by a thirtieth of one at a position of a
// million.  The sines
// of what is left, at most pi / 4, are Taylor polynomials in fp32 (next terms: x^11 / 11! < 2e-9, x^12 / 12! < 2e-10).
__device__ __forceinline__ void sines(double angle, float* s, float* c) {
    const double q = rint(angle * 0.6366197723675814);           // quarter turns
    const float x = (float)fma(q, -1.5707963267948966, angle), x2 = x * x;
    const int n = (int)(q - 4.0 * floor(q * 0.25));
    const float p = x + x * x2 * (-1.f / 6 + x2 * (1.f / 120 + x2 * (-1.f / 5040 + x2 * (1.f / 362880))));
    const float r = 1.f + x2 * (-0.5f + x2 * (1.f / 24 + x2 * (-1.f / 720 + x2 * (1.f / 40320 - x2 * (1.f / 3628800)))));
    const float a = n & 1 ? r : p, b = n & 1 ? p : r;
    *s = n & 2 ? -a : a;
    *c = (n + 1) & 2 ? -b : b;
}

}  // namespace
}  // namespace lcv
