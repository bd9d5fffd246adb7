// mixer_io.h -- element access of the mixer kernels: groups of 8 elements of any dtype as fp32.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fused_io.h"
#include "mixer_kernels.h"

namespace lcv {
namespace {

template <int IO> struct Elem { using T = uint16_t; };
template <> struct Elem<CT_F32> { using T = float; };

template <int IO> __device__ __forceinline__ void store1(void* base, int64_t i, float v) {
    if constexpr (IO == CT_F32) ((float*)base)[i] = v;
    else ((uint16_t*)base)[i] = (uint16_t)(pack2<IO>(v, 0.f) & 0xffffu);
}

// 8 elements in a row from any element on (16-byte accesses need no alignment here).
template <int IO> __device__ __forceinline__ void load8_any(const void* base, int64_t i, float* x) {
    uint4 r[IO == CT_F32 ? 2 : 1];
    __builtin_memcpy(r, (const typename Elem<IO>::T*)base + i, sizeof(r));
    unpack_raw<IO>(r, x);
}
template <int IO> __device__ __forceinline__ void store8_any(void* base, int64_t i, const float* x) {
    typename Elem<IO>::T* p = (typename Elem<IO>::T*)base + i;
    if constexpr (IO == CT_F32) {
        __builtin_memcpy(p, x, 32);
    } else {
        const uint4 w = make_uint4(pack2<IO>(x[0], x[1]), pack2<IO>(x[2], x[3]), pack2<IO>(x[4], x[5]), pack2<IO>(x[6], x[7]));
        __builtin_memcpy(p, &w, 16);
    }
}
// the first n of 8 elements, the others zero
template <int IO> __device__ __forceinline__ void load8_part(const void* base, int64_t i, int n, float* x) {
    if (n >= 8) {
        load8_any<IO>(base, i, x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < n ? load1<IO>(base, i + j) : 0.f;
    }
}
template <int IO> __device__ __forceinline__ void store8_part(void* base, int64_t i, int n, const float* x) {
    if (n >= 8) {
        store8_any<IO>(base, i, x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) store1<IO>(base, i + j, x[j]);
    }
}

// The base of an operand's row (b, h): element offset of its token 0.
__device__ __forceinline__ int64_t row_base(const LinOperand& o, int64_t b, int h) {
    return b * o.s.b + (int64_t)(h / o.share) * o.s.h;
}

__device__ __forceinline__ int64_t row_len(const int32_t* lengths, int64_t b, int64_t N) {
    if (!lengths) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < N ? n : N;
}

// log(gamma), kept finite, also times any number of tokens, so that gamma^0 is 1 where gamma is 0 (a NaN stays one).
__device__ __forceinline__ float log_gamma(const float* log_decay, int h) {
    const float l = log_decay[h];
    return l < -1e20f ? -1e20f : l;
}

// gamma^n, relative to its own size: what the product's rounding leaves out (88 half-units for the smallest powers) is
// put back.
__device__ __forceinline__ float decay_power(float lg, float n) {
    const float x = lg * n, g = expf(x);
    return fmaf(g, fmaf(lg, n, -x), g);
}

// gamma^n as the sum of two floats.  A state that is multiplied over and over takes the product of all its factors, so
// that the rounding of one factor would add up over its memory (gamma^n = 1 - 1e-4: ten thousand times half a unit).
// S hi + S lo rounds once.  (S + S expm1 would do near one, but not for fast decays: 1 + expm1(-16) is 6 % off.)
struct DecayPair {
    float hi, lo;
};
__device__ __forceinline__ DecayPair decay_pair(float lg, float n) {
    const double g = exp((double)lg * (double)n);
    const float hi = (float)g;
    return DecayPair{hi, (float)(g - (double)hi)};
}
template <typename V> __device__ __forceinline__ V decayed(V S, DecayPair g, V add) { return S * g.hi + (S * g.lo + add); }

}  // namespace
}  // namespace lcv
