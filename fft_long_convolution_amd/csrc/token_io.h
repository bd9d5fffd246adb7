// token_io.h -- channels of a token [C] in a lane, and the sigmoid's parts, for the kernels of a recurrent block.
#pragma once
#include "mixer_io.h"

namespace lcv {
namespace {

constexpr float kLog2e = 1.44269504f;

// Single instructions, off by one unit in the last place; exponentials below 2^-126 are zero, and a number below that is zero to
// the roots and the reciprocal (whose inverse is infinite).
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float fast_sqrt(float x) { return __builtin_amdgcn_sqrtf(x); }
__device__ __forceinline__ float fast_rsqrt(float x) { return __builtin_amdgcn_rsqf(x); }
__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.f + fast_exp2(-kLog2e * x)); }

// V channels of one token as they are stored, and as fp32
template <int IO, int V> struct RawV {
    typename Elem<IO>::T e[V];
};
// element `token` + `lane`: the first part is the same for a wave, the second in bytes fits 32 bits (an instruction's own offset)
template <int IO> __device__ __forceinline__ const typename Elem<IO>::T* place_of(const void* base, int64_t token, uint32_t lane) {
    using T = typename Elem<IO>::T;
    const uint32_t bytes = lane * (uint32_t)sizeof(T);
    return (const T*)((const char*)((const T*)base + token) + bytes);
}
template <int IO, int V> __device__ __forceinline__ RawV<IO, V> load_raw_v(const void* base, int64_t token, uint32_t lane) {
    RawV<IO, V> r;
    __builtin_memcpy(&r, place_of<IO>(base, token, lane), sizeof(r));
    return r;
}
template <int IO, int V> __device__ __forceinline__ void widen(const RawV<IO, V>& r, float* x) {
    if constexpr (IO == CT_F32) {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = r.e[v];
    } else if constexpr (V > 1) {
        uint32_t w[V / 2];
        __builtin_memcpy(w, &r, 2 * V);
#pragma unroll
        for (int v = 0; v < V / 2; ++v) {
            x[2 * v] = unpack_lo<IO>(w[v]);
            x[2 * v + 1] = unpack_hi<IO>(w[v]);
        }
    } else {
        x[0] = unpack_lo<IO>(r.e[0]);
    }
}
template <int IO, int V> __device__ __forceinline__ RawV<IO, V> narrow(const float* x) {
    RawV<IO, V> r;
    if constexpr (IO == CT_F32) {
        __builtin_memcpy(&r, x, sizeof(r));
    } else {
        uint32_t w[(V + 1) / 2];
#pragma unroll
        for (int v = 0; v < (V + 1) / 2; ++v) w[v] = pack2<IO>(x[2 * v], 2 * v + 1 < V ? x[2 * v + 1] : 0.f);
        __builtin_memcpy(&r, w, sizeof(r));
    }
    return r;
}
template <int IO, int V> __device__ __forceinline__ void store_raw_v(void* base, int64_t token, uint32_t lane, const RawV<IO, V>& r) {
    __builtin_memcpy((void*)place_of<IO>(base, token, lane), &r, sizeof(r));
}
template <int IO, int V> __device__ __forceinline__ void store_v(void* base, int64_t token, uint32_t lane, const float* x) {
    store_raw_v<IO, V>(base, token, lane, narrow<IO, V>(x));
}

}  // namespace
}  // namespace lcv
