// token_io.h -- channels of a token [C] in a lane, and the sigmoid's parts, for the kernels of a recurrent block.
#pragma once
#include "mixer_io.h"

namespace lcv {
namespace {

__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }       // 1 ulp
__device__ __forceinline__ float fast_sqrt(float x) { return __builtin_amdgcn_sqrtf(x); }     // 1 ulp
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.f + __expf(-x)); }

// V channels of one token as they are stored, and as fp32
template <int IO, int V> struct RawV {
    typename Elem<IO>::T e[V];
};
template <int IO, int V> __device__ __forceinline__ RawV<IO, V> load_raw_v(const void* base, int64_t token, uint32_t lane) {
    RawV<IO, V> r;
    __builtin_memcpy(&r, (const typename Elem<IO>::T*)base + token + lane, sizeof(r));
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
template <int IO, int V> __device__ __forceinline__ void store_v(void* base, int64_t token, uint32_t lane, const float* x) {
    typename Elem<IO>::T* p = (typename Elem<IO>::T*)base + token + lane;
    if constexpr (IO == CT_F32) {
        __builtin_memcpy(p, x, 4 * V);
    } else {
        uint32_t w[(V + 1) / 2];
#pragma unroll
        for (int v = 0; v < (V + 1) / 2; ++v) w[v] = pack2<IO>(x[2 * v], 2 * v + 1 < V ? x[2 * v + 1] : 0.f);
        __builtin_memcpy(p, w, 2 * V);
    }
}

}  // namespace
}  // namespace lcv
