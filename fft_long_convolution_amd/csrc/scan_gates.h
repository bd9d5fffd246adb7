// scan_gates.h -- the gates of the linear recurrence h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t, in fp32.
#pragma once
#include "block_kernels.h"
#include "mixer_io.h"

namespace lcv {
namespace {

__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }       // 1 ulp
__device__ __forceinline__ float fast_sqrt(float x) { return __builtin_amdgcn_sqrtf(x); }     // 1 ulp
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.f + __expf(-x)); }

// A sigmoid s and 1 - s in one register, each to its own size: the smaller of the two, negative where that is 1 - s.
__device__ __forceinline__ float folded_sigmoid(float x) {
    const float e = __expf(-fabsf(x)), small = fmaf(e, fast_rcp(1.f + e), 1e-37f);    // not zero: the sign is kept
    return x >= 0.f ? -small : small;
}
__device__ __forceinline__ float unfolded(float w) { return w > 0.f ? w : 1.f + w; }              // s
__device__ __forceinline__ float slope(float w) { return fabsf(w) * (1.f - fabsf(w)); }           // s (1 - s)

// A decay a and d = 1 - a, each to its own size: memories of thousands of tokens are in d, which 1 - a has lost.
// What a rounded to fp32 leaves out, (1 - a) - d (exact for a >= 1/2), goes along with it in the recurrence: a gate that
// stays where it is would add the same rounding up over its memory.
struct Decay {
    float a, d;
};
__device__ __forceinline__ Decay decay_of_log(float l) {       // a = exp(l), l <= 0
    // -expm1(l) as a Taylor polynomial near zero (next term: 0.25^6 / 5040 of the sum, 5e-8)
    const float p = -l * (1.f + l * (1.f / 2 + l * (1.f / 6 + l * (1.f / 24 + l * (1.f / 120 + l * (1.f / 720))))));
    const float e = __expf(l);
    const bool near = l > -0.25f;
    return Decay{near ? 1.f - p : e, near ? p : 1.f - e};
}
__device__ __forceinline__ Decay decay_of_logit(float z) {     // a = sigmoid(z)
    const float e = __expf(-fabsf(z)), big = fast_rcp(1.f + e), small = e * big;
    const bool slow = z >= 0.f;
    return Decay{slow ? 1.f - small : small, slow ? small : big};
}
__device__ __forceinline__ float residue(Decay g) { return g.a >= 0.5f ? (1.f - g.a) - g.d : 0.f; }

// A state h after one more token (or a run of tokens), the residue r of the decay a along
__device__ __forceinline__ float moved(float a, float r, float h, float u) { return fmaf(a, h, fmaf(r, h, u)); }
__device__ __forceinline__ float times(float x, float a, float r) { return fmaf(x, a, x * r); }

// The decay of a run of tokens.  Under gates that stay where they are every run has the same decay, and a rounding of it adds
// up as a token's would: 1 - a is carried along, 1 - a b = (1 - a) + (1 - b) - (1 - a)(1 - b), and the product itself only
// counts where little is left of it.
__device__ __forceinline__ void lengthen(Decay& run, float a, float d) {
    run.a *= a;
    run.d += fmaf(-run.d, d, d);
}
__device__ __forceinline__ Decay rounded(Decay run) { return Decay{run.d <= 0.5f ? 1.f - run.d : run.a, run.d}; }

// sqrt(1 - a^2)
__device__ __forceinline__ float norm_of(Decay g) { return fast_sqrt(g.d * (1.f + g.a)); }

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
    } else if constexpr (V == 2) {
        uint32_t w;
        __builtin_memcpy(&w, &r, 4);
        x[0] = unpack_lo<IO>(w);
        x[1] = unpack_hi<IO>(w);
    } else {
        x[0] = unpack_lo<IO>(r.e[0]);
    }
}
template <int IO, int V> __device__ __forceinline__ void store_v(void* base, int64_t token, uint32_t lane, const float* x) {
    typename Elem<IO>::T* p = (typename Elem<IO>::T*)base + token + lane;
    if constexpr (IO == CT_F32) {
        __builtin_memcpy(p, x, 4 * V);
    } else {
        const uint32_t w = pack2<IO>(x[0], V == 2 ? x[V - 1] : 0.f);
        __builtin_memcpy(p, &w, 2 * V);
    }
}

}  // namespace
}  // namespace lcv
