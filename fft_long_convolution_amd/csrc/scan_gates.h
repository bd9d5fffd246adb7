// scan_gates.h -- the gates of the linear recurrence h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t, in fp32.
#pragma once
#include "block_kernels.h"
#include "token_io.h"

namespace lcv {
namespace {

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

}  // namespace
}  // namespace lcv
