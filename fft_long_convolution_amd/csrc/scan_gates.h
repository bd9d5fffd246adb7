// scan_gates.h -- the gates of the linear recurrence h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t, in fp32.
#pragma once
#include "block_kernels.h"
#include "token_io.h"

namespace lcv {
namespace {

// A sigmoid s and 1 - s = e s with e = exp(-x), each to its own size; the slope is their product.  Where e is past 2^126, s is too
// small for the reciprocal and both are zero.
struct Sigmoid {
    float s, rest;
};
__device__ __forceinline__ Sigmoid sloped_sigmoid(float x) {
    const float e = fast_exp2(-kLog2e * x), s = fast_rcp(1.f + e);
    return Sigmoid{s, fminf(e, 0x1p126f) * s};
}

// A decay a as c + w: c = 1 and w = a - 1 near one, c = 0 and w = a elsewhere, so that both a and 1 - a keep their own size.
// Memories of thousands of tokens are in 1 - a, which a rounded to fp32 has lost, and a gate that stays where it is would
// add one rounding of a up over its memory.
struct Decay {
    float c, w;
};
__device__ __forceinline__ float value_of(Decay k) { return k.c + k.w; }
__device__ __forceinline__ float loss_of(Decay k) { return (1.f - k.c) - k.w; }                   // 1 - a
__device__ __forceinline__ Decay decay_of_log2(float l) {      // a = 2^l, l <= 0
    // 2^l - 1 near zero by the quartic of least relative error for (2^l - 1) / l on [-0.25 log2(e), 0] (8e-9)
    const float p = l * fmaf(l, fmaf(l, fmaf(l, fmaf(l, 0.00120165572f, 0.00957710668f), 0.055498831f), 0.240226269f), 0.693147182f);
    const bool near = l > -0.36067376f;
    return Decay{near ? 1.f : 0.f, near ? p : fast_exp2(l)};
}
__device__ __forceinline__ Decay decay_of_logit(float z) {     // a = sigmoid(z)
    const float e = fast_exp2(-kLog2e * fabsf(z)), small = e * fast_rcp(1.f + e);
    const bool near = z >= 0.f;
    return Decay{near ? 1.f : 0.f, near ? -small : small};
}
// 1 - a^2 as -w (2 + w) or 1 - w^2, its root and one over that (0 for nothing).  A decay may lose less than 2^-126, which the
// hardware's roots take for zero (an inverse one gives infinity): the least loss there is, 2^-149, is a normal number times 2^32.
__device__ __forceinline__ float energy_of(Decay k) { return fmaf(-k.w, k.w, k.c > 0.f ? -2.f * k.w : 1.f); }
__device__ __forceinline__ float norm_of(Decay k) { return 0x1p-16f * fast_sqrt(0x1p32f * energy_of(k)); }
__device__ __forceinline__ float inverse_norm(float energy) { return energy > 0.f ? 0x1p16f * fast_rsqrt(0x1p32f * energy) : 0.f; }

// A state h after one more token or run of tokens, and x times a decay
__device__ __forceinline__ float moved(Decay k, float h, float u) { return fmaf(k.c, h, fmaf(k.w, h, u)); }
__device__ __forceinline__ float times(Decay k, float x) { return fmaf(k.c, x, k.w * x); }

// The decay of a run of tokens: its value and its loss, 1 - a b = (1 - a) + (1 - b) - (1 - a)(1 - b).  Under gates that stay
// where they are every run has the same decay, and a rounding of it would add up as a token's; the value only counts where
// little is left of it.
struct RunDecay {
    float a, d;
};
__device__ __forceinline__ void lengthen(RunDecay& run, Decay k) {
    const float d = loss_of(k);
    run.a = times(k, run.a);
    run.d += fmaf(-run.d, d, d);
}
__device__ __forceinline__ Decay whole(RunDecay run) {
    const bool near = run.d <= 0.5f;
    return Decay{near ? 1.f : 0.f, near ? -run.d : run.a};
}

}  // namespace
}  // namespace lcv
