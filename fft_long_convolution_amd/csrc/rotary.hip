// rotary.hip -- rotary positions of q and k in one launch.
//
// (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a), a = position * inv_freq[p]: one read and one
// write of q and k, bound by HBM.  A thread owns 8 pairs of one token (or 16 copied elements) in up to four heads,
// which share the pairs' sines, one head at a time with the next one's loads on their way; every access is 16
// bytes, at any element's alignment (half layouts whose halves do not start on a 16-byte group).  Measured, 16384
// tokens of 32 heads of 128, bf16 (268 MB): one head to a thread 70 us, two 54, four 52 (5.1 TB/s, what a copy
// reaches), eight 52; with two or four heads' loads at a time 49 to 59 by layout.
// The angle is formed and reduced to a quarter turn in fp64: position * inv_freq is off by at most 2^-53 of itself there,
// 2.4e-7 of a radian at the largest int32 position, while fp32 would be off by a thirtieth of one at a position of a million.  The sines of what is left,
// at most pi / 4, are Taylor polynomials in fp32 (next terms: x^11 / 11! < 2e-9, x^12 / 12! < 2e-10).
#include "mixer_kernels.h"
#include "mixer_io.h"
#include "mixer_plan.h"

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

template <int IO>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryArgs a, int units, int turns, int per, int hgroups, int64_t total) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    // thread order: units of a token fastest, then groups of heads, then tokens
    const int u = (int)(i % units);
    const int64_t j = i / units;
    const int hg = (int)(j % hgroups);
    const int64_t row = j / hgroups;
    const int64_t b = row / a.N, t = row - b * a.N;
    const int half = a.rot / 2;
    const bool inter = a.flags & LCONV_ROTARY_INTERLEAVED;

    // the unit's two groups of 8 elements (interleaved: 16 in a row), and how many of each there are
    const bool turn = u < turns;
    const int p = 8 * u, n = half - p < 8 ? half - p : 8;
    const int lo = !turn ? a.rot + 16 * (u - turns) : inter ? 2 * p : p;
    const int hi = !turn || inter ? lo + 8 : half + p;
    const int nlo = !turn ? a.D - lo : inter ? 2 * n : n;
    const int nhi = !turn ? a.D - hi : inter ? 2 * n - 8 : n;

    struct Head { Raw8<IO> lo, hi; };
    const int h0 = hg * per, end = h0 + per < a.H + a.G ? h0 + per : a.H + a.G;
    const auto load = [&](int h) LCV_INLINE {
        const bool isk = h >= a.H;
        const LinOperand& o = isk ? a.k : a.q;
        const int64_t xi = b * o.s.b + (int64_t)(isk ? h - a.H : h) * o.s.h + t * o.s.n;
        return Head{raw8_part<IO>(o.p, xi + lo, nlo), raw8_part<IO>(o.p, xi + hi, nhi)};
    };
    Head x = load(h0);
    float c[8], s[8];
    if (turn) {
        const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + t] : t;
        float f[8];
        load8_part<CT_F32>(a.inv_freq, p, n, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sines((double)pos * (double)f[k], &s[k], &c[k]);
            c[k] *= a.magnitude;
            s[k] *= a.flags & LCONV_ROTARY_INVERSE ? -a.magnitude : a.magnitude;
        }
    }
    for (int h = h0; h < end; ++h) {
        const Head now = x;
        if (h + 1 < end) x = load(h + 1);
        const bool isk = h >= a.H;
        const lconv_strides_t ys = isk ? a.yks : a.yqs;
        void* y = isk ? a.yk : a.yq;
        if (!turn && y == (isk ? a.k.p : a.q.p)) continue;     // in place: nothing to copy
        float v[16], z[16];
        unpack_raw<IO>(now.lo.w, v);
        unpack_raw<IO>(now.hi.w, v + 8);
        if (!turn) {
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = v[e];
        } else if (inter) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[2 * e] = v[2 * e] * c[e] - v[2 * e + 1] * s[e];
                z[2 * e + 1] = v[2 * e + 1] * c[e] + v[2 * e] * s[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[e] = v[e] * c[e] - v[e + 8] * s[e];
                z[e + 8] = v[e + 8] * c[e] + v[e] * s[e];
            }
        }
        const int64_t yi = b * ys.b + (int64_t)(isk ? h - a.H : h) * ys.h + t * ys.n;
        store8_part<IO>(y, yi + lo, nlo, z);
        store8_part<IO>(y, yi + hi, nhi, z + 8);
    }
}

template <int IO>
void go(const RotaryArgs& a, hipStream_t stream) {
    const RotaryPlan p = rotary_plan(a.B * a.N, a.D, a.rot, a.H + a.G);
    rotary_kernel<IO><<<(unsigned)((p.threads + 255) / 256), 256, 0, stream>>>(a, p.units, p.turns, p.per, p.hgroups, p.threads);
}

}  // namespace

hipError_t launch_rotary(int dtype, const RotaryArgs& a, hipStream_t stream) {
    if (dtype == LCONV_F32) go<CT_F32>(a, stream);
    else if (dtype == LCONV_F16) go<CT_F16>(a, stream);
    else go<CT_BF16>(a, stream);
    return hipGetLastError();
}

}  // namespace lcv
