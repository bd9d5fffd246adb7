// rotary.hip -- rotary positions of q and k in one launch.
//
// (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a), a = position * inv_freq[p]: one read and one
// write of q and k, bound by HBM.  A thread owns 8 pairs of one token (or 16 copied elements) and walks a
// few heads with them, so that sines are formed once for HEADS heads while there are still enough
// threads; every access is 16 bytes, at any element's alignment (half layouts whose halves do not start
// on a 16-byte group).  The angle is formed and reduced in fp64: position * inv_freq is exact there for
// any int32 position, while fp32 would be off by a fifth of a radian at a position of a million.
#include "mixer_kernels.h"
#include "mixer_io.h"

namespace lcv {
namespace {

constexpr int HEADS = 8;

template <int IO>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryArgs a, int units, int turns, int hgroups, int64_t total) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    // thread order: units of a head fastest, then heads, then tokens
    const int u = (int)(i % units);
    const int64_t j = i / units;
    const int hg = (int)(j % hgroups);
    const int64_t row = j / hgroups;
    const int64_t b = row / a.N, t = row - b * a.N;
    const int half = a.rot / 2;
    const bool inter = a.flags & LCONV_ROTARY_INTERLEAVED;

    // the unit's two groups of 8 elements (interleaved: 16 in a row), and how many of each there are
    int lo, hi, nlo, nhi;
    float c[8], s[8];
    if (u < turns) {
        const int p = 8 * u, n = half - p < 8 ? half - p : 8;
        const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + t] : t;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            double ang = (double)pos * (double)a.inv_freq[k < n ? p + k : p];
            ang -= 6.283185307179586 * rint(ang * 0.15915494309189535);
            sincosf((float)ang, &s[k], &c[k]);
            c[k] *= a.magnitude;
            s[k] *= a.flags & LCONV_ROTARY_INVERSE ? -a.magnitude : a.magnitude;
        }
        lo = inter ? 2 * p : p;
        hi = inter ? lo + 8 : half + p;
        nlo = inter ? 2 * n : n;
        nhi = inter ? 2 * n - 8 : n;
    } else {
        lo = a.rot + 16 * (u - turns);
        hi = lo + 8;
        nlo = a.D - lo;
        nhi = a.D - hi;
    }
    const int heads = a.H + a.G, h1 = (hg + 1) * HEADS < heads ? (hg + 1) * HEADS : heads;
    for (int h = hg * HEADS; h < h1; ++h) {
        const bool isk = h >= a.H;
        const LinOperand& xo = isk ? a.k : a.q;
        const lconv_strides_t ys = isk ? a.yks : a.yqs;
        void* y = isk ? a.yk : a.yq;
        const int hh = isk ? h - a.H : h;
        if (u >= turns && y == xo.p) continue;     // in place: nothing to copy
        const int64_t xi = b * xo.s.b + hh * xo.s.h + t * xo.s.n, yi = b * ys.b + hh * ys.h + t * ys.n;
        float x[16], z[16];
        load8_part<IO>(xo.p, xi + lo, nlo, x);
        load8_part<IO>(xo.p, xi + hi, nhi, x + 8);
        if (u >= turns) {
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] = x[k];
        } else if (inter) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                z[2 * k] = x[2 * k] * c[k] - x[2 * k + 1] * s[k];
                z[2 * k + 1] = x[2 * k + 1] * c[k] + x[2 * k] * s[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                z[k] = x[k] * c[k] - x[k + 8] * s[k];
                z[k + 8] = x[k + 8] * c[k] + x[k] * s[k];
            }
        }
        store8_part<IO>(y, yi + lo, nlo, z);
        store8_part<IO>(y, yi + hi, nhi, z + 8);
    }
}

}  // namespace

hipError_t launch_rotary(int dtype, const RotaryArgs& a, hipStream_t stream) {
    const int turns = (a.rot / 2 + 7) / 8, units = turns + (a.D - a.rot + 15) / 16;
    const int hgroups = (a.H + a.G + HEADS - 1) / HEADS;
    const int64_t total = a.B * a.N * hgroups * units;
    const unsigned grid = (unsigned)((total + 255) / 256);
    if (dtype == LCONV_F32) rotary_kernel<CT_F32><<<grid, 256, 0, stream>>>(a, units, turns, hgroups, total);
    else if (dtype == LCONV_F16) rotary_kernel<CT_F16><<<grid, 256, 0, stream>>>(a, units, turns, hgroups, total);
    else rotary_kernel<CT_BF16><<<grid, 256, 0, stream>>>(a, units, turns, hgroups, total);
    return hipGetLastError();
}

}  // namespace lcv
