// rotary.hip -- rotary positions of q and k in one launch.
//
// (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a), a = position * inv_freq[p]: one read and one
// write of q and k, bound by HBM.  A thread owns 8 pairs of one token (or 16 copied elements) in HEADS heads, whose
// loads are all on their way while it forms the sines they share; every access is 16 bytes, at any element's alignment (half layouts whose halves do not start
// on a 16-byte group).  The angle is formed and reduced in fp64: position * inv_freq is exact there for
// any int32 position, while fp32 would be off by a fifth of a radian at a position of a million.
#include "mixer_kernels.h"
#include "mixer_io.h"

namespace lcv {
namespace {

template <int IO, int HEADS>
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
    const bool turn = u < turns;
    const int p = 8 * u, n = half - p < 8 ? half - p : 8;
    const int lo = !turn ? a.rot + 16 * (u - turns) : inter ? 2 * p : p;
    const int hi = !turn || inter ? lo + 8 : half + p;
    const int nlo = !turn ? a.D - lo : inter ? 2 * n : n;
    const int nhi = !turn ? a.D - hi : inter ? 2 * n - 8 : n;

    // the heads' data first, the sines while it is on its way
    float x[HEADS][16];
    const int h0 = hg * HEADS, heads = a.H + a.G;
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
        const int h = h0 + k;
        if (h >= heads) break;
        const bool isk = h >= a.H;
        const LinOperand& o = isk ? a.k : a.q;
        const int64_t xi = b * o.s.b + (int64_t)(isk ? h - a.H : h) * o.s.h + t * o.s.n;
        load8_part<IO>(o.p, xi + lo, nlo, x[k]);
        load8_part<IO>(o.p, xi + hi, nhi, x[k] + 8);
    }
    float c[8], s[8];
    if (turn) {
        const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + t] : t;
        float f[8];
        load8_part<CT_F32>(a.inv_freq, p, n, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            double ang = (double)pos * (double)f[k];
            ang -= 6.283185307179586 * rint(ang * 0.15915494309189535);
            sincosf((float)ang, &s[k], &c[k]);
            c[k] *= a.magnitude;
            s[k] *= a.flags & LCONV_ROTARY_INVERSE ? -a.magnitude : a.magnitude;
        }
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
        const int h = h0 + k;
        if (h >= heads) break;
        const bool isk = h >= a.H;
        const lconv_strides_t ys = isk ? a.yks : a.yqs;
        void* y = isk ? a.yk : a.yq;
        if (!turn && y == (isk ? a.k.p : a.q.p)) continue;     // in place: nothing to copy
        float z[16];
        if (!turn) {
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = x[k][e];
        } else if (inter) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[2 * e] = x[k][2 * e] * c[e] - x[k][2 * e + 1] * s[e];
                z[2 * e + 1] = x[k][2 * e + 1] * c[e] + x[k][2 * e] * s[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[e] = x[k][e] * c[e] - x[k][e + 8] * s[e];
                z[e + 8] = x[k][e + 8] * c[e] + x[k][e] * s[e];
            }
        }
        const int64_t yi = b * ys.b + (int64_t)(isk ? h - a.H : h) * ys.h + t * ys.n;
        store8_part<IO>(y, yi + lo, nlo, z);
        store8_part<IO>(y, yi + hi, nhi, z + 8);
    }
}

template <int IO>
void go(const RotaryArgs& a, hipStream_t stream) {
    const int turns = (a.rot / 2 + 7) / 8, units = turns + (a.D - a.rot + 15) / 16, heads = a.H + a.G;
    const int64_t each = a.B * a.N * units;
    // four heads to a thread where that still gives every compute unit a few waves of them
    const int per = each * ((heads + 3) / 4) >= 256 * 256 ? 4 : 1;
    const int hgroups = (heads + per - 1) / per;
    const int64_t total = each * hgroups;
    const unsigned grid = (unsigned)((total + 255) / 256);
    if (per == 4) rotary_kernel<IO, 4><<<grid, 256, 0, stream>>>(a, units, turns, hgroups, total);
    else rotary_kernel<IO, 1><<<grid, 256, 0, stream>>>(a, units, turns, hgroups, total);
}

}  // namespace

hipError_t launch_rotary(int dtype, const RotaryArgs& a, hipStream_t stream) {
    if (dtype == LCONV_F32) go<CT_F32>(a, stream);
    else if (dtype == LCONV_F16) go<CT_F16>(a, stream);
    else go<CT_BF16>(a, stream);
    return hipGetLastError();
}

}  // namespace lcv
