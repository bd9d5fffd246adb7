// rotary.hip -- rotary positions of q and k in one launch.
#include "mixer_kernels.h"
#include "mixer_io.h"

namespace lcv {
namespace {

// One thread per (b, token, dimension pair or copied pair); it serves every head, so the sine and
// cosine are computed once per (b, token, pair).
template <int IO>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryArgs a, int64_t total) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int half = a.D / 2;
    const int64_t row = i / half;
    const int p = (int)(i - row * half);
    const int64_t b = row / a.N, t = row - b * a.N;
    int lo = 2 * p, hi = 2 * p + 1;
    float c = 1.f, s = 0.f;
    const bool turned = 2 * p < a.rot;
    if (turned) {
        const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + t] : t;
        double ang = (double)pos * (double)a.inv_freq[p];
        ang -= 6.283185307179586 * rint(ang * 0.15915494309189535);
        sincosf((float)ang, &s, &c);
        if (a.flags & LCONV_ROTARY_INVERSE) s = -s;
        c *= a.magnitude;
        s *= a.magnitude;
        if (!(a.flags & LCONV_ROTARY_INTERLEAVED)) { lo = p; hi = p + a.rot / 2; }
    }
    for (int o = 0; o < 2; ++o) {
        const LinOperand& x = o ? a.k : a.q;
        if (!x.p) continue;
        const lconv_strides_t ys = o ? a.yks : a.yqs;
        void* y = o ? a.yk : a.yq;
        for (int h = 0; h < (o ? a.G : a.H); ++h) {
            const int64_t xi = b * x.s.b + h * x.s.h + t * x.s.n, yi = b * ys.b + h * ys.h + t * ys.n;
            const float u = load1<IO>(x.p, xi + lo), v = load1<IO>(x.p, xi + hi);
            store1<IO>(y, yi + lo, turned ? u * c - v * s : u);
            store1<IO>(y, yi + hi, turned ? v * c + u * s : v);
        }
    }
}

}  // namespace

hipError_t launch_rotary(int dtype, const RotaryArgs& a, hipStream_t stream) {
    const int64_t total = a.B * a.N * (a.D / 2);
    const unsigned grid = (unsigned)((total + 255) / 256);
    if (dtype == LCONV_F32) rotary_kernel<CT_F32><<<grid, 256, 0, stream>>>(a, total);
    else if (dtype == LCONV_F16) rotary_kernel<CT_F16><<<grid, 256, 0, stream>>>(a, total);
    else rotary_kernel<CT_BF16><<<grid, 256, 0, stream>>>(a, total);
    return hipGetLastError();
}

}  // namespace lcv
