// layernorm.hip -- layer norm: forward, and the gradients of its input, weight and bias.
#include "mixer_kernels.h"
#include "mixer_io.h"

namespace lcv {
namespace {

__device__ __forceinline__ float block_sum(float v, float* red) {
    for (int w = 32; w; w >>= 1) v += __shfl_xor(v, w);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];
}

// One workgroup per row.
template <int IO>
__global__ void __launch_bounds__(256) ln_fwd_kernel(NormArgs a) {
    __shared__ float red[4];
    const int64_t row = blockIdx.x, xo = row * a.xs, yo = row * a.ys;
    const int C = (int)a.C;
    float s = 0.f;
    for (int c = threadIdx.x; c < C; c += 256) s += load1<IO>(a.x, xo + c);
    // the first mean is off by the rounding of a sum of the values themselves; what is left of it
    // shows in the centred sum and is taken out
    const float first = block_sum(s, red) / (float)C;
    float s2 = 0.f;
    s = 0.f;
    for (int c = threadIdx.x; c < C; c += 256) {
        const float d = load1<IO>(a.x, xo + c) - first;
        s += d;
        s2 += d * d;
    }
    const float rest = block_sum(s, red) / (float)C;
    const float mean = first + rest;
    const float rstd = 1.f / sqrtf(fmaxf(block_sum(s2, red) / (float)C - rest * rest, 0.f) + a.eps);
    for (int c = threadIdx.x; c < C; c += 256) {
        float y = (load1<IO>(a.x, xo + c) - first - rest) * rstd;
        if (a.weight) y *= load1<IO>(a.weight, c);
        if (a.bias) y += load1<IO>(a.bias, c);
        store1<IO>(a.y, yo + c, y);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <int IO>
__global__ void __launch_bounds__(256) ln_dx_kernel(NormArgs a) {
    __shared__ float red[4];
    const int64_t row = blockIdx.x, xo = row * a.xs, yo = row * a.ys, go = row * a.dys;
    const int C = (int)a.C;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < C; c += 256) {
        float g = load1<IO>(a.dy, go + c);
        if (a.weight) g *= load1<IO>(a.weight, c);
        s1 += g;
        s2 += g * (load1<IO>(a.x, xo + c) - mean) * rstd;
    }
    s1 = block_sum(s1, red) / (float)C;
    s2 = block_sum(s2, red) / (float)C;
    for (int c = threadIdx.x; c < C; c += 256) {
        float g = load1<IO>(a.dy, go + c);
        if (a.weight) g *= load1<IO>(a.weight, c);
        const float xh = (load1<IO>(a.x, xo + c) - mean) * rstd;
        store1<IO>(a.y, yo + c, rstd * (g - s1 - xh * s2));
    }
}

// Partial column sums of block blockIdx.y's rows: part[0 / 1][block][C] for dweight / dbias.  It reads
// dy and x before the dx kernel may overwrite one of them in place.
template <int IO>
__global__ void __launch_bounds__(256) ln_part_kernel(NormArgs a, int64_t nparts) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.C) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += nparts) {
        const float g = load1<IO>(a.dy, row * a.dys + c);
        sw += g * (load1<IO>(a.x, row * a.xs + c) - a.mean[row]) * a.rstd[row];
        sb += g;
    }
    a.part[blockIdx.y * a.C + c] = sw;
    a.part[(nparts + blockIdx.y) * a.C + c] = sb;
}

__global__ void __launch_bounds__(256) ln_sum_kernel(NormArgs a, int64_t nparts) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.C) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t p = 0; p < nparts; ++p) {
        sw += a.part[p * a.C + c];
        sb += a.part[(nparts + p) * a.C + c];
    }
    if (a.dweight) a.dweight[c] = sw;
    if (a.dbias) a.dbias[c] = sb;
}

template <typename F> hipError_t by_dtype(int dtype, F&& f) {
    if (dtype == LCONV_F32) f(std::integral_constant<int, CT_F32>{});
    else if (dtype == LCONV_F16) f(std::integral_constant<int, CT_F16>{});
    else f(std::integral_constant<int, CT_BF16>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layernorm_fwd(int dtype, const NormArgs& a, hipStream_t stream) {
    return by_dtype(dtype, [&](auto io) { ln_fwd_kernel<io.value><<<(unsigned)a.rows, 256, 0, stream>>>(a); });
}

hipError_t launch_layernorm_bwd(int dtype, const NormArgs& a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.dweight || a.dbias) {
        const int64_t np = layernorm_parts(a.rows, a.C);
        const unsigned gx = (unsigned)((a.C + 255) / 256);
        if (np > 0) {
            e = by_dtype(dtype, [&](auto io) { ln_part_kernel<io.value><<<dim3(gx, (unsigned)np), 256, 0, stream>>>(a, np); });
            if (e != hipSuccess) return e;
        }
        ln_sum_kernel<<<gx, 256, 0, stream>>>(a, np);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.rows > 0) e = by_dtype(dtype, [&](auto io) { ln_dx_kernel<io.value><<<(unsigned)a.rows, 256, 0, stream>>>(a); });
    return e;
}

}  // namespace lcv
