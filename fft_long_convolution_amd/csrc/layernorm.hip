// layernorm.hip -- layer norm: forward, and the gradients of its input, weight and bias.
//
//   y = (x - mean) rstd w + b;   with xhat = (x - mean) rstd and h = dy w:
//   dx = rstd (h - mean_C(h) - xhat mean_C(h xhat)),  dw = sum_rows dy xhat,  db = sum_rows dy
// Both are bound by HBM: x (and dy) are read once, y (dx) written once.  A row lives in the registers of
// LANES lanes of one wave (C <= 1024) or of several (C <= 8192), 8-element groups dealt out in
// turn, so the sums need no second read; longer rows are read again through the caches.  Waves walk the
// rows with the weight (and, in the gradient, the column sums of their rows) held in registers.
// Measured, 16384 rows of 4096 in bf16: forward 52 us (5.2 TB/s, what a copy reaches), gradient 83 us (4.8 TB/s with the
// workgroups' column sums) and 7 us for their sum; 333 rows of 1001 in fp32: 5.2, 7.5 and 3.2 us (latency).
//
// The mean takes two sums: the first is off by the rounding of adding up the values themselves, what is
// left of it shows in the sum of the centred values and is taken out of mean and variance.
#include "mixer_kernels.h"
#include "mixer_io.h"
#include "mixer_plan.h"

namespace lcv {
namespace {

// Two sums over a row's lanes.  Rows of several waves join through red, which two sums in a row must not share: then one
// barrier is enough, since the next one is passed only once every wave has read.
template <int LANES> struct RowRed { float v[2][2][LANES > 64 ? (LANES < 256 ? 256 : LANES) / 64 : 1]; };   // by wave of the workgroup
template <int LANES> __device__ __forceinline__ void row_sums(float& a, float& b, RowRed<LANES>& red, int which) {
    constexpr int W = LANES < 64 ? LANES : 64;
#pragma unroll
    for (int w = W / 2; w; w >>= 1) {
        a += __shfl_xor(a, w);
        b += __shfl_xor(b, w);
    }
    if constexpr (LANES > 64) {
        constexpr int N = LANES / 64;
        const int wave = threadIdx.x >> 6, first = wave / N * N;     // of the row
        float *const f = red.v[which][0], *const e = red.v[which][1];
        if ((threadIdx.x & 63) == 0) {
            f[wave] = a;
            e[wave] = b;
        }
        __syncthreads();
        a = f[first];
        b = e[first];
#pragma unroll
        for (int i = 1; i < N; ++i) {
            a += f[first + i];
            b += e[first + i];
        }
    }
}

// A variance below zero is rounding; a row with a NaN or an infinity has none, and its rstd is a NaN (fmaxf would make
// it 1 / sqrt(eps)).  Its mean is what the values add up to: an infinity leaves only NaNs to the centred sum.
__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps); }
__device__ __forceinline__ float mean_of(float first, float rest) { return rest == rest ? first + rest : first; }

// raw 8-element groups of a row: group k of lane l is elements 8 (l + LANES k) ..
template <int IO> struct Group { uint4 r[IO == CT_F32 ? 2 : 1]; };
template <int IO> __device__ __forceinline__ Group<IO> load_group(const void* p, int64_t row, int c, int C) {
    Group<IO> v;
    const typename Elem<IO>::T* q = (const typename Elem<IO>::T*)p + row + c;
    if (c + 8 <= C) {
        __builtin_memcpy(v.r, q, sizeof(v.r));
    } else {
        typename Elem<IO>::T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = c + i < C ? q[i] : (typename Elem<IO>::T)0;
        __builtin_memcpy(v.r, e, sizeof(v.r));
    }
    return v;
}

// elements of group c that the row has
__device__ __forceinline__ int left(int c, int C) { return C - c < 8 ? C - c : 8; }

template <int IO, int LANES, int K>
__global__ void __launch_bounds__(LANES < 256 ? 256 : LANES) ln_fwd_kernel(NormArgs a) {
    __shared__ RowRed<LANES> red;
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;      // rows a workgroup has in hand
    const int lane = threadIdx.x % LANES, C = (int)a.C;
    const float inv = 1.f / (float)C;
    Group<IO> w[K], b[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (lane + LANES * k);
        if (a.weight) w[k] = load_group<IO>(a.weight, 0, c, C);
        if (a.bias) b[k] = load_group<IO>(a.bias, 0, c, C);
    }
    // every lane of a wave takes part in each turn's sums: rows past the last compute on row 0's data
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = r0 + threadIdx.x / LANES;
        const bool on = row < a.rows;
        float x[K][8], s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = 8 * (lane + LANES * k);
            const Group<IO> g = load_group<IO>(a.x, (on ? row : 0) * a.xs, c, C);
            unpack_raw<IO>(g.r, x[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[k][i];
        }
        float none = 0.f, s1 = 0.f, s2 = 0.f;
        row_sums<LANES>(s, none, red, 0);
        const float first = s * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int n = left(8 * (lane + LANES * k), C);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[k][i] = i < n ? x[k][i] - first : 0.f;
                s1 += x[k][i];
                s2 += x[k][i] * x[k][i];
            }
        }
        row_sums<LANES>(s1, s2, red, 1);
        const float rest = s1 * inv, rstd = rstd_of(s2 * inv - rest * rest, a.eps);
        if (!on) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = 8 * (lane + LANES * k);
            if (c >= C) continue;
            float y[8], p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = (x[k][i] - rest) * rstd;
            if (a.weight) {
                unpack_raw<IO>(w[k].r, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= p[i];
            }
            if (a.bias) {
                unpack_raw<IO>(b[k].r, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] += p[i];
            }
            store8_part<IO>(a.y, row * a.ys + c, left(c, C), y);
        }
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean_of(first, rest);
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Rows too long for registers: three passes through the caches, one workgroup to a row.
template <int IO>
__global__ void __launch_bounds__(256) ln_fwd_long_kernel(NormArgs a) {
    __shared__ RowRed<256> red;
    const int C = (int)a.C;
    const float inv = 1.f / (float)C;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t xo = row * a.xs;
        float s = 0.f, x[8], p[8];
        for (int c = 8 * threadIdx.x; c < C; c += 2048) {
            load8_part<IO>(a.x, xo + c, left(c, C), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[i];
        }
        float none = 0.f, s1 = 0.f, s2 = 0.f;
        row_sums<256>(s, none, red, 0);
        const float first = s * inv;
        for (int c = 8 * threadIdx.x; c < C; c += 2048) {
            const int n = left(c, C);
            load8_part<IO>(a.x, xo + c, n, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i < n ? x[i] - first : 0.f;
                s1 += d;
                s2 += d * d;
            }
        }
        row_sums<256>(s1, s2, red, 1);
        const float rest = s1 * inv, rstd = rstd_of(s2 * inv - rest * rest, a.eps);
        for (int c = 8 * threadIdx.x; c < C; c += 2048) {
            const int n = left(c, C);
            load8_part<IO>(a.x, xo + c, n, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (x[i] - first - rest) * rstd;
            if (a.weight) {
                load8_part<IO>(a.weight, c, n, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= p[i];
            }
            if (a.bias) {
                load8_part<IO>(a.bias, c, n, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] += p[i];
            }
            store8_part<IO>(a.y, row * a.ys + c, n, x);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean_of(first, rest);
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// The gradient: dx of every row, and the column sums of the workgroup's rows to part[0 / 1][block][C], or, of a workgroup
// alone, to dweight and dbias.
// A row is read before it is written, so dx may stand in place of dy or x.
template <int IO, int LANES, int K>
__global__ void __launch_bounds__(LANES < 256 ? 256 : LANES) ln_bwd_kernel(NormArgs a) {
    __shared__ RowRed<LANES> red;
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;
    const int lane = threadIdx.x % LANES, C = (int)a.C;
    const float inv = 1.f / (float)C;
    const bool sums = a.dweight || a.dbias, alone = gridDim.x == 1;
    Group<IO> w[K];
    float sw[K][8], sb[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (a.weight) w[k] = load_group<IO>(a.weight, 0, 8 * (lane + LANES * k), C);
#pragma unroll
        for (int i = 0; i < 8; ++i) sw[k][i] = sb[k][i] = 0.f;
    }
    int which = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS, which ^= 1) {
        const int64_t row = r0 + threadIdx.x / LANES, at = row < a.rows ? row : 0;
        const bool on = row < a.rows;
        const float mean = a.mean[at], rstd = a.rstd[at];
        float xh[K][8], g[K][8], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = 8 * (lane + LANES * k), n = on ? left(c, C) : 0;
            const Group<IO> gx = load_group<IO>(a.x, at * a.xs, c, C), gg = load_group<IO>(a.dy, at * a.dys, c, C);
            unpack_raw<IO>(gx.r, xh[k]);
            unpack_raw<IO>(gg.r, g[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[k][i] = i < n ? (xh[k][i] - mean) * rstd : 0.f;
                if (i >= n) g[k][i] = 0.f;
                sw[k][i] += g[k][i] * xh[k][i];
                sb[k][i] += g[k][i];
            }
            if (a.weight) {
                float p[8];
                unpack_raw<IO>(w[k].r, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[k][i] *= p[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1 += g[k][i];
                s2 += g[k][i] * xh[k][i];
            }
        }
        row_sums<LANES>(s1, s2, red, which);
        s1 *= inv;
        s2 *= inv;
        if (!on) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = 8 * (lane + LANES * k);
            if (c >= C) continue;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rstd * (g[k][i] - s1 - xh[k][i] * s2);
            store8_part<IO>(a.y, row * a.ys + c, left(c, C), d);
        }
    }
    if (!sums) return;
    // the rows of one workgroup join through LDS, in the order of its row groups
    __shared__ float join[LANES < 256 ? 2 * 8 * 256 : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if constexpr (LANES < 256) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                join[i * 256 + threadIdx.x] = sw[k][i];
                join[(8 + i) * 256 + threadIdx.x] = sb[k][i];
            }
            __syncthreads();
            if (threadIdx.x < LANES) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float u = 0.f, v = 0.f;
#pragma unroll
                    for (int q = 0; q < ROWS; ++q) {
                        u += join[i * 256 + q * LANES + lane];
                        v += join[(8 + i) * 256 + q * LANES + lane];
                    }
                    sw[k][i] = u;
                    sb[k][i] = v;
                }
            }
        }
        const int c = 8 * (lane + LANES * k);
        if (threadIdx.x < LANES && c < C) {
            const int64_t o = (int64_t)blockIdx.x * C + c, nb = (int64_t)gridDim.x * C;
            float* const pw = alone ? a.dweight : a.part;
            float* const pb = alone ? a.dbias : a.part + nb;
            if (pw) store8_part<CT_F32>(pw, o, left(c, C), sw[k]);
            if (pb) store8_part<CT_F32>(pb, o, left(c, C), sb[k]);
        }
    }
}

template <int IO>
__global__ void __launch_bounds__(256) ln_dx_long_kernel(NormArgs a) {
    __shared__ RowRed<256> red;
    int which = 0;
    const int C = (int)a.C;
    const float inv = 1.f / (float)C;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, which ^= 1) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.f, s2 = 0.f, x[8], g[8], p[8];
        const auto load = [&](int c, int n) LCV_INLINE {
            load8_part<IO>(a.x, row * a.xs + c, n, x);
            load8_part<IO>(a.dy, row * a.dys + c, n, g);
            if (a.weight) {
                load8_part<IO>(a.weight, c, n, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] *= p[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = i < n ? (x[i] - mean) * rstd : 0.f;
        };
        for (int c = 8 * threadIdx.x; c < C; c += 2048) {
            load(c, left(c, C));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1 += g[i];
                s2 += g[i] * x[i];
            }
        }
        row_sums<256>(s1, s2, red, which);
        s1 *= inv;
        s2 *= inv;
        for (int c = 8 * threadIdx.x; c < C; c += 2048) {
            const int n = left(c, C);
            load(c, n);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = rstd * (g[i] - s1 - x[i] * s2);
            store8_part<IO>(a.y, row * a.ys + c, n, x);
        }
    }
}

// Column sums for rows too long for registers: block blockIdx.y takes every gridDim.y-th row.  It runs
// before the kernel above may write dx over dy or x.
template <int IO>
__global__ void __launch_bounds__(256) ln_part_long_kernel(NormArgs a) {
    const int c = 8 * (blockIdx.x * 256 + threadIdx.x), C = (int)a.C;
    if (c >= C) return;
    const int n = left(c, C);
    float sw[8] = {}, sb[8] = {}, x[8], g[8];
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        load8_part<IO>(a.x, row * a.xs + c, n, x);
        load8_part<IO>(a.dy, row * a.dys + c, n, g);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sw[i] += g[i] * ((x[i] - mean) * rstd);
            sb[i] += g[i];
        }
    }
    const int64_t o = (int64_t)blockIdx.y * C + c, nb = (int64_t)gridDim.y * C;
    store8_part<CT_F32>(a.part, o, n, sw);
    store8_part<CT_F32>(a.part, nb + o, n, sb);
}

// dweight and dbias from the blocks' partial sums: a workgroup takes 32 columns, its 8 groups of lanes
// every eighth block, and joins the groups in order.
__global__ void __launch_bounds__(256) ln_sum_kernel(const float* part, float* dweight, float* dbias, int np, int C) {
    __shared__ float join[2][8][32];
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
    float u = 0.f, v = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int p = q; p < np; p += 8) {
            u += part[(int64_t)p * C + c];
            v += part[(int64_t)(np + p) * C + c];
        }
    }
    join[0][q][l] = u;
    join[1][q][l] = v;
    __syncthreads();
    if (q > 1 || c >= C) return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += join[q][i][l];
    float* out = q ? dbias : dweight;
    if (out) out[c] = s;
}

template <typename F> hipError_t by_dtype(int dtype, F&& f) {
    if (dtype == LCONV_F32) f(std::integral_constant<int, CT_F32>{});
    else if (dtype == LCONV_F16) f(std::integral_constant<int, CT_F16>{});
    else f(std::integral_constant<int, CT_BF16>{});
    return hipGetLastError();
}

// f(lanes, groups per lane) for rows of C <= 8192: as few lanes as hold two groups each of the widest row, since every
// further wave adds a step to the sums.  Measured (bf16, us, forward / gradient): 65536 rows of 128, 16 lanes 10 / 21,
// 64 lanes 25 / 56; 32768 of 1024, 64 lanes 24 / 44, 128 lanes 26 / 44, 256 lanes 49 / 57; 16384 of 2048, 64 lanes with
// four groups 25 / 46 (of 1500: 27 / 56), 128 lanes 25 / 46 (28 / 51); 16384 of 4096, 256 lanes 47 / 89, 512 lanes 52 / 82;
// 8192 of 8192, 256 lanes with four groups 45 / 103, 512 lanes 47 / 90, read again through the caches 67 / 178.
template <bool GRAD, typename F> void by_width(int64_t C, F&& f) {
    const auto go = [&](auto lanes, auto k) { f(lanes, k); };
    using std::integral_constant;
    if (C <= 128) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (C <= 512) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (C <= 1024) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (C <= 2048) go(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    else if (C <= 4096) go(integral_constant<int, GRAD ? 512 : 256>{}, integral_constant<int, GRAD ? 1 : 2>{});
    else go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_layernorm_fwd(int dtype, const NormArgs& a, hipStream_t stream) {
    if (a.C > kNormRegisterC) {
        const unsigned grid = (unsigned)(a.rows < 4096 ? a.rows : 4096);
        return by_dtype(dtype, [&](auto io) { ln_fwd_long_kernel<io.value><<<grid, 256, 0, stream>>>(a); });
    }
    return by_dtype(dtype, [&](auto io) {
        by_width<false>(a.C, [&](auto lanes, auto k) {
            constexpr int threads = lanes.value < 256 ? 256 : lanes.value;
            const int64_t wgs = (a.rows + threads / lanes.value - 1) / (threads / lanes.value);
            const unsigned grid = (unsigned)(wgs < 2048 ? wgs : 2048);
            ln_fwd_kernel<io.value, lanes.value, k.value><<<grid, threads, 0, stream>>>(a);
        });
    });
}

hipError_t launch_layernorm_bwd(int dtype, const NormArgs& a, hipStream_t stream) {
    const bool sums = a.dweight || a.dbias;
    const int64_t np = a.rows > 0 ? layernorm_parts(a.rows, a.C) : 0;   // no rows: no partial sums to read
    hipError_t e = hipSuccess;
    if (a.rows > 0 && a.C <= kNormRegisterC) {
        e = by_dtype(dtype, [&](auto io) {
            by_width<true>(a.C, [&](auto lanes, auto k) {
                ln_bwd_kernel<io.value, lanes.value, k.value><<<(unsigned)np, lanes.value < 256 ? 256 : lanes.value, 0, stream>>>(a);
            });
        });
    } else if (a.rows > 0) {
        if (sums) {
            const unsigned gx = (unsigned)((a.C + 2047) / 2048);
            e = by_dtype(dtype, [&](auto io) { ln_part_long_kernel<io.value><<<dim3(gx, (unsigned)np), 256, 0, stream>>>(a); });
            if (e != hipSuccess) return e;
        }
        const unsigned grid = (unsigned)(a.rows < 4096 ? a.rows : 4096);
        e = by_dtype(dtype, [&](auto io) { ln_dx_long_kernel<io.value><<<grid, 256, 0, stream>>>(a); });
    }
    if (e != hipSuccess || !sums || (np == 1 && a.rows > 0 && a.C <= kNormRegisterC)) return e;
    ln_sum_kernel<<<(unsigned)((a.C + 31) / 32), 256, 0, stream>>>(a.part, a.dweight, a.dbias, (int)np, (int)a.C);
    return hipGetLastError();
}

}  // namespace lcv
