// shortconv.hip -- the short causal convolution along tokens: forward, gradients, single tokens.
//
//   p_t = b + sum_{j<K} w_j x_{t-K+1+j},  y = p or p sigmoid(p)
//   dp = dy (p' = 1 or sigmoid(p) (1 + p (1 - sigmoid(p)))),  dx_s = sum_j w_j dp_{s+K-1-j},  dw_j = sum dp_t x_{t-K+1+j}
// K is at most 8: one read of x and one write of y (gradients: two reads, one write), bound by HBM.  A wave takes 64 to 256
// channels of a run of tokens, a lane one or four of them, with the last K inputs and the weights in its registers; the K - 1
// inputs before a run are read again, through the caches.  A token is the same for a whole wave, so lengths and ends cost
// scalar instructions only.  Measured at 8 x 2048 x 4096, K = 4, SiLU, bf16: 48 us forward (268 MB, 5.6 TB/s in a row of calls, part
// of it from the caches; 52 with other inputs each call) and 96 for the gradients and their sum (403 MB at 4.4 TB/s without the sum's
// 5 us; 32 vector instructions to a token and channel are 55 us of issue); in fp32 116 (537 MB, 4.6 TB/s) and 175 (805 MB, 4.7).
#include "block_kernels.h"
#include "token_io.h"

namespace lcv {
namespace {

constexpr int kBatch = 8, kGradBatch = 4;      // tokens whose loads are on their way together

template <int V> struct Lane {
    float v[V];
};

// where a wave works: row b, tokens t0 .. t1, of them len in the row; channels c .. of a lane (past the last: those of the last
// lane that has some, with the same results at the same places)
struct Run {
    int64_t b, t0, t1, len;
    bool first;
};
__device__ __forceinline__ Run run_of(const ConvArgs& a, uint32_t i) {
    Run r;
    const uint32_t b = i / (uint32_t)a.runs, k = i - b * (uint32_t)a.runs;
    r.b = b;
    r.t0 = k * a.run;
    r.t1 = r.t0 + a.run < a.N ? r.t0 + a.run : a.N;
    r.len = row_len(a.lengths, r.b, a.N);
    r.first = k == 0;
    return r;
}
// workgroups with the same tokens lie side by side
template <int V> __device__ __forceinline__ uint32_t channel_of(const ConvArgs& a, uint32_t* group) {
    *group = blockIdx.x / (uint32_t)a.cgroups;
    const int64_t c = ((int64_t)(blockIdx.x - *group * (uint32_t)a.cgroups) * 64 + (threadIdx.x & 63)) * V;
    return (uint32_t)(c < a.C - V ? c : a.C - V);
}

// x of token t, which may lie before the row's first; zero at and behind its end
template <int IO, int V, int K>
__device__ __forceinline__ Lane<V> input(const ConvArgs& a, const Run& r, int64_t t, uint32_t c) {
    Lane<V> x{};
    if (t >= r.len) return x;
    if (t >= 0) widen<IO, V>(load_raw_v<IO, V>(a.x.p, r.b * a.x.b + t * a.x.n, c), x.v);
    else if (a.state_in) widen<IO, V>(load_raw_v<IO, V>(a.state_in, (r.b * (K - 1) + t + K - 1) * a.C, c), x.v);
    return x;
}

template <int IO, int V, int K> struct Taps {
    float w[K][V], b[V];
    __device__ __forceinline__ Taps(const void* w_, const void* bias, uint32_t c) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][v] = load1<IO>(w_, (int64_t)(c + v) * K + j);
            b[v] = bias ? load1<IO>(bias, c + v) : 0.f;
        }
    }
};

template <int IO, int V, int K> __global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs a) {
    uint32_t group;
    const uint32_t c = channel_of<V>(a, &group), i = group * 4 + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= a.B * a.runs) return;
    const Run r = run_of(a, i);
    const Taps<IO, V, K> taps(a.w, a.bias, c);
    Lane<V> win[K];                      // win[j] = x_{t-K+1+j}
#pragma unroll
    for (int j = 0; j < K - 1; ++j) win[j + 1] = input<IO, V, K>(a, r, r.t0 - (K - 1) + j, c);
    if (a.state_out && r.first) {
        Lane<V> s[K];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s[j] = input<IO, V, K>(a, r, r.len - (K - 1) + j, c);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) store_v<IO, V>(a.state_out, (r.b * (K - 1) + j) * a.C, c, s[j].v);
    }
    const int64_t xr = r.b * a.x.b, yr = r.b * a.yb;
    const int64_t end = r.t1 < r.len ? r.t1 : r.len;
    RawV<IO, V> next[kBatch], now[kBatch];
    const auto load = [&](int64_t t) LCV_INLINE {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) next[k] = load_raw_v<IO, V>(a.x.p, xr + (t + k < end ? t + k : end - 1) * a.x.n, c);
    };
    int64_t t = r.t0;
    if (t < end) load(t);
    for (; t < end; t += kBatch) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) now[k] = next[k];
        load(t + kBatch);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) win[j] = win[j + 1];
            widen<IO, V>(now[k], win[K - 1].v);
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p = taps.b[v];
#pragma unroll
                for (int j = 0; j < K; ++j) p = fmaf(taps.w[j][v], win[j].v[v], p);
                y[v] = a.silu ? p * sigmoid(p) : p;
            }
            if (t + k < end) store_v<IO, V>(a.y, yr + (t + k) * a.yn, c, y);
        }
    }
    const float zero[V] = {};
    for (t = end > r.t0 ? end : r.t0; t < r.t1; ++t) store_v<IO, V>(a.y, yr + t * a.yn, c, zero);
}

template <int IO, int V, int K> __global__ void __launch_bounds__(256) conv_bwd_kernel(ConvArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    uint32_t group;
    const uint32_t c = channel_of<V>(a, &group);
    const Taps<IO, V, K> taps(a.w, a.bias, c);
    float dw[K][V] = {}, db[V] = {};
    const uint32_t total = (uint32_t)(a.B * a.runs);
    for (uint32_t i = group * 4 + wave; i < total; i += (uint32_t)a.groups * 4) {
        const Run r = run_of(a, i);
        const int64_t xr = r.b * a.x.b, dr = r.b * a.dy.b;
        const int64_t mine = r.t1 < r.len ? r.t1 : r.len, last = (r.t1 + K - 1 < r.len ? r.t1 + K - 1 : r.len) - 1;
        Lane<V> win[K], acc[K];          // acc[j] = dx of token t-K+1+j, what the tokens up to t add
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j + 1] = input<IO, V, K>(a, r, r.t0 - (K - 1) + j, c);
#pragma unroll
        for (int j = 0; j < K; ++j) acc[j] = Lane<V>{};
        RawV<IO, V> nx[kGradBatch], nd[kGradBatch], x[kGradBatch], d[kGradBatch];
        const auto load = [&](int64_t t) LCV_INLINE {
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) {
                const int64_t at = t + k <= last ? t + k : last;
                nx[k] = load_raw_v<IO, V>(a.x.p, xr + at * a.x.n, c);
                nd[k] = load_raw_v<IO, V>(a.dy.p, dr + at * a.dy.n, c);
            }
        };
        // INNER: tokens of this run and of the row
        const auto batch = [&](int64_t t0, auto inner) LCV_INLINE {
            constexpr bool INNER = decltype(inner)::value;
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) x[k] = nx[k], d[k] = nd[k];
            if (INNER || r.len > 0) load(t0 + kGradBatch);
#pragma unroll
            for (int k = 0; k < kGradBatch; ++k) {
                const int64_t t = t0 + k, s = t - (K - 1);
                const bool on = INNER || t < r.len, own = INNER || t < mine;
                float xv[V], dv[V];
                widen<IO, V>(x[k], xv);
                widen<IO, V>(d[k], dv);
#pragma unroll
                for (int j = 0; j < K - 1; ++j) win[j] = win[j + 1], acc[j] = acc[j + 1];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[K - 1].v[v] = on ? xv[v] : 0.f;
                    if (a.silu) {
                        float p = taps.b[v];
#pragma unroll
                        for (int j = 0; j < K; ++j) p = fmaf(taps.w[j][v], win[j].v[v], p);
                        // s (1 + p (1 - s)), 1 - s = e s to its own size (where e is cut off, s is too small for the reciprocal and zero)
                        const float e = fast_exp2(-kLog2e * p), sig = fast_rcp(1.f + e);
                        dv[v] *= sig * fmaf(p, fminf(e, 0x1p126f) * sig, 1.f);
                    }
                }
                // what the row does not have is left out, not multiplied by zero: an input or a weight may be no number
                acc[K - 1] = Lane<V>{};
                if (on) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int j = 0; j < K; ++j) acc[j].v[v] = fmaf(taps.w[j][v], dv[v], acc[j].v[v]);
                }
                if (own) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += dv[v];
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][v] = fmaf(dv[v], win[j].v[v], dw[j][v]);
                    }
                }
                // dx of token s is complete
                if (s >= r.t0 ? s < r.t1 : (r.first && a.state_out && s >= -(K - 1))) {
                    if (a.dstate_out && s >= r.len - (K - 1) && s < r.len) {
                        float more[V];
                        widen<IO, V>(load_raw_v<IO, V>(a.dstate_out, (r.b * (K - 1) + s - r.len + K - 1) * a.C, c), more);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[0].v[v] += more[v];
                    }
                    if (s >= 0) store_v<IO, V>(a.y, r.b * a.yb + s * a.yn, c, acc[0].v);
                    else store_v<IO, V>(a.state_out, (r.b * (K - 1) + s + K - 1) * a.C, c, acc[0].v);
                }
            }
        };
        if (r.len > 0) load(r.t0);
        int64_t t0 = r.t0;
        for (; t0 + kGradBatch <= mine; t0 += kGradBatch) batch(t0, std::true_type{});
        for (; t0 < r.t1 + K - 1; t0 += kGradBatch) batch(t0, std::false_type{});
    }
    if (!a.part) return;
    // the waves join through LDS, in their order
    __shared__ float join[4][K + 1][V][64];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K; ++j) join[wave][j][v][lane] = dw[j][v];
        join[wave][K][v][lane] = db[v];
    }
    __syncthreads();
    if (wave) return;
    for (int j = 0; j <= K; ++j) {
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = (join[0][j][v][lane] + join[1][j][v][lane]) + (join[2][j][v][lane] + join[3][j][v][lane]);
        __builtin_memcpy(a.part + ((int64_t)group * (K + 1) + j) * a.C + c, s, sizeof(s));
    }
}

// The weights' gradients from the workgroups' sums: a workgroup takes 32 channels of a tap (or the bias), its 8 groups of lanes
// every eighth part, and joins the groups in order.
__global__ void __launch_bounds__(256) conv_sum_kernel(const float* part, float* dw, float* db, int parts, int K, int64_t C) {
    __shared__ float join[8][32];
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5, j = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * 32 + l;
    float u = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int k = q; k < parts; k += 8) u += part[((int64_t)k * (K + 1) + j) * C + c];
    }
    join[q][l] = u;
    __syncthreads();
    if (q || c >= C) return;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += join[k][l];
    if (j < K && dw) dw[c * K + j] = s;
    if (j == K && db) db[c] = s;
}

// One token: the window is the pool's K - 1 inputs and x; they move on by one in place.  Latency for few rows (64 x 2048, K = 4, in
// bf16: 3.3 us), HBM for many.
template <int IO, int V, int K> __global__ void __launch_bounds__(256) conv_step_kernel(ConvStepArgs a) {
    const int64_t per = a.C / V, i = (int64_t)blockIdx.x * 256 + threadIdx.x, b = i / per;
    const uint32_t c = (uint32_t)(i - b * per) * V;
    if (b >= a.B) return;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    float y[V] = {};
    if (slot >= 0 && slot < a.nslots) {
        RawV<IO, V> win[K];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j] = load_raw_v<IO, V>(a.state, (slot * (K - 1) + j) * a.C, c);
        win[K - 1] = load_raw_v<IO, V>(a.x.p, b * a.x.b, c);
        const Taps<IO, V, K> taps(a.w, a.bias, c);
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = taps.b[v];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float x[V];
            widen<IO, V>(win[j], x);
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = fmaf(taps.w[j][v], x[v], y[v]);
        }
        if (a.silu) {
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] *= sigmoid(y[v]);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            __builtin_memcpy((typename Elem<IO>::T*)a.state + (slot * (K - 1) + j) * a.C + c, &win[j + 1], sizeof(win[0]));
    }
    store_v<IO, V>(a.y, b * a.yb, c, y);
}

template <typename T> __global__ void __launch_bounds__(256) conv_state_kernel(const T* in, T* out, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) out[i] = in ? in[i] : (T)0;
}

template <typename F> hipError_t by_dtype(int dtype, F&& f) {
    if (dtype == LCONV_F32) f(std::integral_constant<int, CT_F32>{});
    else if (dtype == LCONV_F16) f(std::integral_constant<int, CT_F16>{});
    else f(std::integral_constant<int, CT_BF16>{});
    return hipGetLastError();
}
template <typename F> void by_taps(int K, int vec, F&& f) {
    using std::integral_constant;
    const auto go = [&](auto k) {
        if (vec == 4) f(integral_constant<int, 4>{}, k);
        else f(integral_constant<int, 1>{}, k);
    };
    switch (K) {
        case 2: return go(integral_constant<int, 2>{});
        case 3: return go(integral_constant<int, 3>{});
        case 4: return go(integral_constant<int, 4>{});
        case 5: return go(integral_constant<int, 5>{});
        case 6: return go(integral_constant<int, 6>{});
        case 7: return go(integral_constant<int, 7>{});
        default: return go(integral_constant<int, 8>{});
    }
}

}  // namespace

hipError_t launch_conv_fwd(int dtype, const ConvArgs& a, hipStream_t stream) {
    return by_dtype(dtype, [&](auto io) {
        by_taps(a.K, a.vec, [&](auto v, auto k) {
            conv_fwd_kernel<io.value, v.value, k.value><<<(unsigned)a.cgroups * (unsigned)a.groups, 256, 0, stream>>>(a);
        });
    });
}

hipError_t launch_conv_bwd(int dtype, const ConvArgs& a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.groups > 0)
        e = by_dtype(dtype, [&](auto io) {
            by_taps(a.K, a.vec, [&](auto v, auto k) {
                conv_bwd_kernel<io.value, v.value, k.value><<<(unsigned)a.cgroups * (unsigned)a.groups, 256, 0, stream>>>(a);
            });
        });
    if (e != hipSuccess || (!a.dw && !a.db)) return e;
    conv_sum_kernel<<<dim3((unsigned)((a.C + 31) / 32), a.K + 1), 256, 0, stream>>>(a.part, a.dw, a.db, a.groups, a.K, a.C);
    return hipGetLastError();
}

hipError_t launch_conv_step(int dtype, const ConvStepArgs& a, hipStream_t stream) {
    return by_dtype(dtype, [&](auto io) {
        by_taps(a.K, a.C % 4 == 0 ? 4 : 1, [&](auto v, auto k) {
            const unsigned grid = (unsigned)((a.B * (a.C / v.value) + 255) / 256);
            conv_step_kernel<io.value, v.value, k.value><<<grid, 256, 0, stream>>>(a);
        });
    });
}

hipError_t launch_conv_state(int dtype, const void* in, void* out, int64_t n, hipStream_t stream) {
    const int64_t g = (n + 255) / 256;
    const unsigned grid = (unsigned)(g < 8192 ? g : 8192);
    if (dtype == LCONV_F32) conv_state_kernel<<<grid, 256, 0, stream>>>((const uint32_t*)in, (uint32_t*)out, n);
    else conv_state_kernel<<<grid, 256, 0, stream>>>((const uint16_t*)in, (uint16_t*)out, n);
    return hipGetLastError();
}

}  // namespace lcv
