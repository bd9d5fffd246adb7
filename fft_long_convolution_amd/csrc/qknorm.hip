// qknorm.hip -- norms of q and k for each head, with their rotary positions in the same pass, and the gradients.
//
//   u = x (centred: x - mean),  r = 1 / sqrt(mean(u^2) + eps),  y = turn(r u w)
//   n = turn^-1(dy), h = n w:  dx = r (h - u r^2 mean(h u)) (centred: less its mean),  dw = sum n r u
// One read and one write of q and k (gradients: two reads, one write), bound by HBM.  A head's row lives in the registers of
// up to 64 lanes, two groups of 8 elements each, laid out as the pairs that turn together, so that sums cross lanes and
// turns do not.  A group of lanes takes one token of up to four heads: they share the sines, and the next head's loads are on
// their way.
#include "block_kernels.h"
#include "mixer_io.h"
#include "rotary_turn.h"

namespace lcv {
namespace {

template <int LANES> __device__ __forceinline__ void lane_sums(float& a, float& b) {
#pragma unroll
    for (int w = LANES / 2; w; w >>= 1) {
        a += __shfl_xor(a, w);
        b += __shfl_xor(b, w);
    }
}

// the unit of a head that a lane has: its two groups of 8 elements (interleaved pairs, and elements that do not turn: 16 in a
// row) and how many of each there are
struct Unit {
    bool turn;
    int p, n, lo, hi, nlo, nhi;
};
__device__ __forceinline__ Unit unit_of(const QkArgs& a, int u, int turns, int units) {
    Unit t;
    const int half = a.rot / 2;
    const bool inter = a.flags & LCONV_ROTARY_INTERLEAVED;
    t.turn = u < turns;
    t.p = 8 * u;
    t.n = !t.turn ? 0 : half - t.p < 8 ? half - t.p : 8;
    t.lo = !t.turn ? a.rot + 16 * (u - turns) : inter ? 2 * t.p : t.p;
    t.hi = !t.turn || inter ? t.lo + 8 : half + t.p;
    t.nlo = !t.turn ? a.D - t.lo : inter ? 2 * t.n : t.n;
    t.nhi = !t.turn ? a.D - t.hi : inter ? 2 * t.n - 8 : t.n;
    if (u >= units) t.lo = t.hi = t.nlo = t.nhi = 0;       // a lane past the head
    return t;
}

template <int IO> struct Head { Raw8<IO> lo, hi; };
template <int IO> __device__ __forceinline__ Head<IO> load_head(const void* p, int64_t at, const Unit& t) {
    return Head<IO>{raw8_part<IO>(p, at + t.lo, t.nlo), raw8_part<IO>(p, at + t.hi, t.nhi)};
}
template <int IO> __device__ __forceinline__ void widen(const Head<IO>& h, float* x) {
    unpack_raw<IO>(h.lo.w, x);
    unpack_raw<IO>(h.hi.w, x + 8);
}

// pairs by their sines (s negated: back)
__device__ __forceinline__ void turn_pairs(float* v, const float* c, const float* s, float sign, bool inter) {
    if (inter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = v[2 * e], y = v[2 * e + 1];
            v[2 * e] = x * c[e] - y * (sign * s[e]);
            v[2 * e + 1] = y * c[e] + x * (sign * s[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = v[e], y = v[e + 8];
            v[e] = x * c[e] - y * (sign * s[e]);
            v[e + 8] = y * c[e] + x * (sign * s[e]);
        }
    }
}

__device__ __forceinline__ void token_sines(const QkArgs& a, const Unit& t, int64_t b, int64_t n, float* c, float* s) {
    const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + n] : n;
    float f[8];
    load8_part<CT_F32>(a.inv_freq, t.p, t.n, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        sines((double)pos * (double)f[k], &s[k], &c[k]);
        c[k] *= a.magnitude;
        s[k] *= a.magnitude;
    }
}

// how many of a lane's 16 elements are the head's, by index
__device__ __forceinline__ bool has(const Unit& t, int e) { return e < 8 ? e < t.nlo : e - 8 < t.nhi; }

// u = x (centred: less its mean) in place; returns r.  The mean takes two sums: what the first one's rounding leaves shows in the
// sum of the centred values.
template <int LANES, bool CENTRED> __device__ __forceinline__ float normed(float* x, const Unit& t, int D, float eps) {
    const float inv = 1.f / (float)D;
    float s = 0.f, q = 0.f;
    if constexpr (CENTRED) {
        float none = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s += x[e];
        lane_sums<LANES>(s, none);
        const float first = s * inv;
        s = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e] = has(t, e) ? x[e] - first : 0.f;
            s += x[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) q += x[e] * x[e];
    lane_sums<LANES>(s, q);
    float var = q * inv;
    if constexpr (CENTRED) {
        const float rest = s * inv;
        var -= rest * rest;
        var = var < 0.f ? 0.f : var;       // rounding; a NaN stays one
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = has(t, e) ? x[e] - rest : 0.f;
    }
    return 1.f / sqrtf(var + eps);
}

template <int IO> __device__ __forceinline__ void load_weights(const QkArgs& a, const Unit& t, float (*w)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (a.w[i]) {
            widen<IO>(load_head<IO>(a.w[i], 0, t), w[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[i][e] = 1.f;
        }
    }
}

template <int IO, int LANES, bool CENTRED>
__global__ void __launch_bounds__(256) qknorm_fwd_kernel(QkArgs a, QkPlan p) {
    const int64_t g = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
    const bool any = g < p.items;                       // lanes of a group go together; a group past the last does as the first
    const uint32_t item = (uint32_t)(any ? g : 0), row = item / (uint32_t)p.hgroups, hg = item - row * (uint32_t)p.hgroups;
    const int64_t b = row / (uint64_t)a.N, n = row - b * a.N;
    const bool inter = a.flags & LCONV_ROTARY_INTERLEAVED;
    const Unit t = unit_of(a, threadIdx.x % LANES, p.turns, p.units);
    const int h0 = (int)hg * p.per, all = a.heads[0] + a.heads[1], end = h0 + p.per < all ? h0 + p.per : all;
    const auto load = [&](int h) LCV_INLINE {
        const int i = h >= a.heads[0];
        return load_head<IO>(a.x[i], b * a.xs[i].b + (int64_t)(i ? h - a.heads[0] : h) * a.xs[i].h + n * a.xs[i].n, t);
    };
    Head<IO> next = load(h0);
    float w[2][16], c[8], s[8];
    load_weights<IO>(a, t, w);
    if (t.turn) token_sines(a, t, b, n, c, s);
    for (int h = h0; h < end; ++h) {
        const Head<IO> now = next;
        if (h + 1 < end) next = load(h + 1);
        const int i = h >= a.heads[0];
        float x[16];
        widen<IO>(now, x);
        const float r = normed<LANES, CENTRED>(x, t, a.D, a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= r * (i ? w[1][e] : w[0][e]);
        if (t.turn) turn_pairs(x, c, s, 1.f, inter);
        if (any) {
            const int64_t at = b * a.ys[i].b + (int64_t)(i ? h - a.heads[0] : h) * a.ys[i].h + n * a.ys[i].n;
            store8_part<IO>(a.y[i], at + t.lo, t.nlo, x);
            store8_part<IO>(a.y[i], at + t.hi, t.nhi, x + 8);
        }
    }
}

template <int IO, int LANES, bool CENTRED>
__global__ void __launch_bounds__(256) qknorm_bwd_kernel(QkArgs a, QkPlan p) {
    constexpr int GROUPS = 256 / LANES;
    const bool inter = a.flags & LCONV_ROTARY_INTERLEAVED;
    const int lane = threadIdx.x % LANES, all = a.heads[0] + a.heads[1];
    const Unit t = unit_of(a, lane, p.turns, p.units);
    const float inv = 1.f / (float)a.D;
    float w[2][16], sum[2][16] = {};
    load_weights<IO>(a, t, w);
    for (int64_t g0 = (int64_t)blockIdx.x * GROUPS; g0 < p.items; g0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t g = g0 + threadIdx.x / LANES;
        const bool any = g < p.items;
        const uint32_t item = (uint32_t)(any ? g : 0), row = item / (uint32_t)p.hgroups, hg = item - row * (uint32_t)p.hgroups;
        const int64_t b = row / (uint64_t)a.N, n = row - b * a.N;
        const int h0 = (int)hg * p.per, end = h0 + p.per < all ? h0 + p.per : all;
        Head<IO> nx, nd;
        const auto load = [&](int h) LCV_INLINE {
            const int i = h >= a.heads[0];
            const int64_t hh = i ? h - a.heads[0] : h;
            nx = load_head<IO>(a.x[i], b * a.xs[i].b + hh * a.xs[i].h + n * a.xs[i].n, t);
            nd = load_head<IO>(a.dy[i], b * a.dys[i].b + hh * a.dys[i].h + n * a.dys[i].n, t);
        };
        load(h0);
        float c[8], s[8];
        if (t.turn) token_sines(a, t, b, n, c, s);
        for (int h = h0; h < end; ++h) {
            float u[16], d[16];
            widen<IO>(nx, u);
            widen<IO>(nd, d);
            if (h + 1 < end) load(h + 1);
            const int i = h >= a.heads[0];
            const float r = normed<LANES, CENTRED>(u, t, a.D, a.eps);
            if (t.turn) turn_pairs(d, c, s, -1.f, inter);
            float hu = 0.f, hs = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                u[e] *= r;
                const float term = any ? d[e] * u[e] : 0.f;
                sum[0][e] += i ? 0.f : term;
                sum[1][e] += i ? term : 0.f;
                d[e] *= i ? w[1][e] : w[0][e];
                hu += d[e] * u[e];
                if constexpr (CENTRED) hs += has(t, e) ? d[e] : 0.f;
            }
            lane_sums<LANES>(hu, hs);
            hu *= inv;
            hs *= inv;
#pragma unroll
            for (int e = 0; e < 16; ++e) d[e] = r * (d[e] - u[e] * hu - (CENTRED ? hs : 0.f));
            if (any) {
                const int64_t at = b * a.ys[i].b + (int64_t)(i ? h - a.heads[0] : h) * a.ys[i].h + n * a.ys[i].n;
                store8_part<IO>(a.y[i], at + t.lo, t.nlo, d);
                store8_part<IO>(a.y[i], at + t.hi, t.nhi, d + 8);
            }
        }
    }
    if (!a.part) return;
    // the groups of a wave join by lanes, the waves through LDS, in a fixed order
    __shared__ float join[4][2][16][LANES];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
#pragma unroll
            for (int k = LANES; k < 64; k *= 2) sum[i][e] += __shfl_xor(sum[i][e], k);
            if ((threadIdx.x & 63) < LANES) join[threadIdx.x >> 6][i][e][lane] = sum[i][e];
        }
    __syncthreads();
    if (threadIdx.x >= LANES) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[i][e] = (join[0][i][e][lane] + join[1][i][e][lane]) + (join[2][i][e][lane] + join[3][i][e][lane]);
        const int64_t at = ((int64_t)blockIdx.x * 2 + i) * a.D;
        store8_part<CT_F32>(a.part, at + t.lo, t.nlo, sum[i]);
        store8_part<CT_F32>(a.part, at + t.hi, t.nhi, sum[i] + 8);
    }
}

// The weights' gradients from the workgroups' sums: a workgroup takes 32 columns of q or k, its 8 groups of lanes every eighth
// part, and joins the groups in order.
__global__ void __launch_bounds__(256) qknorm_sum_kernel(const float* part, float* dq, float* dk, int parts, int D) {
    __shared__ float join[8][32];
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + l, i = blockIdx.y;
    float u = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int k = q; k < parts; k += 8) u += part[((int64_t)k * 2 + i) * D + c];
    }
    join[q][l] = u;
    __syncthreads();
    float* out = i ? dk : dq;
    if (q || c >= D || !out) return;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += join[k][l];
    out[c] = s;
}

template <typename F> void by_lanes(int lanes, F&& f) {
    using std::integral_constant;
    if (lanes <= 1) f(integral_constant<int, 1>{});
    else if (lanes == 2) f(integral_constant<int, 2>{});
    else if (lanes == 4) f(integral_constant<int, 4>{});
    else if (lanes == 8) f(integral_constant<int, 8>{});
    else if (lanes == 16) f(integral_constant<int, 16>{});
    else if (lanes == 32) f(integral_constant<int, 32>{});
    else f(integral_constant<int, 64>{});
}
template <typename F> hipError_t by_dtype(int dtype, F&& f) {
    if (dtype == LCONV_F32) f(std::integral_constant<int, CT_F32>{});
    else if (dtype == LCONV_F16) f(std::integral_constant<int, CT_F16>{});
    else f(std::integral_constant<int, CT_BF16>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qknorm_fwd(int dtype, const QkArgs& a, hipStream_t stream) {
    const QkPlan p = qk_plan(a.B * a.N, a.D, a.rot, a.heads[0] + a.heads[1]);
    const unsigned grid = (unsigned)((p.items * p.lanes + 255) / 256);
    return by_dtype(dtype, [&](auto io) {
        by_lanes(p.lanes, [&](auto lanes) {
            if (a.flags & LCONV_QKNORM_CENTRED) qknorm_fwd_kernel<io.value, lanes.value, true><<<grid, 256, 0, stream>>>(a, p);
            else qknorm_fwd_kernel<io.value, lanes.value, false><<<grid, 256, 0, stream>>>(a, p);
        });
    });
}

hipError_t launch_qknorm_bwd(int dtype, const QkArgs& a, hipStream_t stream) {
    const int64_t tokens = a.B * a.N;
    int parts = 0;
    hipError_t e = hipSuccess;
    if (tokens > 0) {
        const QkPlan p = qk_plan(tokens, a.D, a.rot, a.heads[0] + a.heads[1]);
        parts = (int)qk_parts(p);
        e = by_dtype(dtype, [&](auto io) {
            by_lanes(p.lanes, [&](auto lanes) {
                if (a.flags & LCONV_QKNORM_CENTRED) qknorm_bwd_kernel<io.value, lanes.value, true><<<parts, 256, 0, stream>>>(a, p);
                else qknorm_bwd_kernel<io.value, lanes.value, false><<<parts, 256, 0, stream>>>(a, p);
            });
        });
    }
    if (e != hipSuccess || (!a.dw[0] && !a.dw[1])) return e;
    qknorm_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32), 2), 256, 0, stream>>>(a.part, a.dw[0], a.dw[1], parts, a.D);
    return hipGetLastError();
}

}  // namespace lcv
