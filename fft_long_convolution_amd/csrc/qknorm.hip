// qknorm.hip -- norms of q and k for each head, with their rotary positions in the same pass, and the gradients.
//
//   u = x (centred: x - mean),  r = 1 / sqrt(mean(u^2) + eps),  y = turn(r u w)
//   n = turn^-1(dy), h = n w:  dx = r (h - u r^2 mean(h u)) (centred: less its mean),  dw = sum n r u
// One read and one write of q and k (gradients: two reads, one write), bound by HBM.  A head's row lives in the registers of
// up to 64 lanes, two groups of 8 elements each, laid out as the pairs that turn together, so that sums cross lanes and
// turns do not.  A group of lanes takes one token of up to four heads: they share the sines, and the next head's loads are on
// their way.  Measured (bf16, D = 128, 16 + 16 heads of 4 x 4096 tokens, other inputs each call): 55 us forward (268 MB, 4.9 TB/s;
// 47 where the call before has left its inputs in the cache), 83 for the gradients and their sums (403 MB, 4.9 TB/s); one token
// of 64 x (16 + 4) heads 4.2 us, a launch and the sines' arithmetic in 64 bits.
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
// FULL: every lane has two whole groups
template <int IO, bool FULL> __device__ __forceinline__ Head<IO> load_head(const void* p, int64_t at, const Unit& t) {
    return Head<IO>{raw8_part<IO>(p, at + t.lo, FULL ? 8 : t.nlo), raw8_part<IO>(p, at + t.hi, FULL ? 8 : t.nhi)};
}
template <int IO, bool FULL> __device__ __forceinline__ void store_head(void* p, int64_t at, const Unit& t, const float* x) {
    store8_part<IO>(p, at + t.lo, FULL ? 8 : t.nlo, x);
    store8_part<IO>(p, at + t.hi, FULL ? 8 : t.nhi, x + 8);
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

template <bool FULL> __device__ __forceinline__ void token_sines(const QkArgs& a, const Unit& t, int64_t b, int64_t n, float* c, float* s) {
    const int64_t pos = a.positions ? (int64_t)a.positions[b * a.pos_stride + n] : n;
    float f[8];
    load8_part<CT_F32>(a.inv_freq, t.p, FULL ? 8 : t.n, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        sines((double)pos * (double)f[k], &s[k], &c[k]);
        c[k] *= a.magnitude;
        s[k] *= a.magnitude;
    }
}

// how many of a lane's 16 elements are the head's, by index
template <bool FULL> __device__ __forceinline__ bool has(const Unit& t, int e) { return FULL || (e < 8 ? e < t.nlo : e - 8 < t.nhi); }

// u = x (centred: less its mean) in place; returns r.  The mean takes two sums: what the first one's rounding leaves shows in the
// sum of the centred values.
template <int LANES, bool CENTRED, bool FULL> __device__ __forceinline__ float normed(float* x, const Unit& t, int D, float eps) {
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
            x[e] = has<FULL>(t, e) ? x[e] - first : 0.f;
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
        for (int e = 0; e < 16; ++e) x[e] = has<FULL>(t, e) ? x[e] - rest : 0.f;
    }
    return 1.f / sqrtf(var + eps);
}

template <int IO, bool FULL> __device__ __forceinline__ void load_weights(const QkArgs& a, const Unit& t, float (*w)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (a.w[i]) {
            widen<IO>(load_head<IO, FULL>(a.w[i], 0, t), w[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[i][e] = 1.f;
        }
    }
}

template <int IO, int LANES, bool CENTRED, bool FULL>
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
        return load_head<IO, FULL>(a.x[i], b * a.xs[i].b + (int64_t)(i ? h - a.heads[0] : h) * a.xs[i].h + n * a.xs[i].n, t);
    };
    Head<IO> next = load(h0);
    float w[2][16], c[8], s[8];
    load_weights<IO, FULL>(a, t, w);
    if (t.turn) token_sines<FULL>(a, t, b, n, c, s);
    for (int h = h0; h < end; ++h) {
        const Head<IO> now = next;
        if (h + 1 < end) next = load(h + 1);
        const int i = h >= a.heads[0];
        float x[16];
        widen<IO>(now, x);
        const float r = normed<LANES, CENTRED, FULL>(x, t, a.D, a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= r * (i ? w[1][e] : w[0][e]);
        if (t.turn) turn_pairs(x, c, s, 1.f, inter);
        if (any) {
            const int64_t at = b * a.ys[i].b + (int64_t)(i ? h - a.heads[0] : h) * a.ys[i].h + n * a.ys[i].n;
            store_head<IO, FULL>(a.y[i], at, t, x);
        }
    }
}

// Workgroups first .. of the grid are q's, the others k's.
template <int IO, int LANES, bool CENTRED, bool FULL>
__global__ void __launch_bounds__(256) qknorm_bwd_kernel(QkArgs a, QkGradPlan g) {
    constexpr int GROUPS = 256 / LANES;
    const int i = (int)blockIdx.x >= g.parts[0], parts = g.parts[i], block = (int)blockIdx.x - (i ? g.parts[0] : 0), heads = a.heads[i];
    const QkPlan& p = g.p[i];
    const bool inter = a.flags & LCONV_ROTARY_INTERLEAVED;
    const int lane = threadIdx.x % LANES;
    const Unit t = unit_of(a, lane, p.turns, p.units);
    const float inv = 1.f / (float)a.D;
    Head<IO> w{};
    if (a.w[i]) w = load_head<IO, FULL>(a.w[i], 0, t);
    float sum[16] = {};
    for (int64_t g0 = (int64_t)block * GROUPS; g0 < p.items; g0 += (int64_t)parts * GROUPS) {
        const int64_t at = g0 + threadIdx.x / LANES;
        const bool any = at < p.items;
        const uint32_t item = (uint32_t)(any ? at : 0), row = item / (uint32_t)p.hgroups, hg = item - row * (uint32_t)p.hgroups;
        const int64_t b = row / (uint64_t)a.N, n = row - b * a.N;
        const int h0 = (int)hg * p.per, end = h0 + p.per < heads ? h0 + p.per : heads;
        Head<IO> nx, nd;
        const auto load = [&](int h) LCV_INLINE {
            nx = load_head<IO, FULL>(a.x[i], b * a.xs[i].b + (int64_t)h * a.xs[i].h + n * a.xs[i].n, t);
            nd = load_head<IO, FULL>(a.dy[i], b * a.dys[i].b + (int64_t)h * a.dys[i].h + n * a.dys[i].n, t);
        };
        load(h0);
        float c[8], s[8];
        if (t.turn) token_sines<FULL>(a, t, b, n, c, s);
        for (int h = h0; h < end; ++h) {
            float u[16], d[16], wf[16];
            widen<IO>(nx, u);
            widen<IO>(nd, d);
            if (h + 1 < end) load(h + 1);
            const float r = normed<LANES, CENTRED, FULL>(u, t, a.D, a.eps);
            if (t.turn) turn_pairs(d, c, s, -1.f, inter);
            widen<IO>(w, wf);
            float hu = 0.f, hs = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                u[e] *= r;
                sum[e] += any ? d[e] * u[e] : 0.f;
                if (a.w[i]) d[e] *= wf[e];
                hu += d[e] * u[e];
                if constexpr (CENTRED) hs += has<FULL>(t, e) ? d[e] : 0.f;
            }
            lane_sums<LANES>(hu, hs);
            hu *= inv;
            hs *= inv;
#pragma unroll
            for (int e = 0; e < 16; ++e) d[e] = r * (d[e] - u[e] * hu - (CENTRED ? hs : 0.f));
            if (any) {
                const int64_t to = b * a.ys[i].b + (int64_t)h * a.ys[i].h + n * a.ys[i].n;
                store_head<IO, FULL>(a.y[i], to, t, d);
            }
        }
    }
    if (!a.part) return;
    // the groups of a wave join by lanes, the waves through LDS, in a fixed order
    __shared__ float join[4][16][LANES];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int k = LANES; k < 64; k *= 2) sum[e] += __shfl_xor(sum[e], k);
        if ((threadIdx.x & 63) < LANES) join[threadIdx.x >> 6][e][lane] = sum[e];
    }
    __syncthreads();
    if (threadIdx.x >= LANES) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] = (join[0][e][lane] + join[1][e][lane]) + (join[2][e][lane] + join[3][e][lane]);
    const int64_t to = (int64_t)blockIdx.x * a.D;
    store_head<CT_F32, FULL>(a.part, to, t, sum);
}

// The weights' gradients from the workgroups' sums: a workgroup takes 32 columns of q or k, its 32 groups of lanes every
// 32nd part, and joins the groups in order.
__global__ void __launch_bounds__(1024) qknorm_sum_kernel(const float* part, float* dq, float* dk, int qparts, int kparts, int D) {
    __shared__ float join[32][33];
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + l, i = blockIdx.y, end = i ? qparts + kparts : qparts;
    float u = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int k = (i ? qparts : 0) + q; k < end; k += 32) u += part[(int64_t)k * D + c];
    }
    join[q][l] = u;
    __syncthreads();
    float* out = i ? dk : dq;
    if (q || c >= D || !out) return;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += join[k][l];
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

// f(centred, full) for a call
template <typename F> void by_form(const QkArgs& a, const QkPlan& p, F&& f) {
    using std::integral_constant;
    const bool full = a.rot % 16 == 0 && (a.D - a.rot) % 16 == 0 && p.lanes == p.units;
    const auto go = [&](auto centred) {
        if (full) f(centred, integral_constant<bool, true>{});
        else f(centred, integral_constant<bool, false>{});
    };
    if (a.flags & LCONV_QKNORM_CENTRED) go(integral_constant<bool, true>{});
    else go(integral_constant<bool, false>{});
}

}  // namespace

hipError_t launch_qknorm_fwd(int dtype, const QkArgs& a, hipStream_t stream) {
    const QkPlan p = qk_plan(a.B * a.N, a.D, a.rot, a.heads[0] + a.heads[1]);
    const unsigned grid = (unsigned)((p.items * p.lanes + 255) / 256);
    return by_dtype(dtype, [&](auto io) {
        by_lanes(p.lanes, [&](auto lanes) {
            by_form(a, p, [&](auto centred, auto full) {
                qknorm_fwd_kernel<io.value, lanes.value, centred.value, full.value><<<grid, 256, 0, stream>>>(a, p);
            });
        });
    });
}

hipError_t launch_qknorm_bwd(int dtype, const QkArgs& a, hipStream_t stream) {
    const int64_t tokens = a.B * a.N;
    QkGradPlan g{};
    hipError_t e = hipSuccess;
    if (tokens > 0 && a.heads[0] + a.heads[1] > 0) {
        g = qk_grad_plan(tokens, a.D, a.rot, a.heads[0], a.heads[1]);
        const unsigned grid = (unsigned)(g.parts[0] + g.parts[1]);
        const QkPlan& p = g.p[a.heads[0] ? 0 : 1];
        e = by_dtype(dtype, [&](auto io) {
            by_lanes(p.lanes, [&](auto lanes) {
                by_form(a, p, [&](auto centred, auto full) {
                    qknorm_bwd_kernel<io.value, lanes.value, centred.value, full.value><<<grid, 256, 0, stream>>>(a, g);
                });
            });
        });
    }
    if (e != hipSuccess || (!a.dw[0] && !a.dw[1])) return e;
    qknorm_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32), 2), 1024, 0, stream>>>(a.part, a.dw[0], a.dw[1], g.parts[0], g.parts[1], a.D);
    return hipGetLastError();
}

}  // namespace lcv
