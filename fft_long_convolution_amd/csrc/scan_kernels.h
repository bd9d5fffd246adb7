// scan_kernels.h -- the gated linear recurrence over prompts, and its gradients.
//
//   h_t = a_t h_{t-1} + u_t,  u = m s x;   gradients: G_t = dy_t + g_{t+1},  g_t = a_t G_t
// A wave takes 64 or 128 channels of 8 tokens, a lane one or two of the channels, so that the recurrence itself never
// crosses lanes.  Of its tokens a wave first needs only the product of their decays and what they add up to from zero;
// the 8 waves of a workgroup join these in order through LDS, one barrier to a tile of 64 tokens, and every wave then runs its
// tokens from its own first state.  The workgroup walks along the sequence with the state in registers and the next tile's
// loads on their way: one pass over the data.  Calls of few rows are cut into segments along the sequence: a first launch
// finds the segments' products and sums, the second begins each segment with the join of those before it.
#pragma once
#include "scan_gates.h"

namespace lcv {
namespace {

// tokens of a wave's turn as loaded
template <int IO, int V> struct Turn {
    RawV<IO, V> e[kScanTokens];
};
template <int IO, int V>
__device__ __forceinline__ void load_turn(Turn<IO, V>& r, const TokOperand& o, int64_t row, int64_t t, int64_t len, uint32_t c) {
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j) {
        const int64_t at = t + j < len ? t + j : len - 1;      // past the end: a token that there is, not used
        r.e[j] = load_raw_v<IO, V>(o.p, row + at * o.n, c);
    }
}

// a, 1 - a, m and the (folded) sigmoid behind a rate, of one token's channels
template <int V> struct Gate {
    float a[V], d[V], m[V], p[V];
};
template <int IO, int V>
__device__ __forceinline__ void gates(Gate<V>* g, const Turn<IO, V>& z, const float* rate, int gate, int mix) {
    float x[kScanTokens][V];
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j) widen<IO, V>(z.e[j], x[j]);
    const auto each = [&](auto&& f) LCV_INLINE {
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) f(g[j], x[j][v], v);
    };
    const auto set = [](Gate<V>& t, int v, Decay k) LCV_INLINE { t.a[v] = k.a; t.d[v] = k.d; };
    if (gate == LCONV_GATE_SIGMOID) {
        each([&](Gate<V>& t, float x, int v) LCV_INLINE { set(t, v, decay_of_logit(x)); });
    } else if (gate == LCONV_GATE_LOG) {
        each([&](Gate<V>& t, float x, int v) LCV_INLINE { set(t, v, decay_of_log(x)); });
    } else {
        each([&](Gate<V>& t, float x, int v) LCV_INLINE {
            t.p[v] = folded_sigmoid(x);
            set(t, v, decay_of_log(-rate[v] * unfolded(t.p[v])));
        });
    }
    if (mix == LCONV_MIX_NORM) each([&](Gate<V>& t, float, int v) LCV_INLINE { t.m[v] = norm_of(Decay{t.a[v], t.d[v]}); });
    else if (mix == LCONV_MIX_CONVEX) each([&](Gate<V>& t, float, int v) LCV_INLINE { t.m[v] = t.d[v]; });
    else each([&](Gate<V>& t, float, int v) LCV_INLINE { t.m[v] = 1.f; });
}

// where a workgroup works: row b, channels c .. of a lane, tokens first .. end of a segment.  A lane past the last channels
// takes those of the last lane that has some, and writes the same values to the same places: no load or store is under a
// lane's condition.
template <int V> struct Place {
    int64_t b, first, end;
    int seg, cb, wave;
    uint32_t c;
};
template <int V> __device__ __forceinline__ Place<V> place(const ScanArgs& a) {
    Place<V> w;
    const uint32_t per = (uint32_t)a.cblocks, i = blockIdx.x, bs = i / per;
    w.cb = (int)(i - bs * per);
    w.b = bs / (uint32_t)a.nseg;
    w.seg = (int)(bs - (uint32_t)w.b * (uint32_t)a.nseg);
    w.first = w.seg * a.seg_len;
    w.end = w.first + a.seg_len < a.N ? w.first + a.seg_len : a.N;
    w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c = (int64_t)w.cb * 64 * V + (threadIdx.x & 63) * V;
    w.c = (uint32_t)(c < a.C ? c : a.C - V);
    return w;
}

template <int V> struct LaneF { float v[V]; };
template <int V> __device__ __forceinline__ LaneF<V> load_f(const float* p) {
    LaneF<V> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
template <int V> __device__ __forceinline__ void store_f(float* p, const float* x) { __builtin_memcpy(p, x, 4 * V); }

// A segment for the state h that enters it from one side, [3][C]: its decay, the decay's residue, what it adds up from zero
template <int V> __device__ __forceinline__ void join_segment(float* h, const ScanArgs& a, const Place<V>& w, int k) {
    const float* s = a.seg + (w.b * a.nseg + k) * 3 * a.C + w.c;
    const LaneF<V> A = load_f<V>(s), r = load_f<V>(s + a.C), H = load_f<V>(s + 2 * a.C);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = moved(A.v[v], r.v[v], h[v], H.v[v]);
}
template <int V> __device__ __forceinline__ void leave_segment(const float* h, const Decay* all, const ScanArgs& a, const Place<V>& w) {
    float* s = a.seg + (w.b * a.nseg + w.seg) * 3 * a.C + w.c;
    float A[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Decay k = rounded(all[v]);
        A[v] = k.a;
        r[v] = residue(k);
    }
    store_f<V>(s, A);
    store_f<V>(s + a.C, r);
    store_f<V>(s + 2 * a.C, h);
}

// What a wave leaves for the others, and what they do with it: decay, residue, and one or two sums
template <int V> __device__ __forceinline__ void leave(float* to, const Decay* run, const float* H) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Decay k = rounded(run[v]);
        to[v] = k.a;
        to[V + v] = residue(k);
        to[2 * V + v] = H[v];
    }
}
template <int V> __device__ __forceinline__ void lengthen_by(Decay* all, const float* from) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float d = (1.f - from[v]) - from[V + v];
        all[v].a = times(all[v].a, from[v], from[V + v]);
        all[v].d += fmaf(-all[v].d, d, d);
    }
}

// STATES: only the segments' decays and sums.
template <int IO, int V, bool GATED, bool STATES>
__global__ void __launch_bounds__(64 * kScanWaves) scan_fwd_kernel(ScanArgs a) {
    __shared__ float join[2][kScanWaves][64][3 * V];
    const Place<V> w = place<V>(a);
    const int lane = threadIdx.x & 63, waves = a.waves;
    const int64_t len = row_len(a.lengths, w.b, a.N), end = w.end < len ? w.end : len;
    const int64_t xr = w.b * a.x.b, zr = w.b * a.z.b, ir = GATED ? w.b * a.i.b : 0;
    const int64_t sc = w.b * a.C + w.c;
    float rate[V], h[V];
    Decay all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = a.rate ? a.rate[w.c + v] : 0.f;
        h[v] = (STATES ? w.seg == a.nseg - 1 : a.nseg == 1) && a.state_in ? a.state_in[sc + v] : 0.f;
        all[v] = Decay{1.f, 0.f};
    }
    // Nothing follows the last segment: its place in the workspace keeps the state that enters the row, which the main pass
    // takes from there, since its last segment may write another state over it before the first one begins.
    if constexpr (STATES) {
        if (w.seg == a.nseg - 1) {
            if (w.wave == 0) leave_segment<V>(h, all, a, w);
            return;
        }
    } else if (a.nseg > 1) {
        join_segment<V>(h, a, w, a.nseg - 1);
        for (int k = 0; k < w.seg; ++k) join_segment<V>(h, a, w, k);
    }
    const int64_t mine = (int64_t)w.wave * kScanTokens;
    const int tile = waves * kScanTokens;
    Turn<IO, V> x, z, i, nx, nz, ni;
    const auto load = [&](int64_t t) LCV_INLINE {
        load_turn<IO, V>(nx, a.x, xr, t, end, w.c);
        load_turn<IO, V>(nz, a.z, zr, t, end, w.c);
        if constexpr (GATED) load_turn<IO, V>(ni, a.i, ir, t, end, w.c);
    };
    if (w.first < end) load(w.first + mine);
    int buf = 0;
    const auto turn = [&](int64_t t0, auto full) LCV_INLINE {
        const int64_t t = t0 + mine;
        x = nx; z = nz;
        if constexpr (GATED) i = ni;
        load(t + tile);
        Gate<V> g[kScanTokens];
        gates<IO, V>(g, z, rate, a.gate, a.mix);
        float dk[kScanTokens][V], rs[kScanTokens][V], u[kScanTokens][V], H[V];
        Decay run[V];
#pragma unroll
        for (int v = 0; v < V; ++v) run[v] = Decay{1.f, 0.f}, H[v] = 0.f;
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j) {
            float xv[V], iv[V];
            widen<IO, V>(x.e[j], xv);
            if constexpr (GATED) widen<IO, V>(i.e[j], iv);
            const bool on = full || t + j < end;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float in = g[j].m[v] * xv[v];
                dk[j][v] = on ? g[j].a[v] : 1.f;
                rs[j][v] = on ? residue(Decay{g[j].a[v], g[j].d[v]}) : 0.f;
                u[j][v] = on ? (GATED ? in * sigmoid(iv[v]) : in) : 0.f;
                H[v] = moved(dk[j][v], rs[j][v], H[v], u[j][v]);
                lengthen(run[v], dk[j][v], on ? g[j].d[v] : 0.f);
            }
        }
        leave<V>(join[buf][w.wave][lane], run, H);
        __syncthreads();
        if (!STATES && a.marks && w.wave == 0)
            store_f<V>(a.marks + (w.b * ((a.N + kScanTile - 1) / kScanTile) + t0 / kScanTile) * a.C + w.c, h);
        float s[V] = {};
        for (int k = 0; k < waves; ++k) {
            const bool me = k == w.wave;
            const float* from = join[buf][k][lane];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = me ? h[v] : s[v];
                h[v] = moved(from[v], from[V + v], h[v], from[2 * V + v]);
            }
            if constexpr (STATES) lengthen_by<V>(all, from);
        }
        if constexpr (!STATES) {
#pragma unroll
            for (int j = 0; j < kScanTokens; ++j) {
                float y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = moved(dk[j][v], rs[j][v], s[v], u[j][v]);
                    y[v] = full || t + j < end ? s[v] : 0.f;
                }
                if (full || t + j < w.end) store_v<IO, V>(a.y, w.b * a.yb + (t + j) * a.yn, w.c, y);
            }
        }
    };
    for (int64_t t0 = w.first; t0 < end; t0 += tile, buf ^= 1) {
        if (t0 + tile <= end) turn(t0, std::true_type{});
        else turn(t0, std::false_type{});
    }
    if constexpr (STATES) {
        if (w.wave == 0) leave_segment<V>(h, all, a, w);
    } else {
        // tokens behind the tiles of the row's own, and marks that no token needs
        const float zero[V] = {};
        int64_t t0 = end > w.first ? w.first + (end - w.first + tile - 1) / tile * tile : w.first;
        for (int64_t t = t0 + w.wave; t < w.end; t += waves) store_v<IO, V>(a.y, w.b * a.yb + t * a.yn, w.c, zero);
        if (a.state_out && w.seg == a.nseg - 1 && w.wave == 0) store_f<V>(a.state_out + sc, h);
    }
}

// The gradients, from the last tile to the first: a tile's states again from its mark, G from the carry.
// REACH: only the segments' products and what they hand to the left.
template <int IO, int V, bool GATED, bool REACH>
__global__ void __launch_bounds__(64 * kScanWaves) scan_bwd_kernel(ScanArgs a) {
    constexpr int W = REACH ? 3 * V : 4 * V;
    __shared__ float join[2][kScanWaves][64][W];
    const Place<V> w = place<V>(a);
    const int lane = threadIdx.x & 63, waves = a.waves;
    const int64_t len = row_len(a.lengths, w.b, a.N), end = w.end < len ? w.end : len;
    const int64_t xr = w.b * a.x.b, zr = w.b * a.z.b, ir = GATED ? w.b * a.i.b : 0, dr = w.b * a.dy.b;
    const int64_t sc = w.b * a.C + w.c, marks = (a.N + kScanTile - 1) / kScanTile;
    float rate[V], carry[V], drate[V];
    Decay all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = a.rate ? a.rate[w.c + v] : 0.f;
        carry[v] = (REACH ? w.seg == 0 : a.nseg == 1) && a.state_in ? a.state_in[sc + v] : 0.f;
        all[v] = Decay{1.f, 0.f};
        drate[v] = 0.f;
    }
    if constexpr (REACH) {      // as in the forward pass, from the other end
        if (w.seg == 0) {
            if (w.wave == 0) leave_segment<V>(carry, all, a, w);
            return;
        }
    } else if (a.nseg > 1) {
        join_segment<V>(carry, a, w, 0);
        for (int k = a.nseg - 1; k > w.seg; --k) join_segment<V>(carry, a, w, k);
    }
    const int64_t mine = (int64_t)w.wave * kScanTokens;
    const int tile = waves * kScanTokens;
    const float zero[V] = {};
    Turn<IO, V> x, z, i, dy, nx, nz, ni, nd;
    LaneF<V> mark{}, nmark{};
    const auto load = [&](int64_t t0) LCV_INLINE {
        const int64_t t = t0 + mine;
        load_turn<IO, V>(nz, a.z, zr, t, end, w.c);
        load_turn<IO, V>(nd, a.dy, dr, t, end, w.c);
        if constexpr (!REACH) {
            load_turn<IO, V>(nx, a.x, xr, t, end, w.c);
            if constexpr (GATED) load_turn<IO, V>(ni, a.i, ir, t, end, w.c);
            nmark = load_f<V>(a.marks + (w.b * marks + t0 / kScanTile) * a.C + w.c);
        }
    };
    const int64_t tiles = end > w.first ? (end - w.first + tile - 1) / tile : 0;
    if constexpr (!REACH) {
        for (int64_t t = w.first + tiles * tile + w.wave; t < w.end; t += waves) {
            store_v<IO, V>(a.dx, w.b * a.dxb + t * a.dxn, w.c, zero);
            store_v<IO, V>(a.dz, w.b * a.dzb + t * a.dzn, w.c, zero);
            if constexpr (GATED) store_v<IO, V>(a.di, w.b * a.dib + t * a.din, w.c, zero);
        }
    }
    if (tiles) load(w.first + (tiles - 1) * tile);
    int buf = 0;
    const auto turn = [&](int64_t t0, auto full) LCV_INLINE {
        const int64_t t = t0 + mine;
        x = nx; z = nz; dy = nd; mark = nmark;
        if constexpr (GATED) i = ni;
        load(t0 > w.first ? t0 - tile : t0);
        Gate<V> g[kScanTokens];
        gates<IO, V>(g, z, rate, a.gate, REACH ? LCONV_MIX_PLAIN : a.mix);
        float dk[kScanTokens][V], rs[kScanTokens][V], d[kScanTokens][V], H[V], R[V];
        Decay run[V];
#pragma unroll
        for (int v = 0; v < V; ++v) run[v] = Decay{1.f, 0.f}, H[v] = R[v] = 0.f;
        float xv[kScanTokens][V], sv[kScanTokens][V], before[kScanTokens][V];
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j) {
            const bool on = full || t + j < end;
            widen<IO, V>(dy.e[j], d[j]);
            if constexpr (!REACH) widen<IO, V>(x.e[j], xv[j]);
            if constexpr (GATED && !REACH) {
                widen<IO, V>(i.e[j], sv[j]);
#pragma unroll
                for (int v = 0; v < V; ++v) sv[j][v] = folded_sigmoid(sv[j][v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dk[j][v] = on ? g[j].a[v] : 1.f;
                rs[j][v] = on ? residue(Decay{g[j].a[v], g[j].d[v]}) : 0.f;
                d[j][v] = on ? d[j][v] : 0.f;
                if constexpr (!REACH) {
                    const float in = g[j].m[v] * xv[j][v];
                    H[v] = moved(dk[j][v], rs[j][v], H[v], on ? (GATED ? in * unfolded(sv[j][v]) : in) : 0.f);
                }
                lengthen(run[v], dk[j][v], on ? g[j].d[v] : 0.f);
            }
        }
#pragma unroll
        for (int j = kScanTokens - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float G = d[j][v] + R[v];
                R[v] = times(G, dk[j][v], rs[j][v]);
            }
        leave<V>(join[buf][w.wave][lane], run, R);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if constexpr (!REACH) join[buf][w.wave][lane][3 * V + v] = H[v];
        __syncthreads();
        float s[V] = {};
        for (int q = waves - 1; q >= 0; --q) {
            const bool me = q == w.wave;
            const float* from = join[buf][q][lane];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = me ? carry[v] : s[v];
                carry[v] = moved(from[v], from[V + v], carry[v], from[2 * V + v]);
            }
            if constexpr (REACH) lengthen_by<V>(all, from);
        }
        if constexpr (!REACH) {
            for (int q = 0; q < w.wave; ++q) {
                const float* from = join[buf][q][lane];
#pragma unroll
                for (int v = 0; v < V; ++v) mark.v[v] = moved(from[v], from[V + v], mark.v[v], from[3 * V + v]);
            }
#pragma unroll
            for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float in = g[j].m[v] * xv[j][v];
                    before[j][v] = mark.v[v];
                    mark.v[v] = moved(dk[j][v], rs[j][v], mark.v[v], GATED ? in * unfolded(sv[j][v]) : in);
                }
#pragma unroll
            for (int j = kScanTokens - 1; j >= 0; --j) {
                const bool on = full || t + j < end;
                float ox[V], oz[V], oi[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float G = d[j][v] + s[v], av = dk[j][v];
                    s[v] = times(G, av, rs[j][v]);
                    const float sg = GATED ? unfolded(sv[j][v]) : 1.f, sx = sg * xv[j][v], Gm = G * g[j].m[v];
                    ox[v] = Gm * sg;
                    if constexpr (GATED) oi[v] = Gm * xv[j][v] * slope(sv[j][v]);
                    // of log a: a (G h_{t-1}) + (G s x) dm / dlog a; a norm that is zero has the gradient zero
                    float dl = av * (G * before[j][v]);
                    if (a.mix == LCONV_MIX_CONVEX) dl -= av * (G * sx);
                    if (a.mix == LCONV_MIX_NORM) dl -= g[j].m[v] > 0.f ? G * sx * (av * av * fast_rcp(g[j].m[v])) : 0.f;
                    if (a.gate == LCONV_GATE_SIGMOID) dl *= g[j].d[v];
                    if (a.gate == LCONV_GATE_RATE) {
                        drate[v] -= on ? dl * unfolded(g[j].p[v]) : 0.f;
                        dl *= -rate[v] * slope(g[j].p[v]);
                    }
                    ox[v] = on ? ox[v] : 0.f;
                    oz[v] = on ? dl : 0.f;
                    if constexpr (GATED) oi[v] = on ? oi[v] : 0.f;
                }
                if (full || t + j < w.end) {
                    store_v<IO, V>(a.dx, w.b * a.dxb + (t + j) * a.dxn, w.c, ox);
                    store_v<IO, V>(a.dz, w.b * a.dzb + (t + j) * a.dzn, w.c, oz);
                    if constexpr (GATED) store_v<IO, V>(a.di, w.b * a.dib + (t + j) * a.din, w.c, oi);
                }
            }
        }
    };
    for (int64_t k = tiles - 1; k >= 0; --k, buf ^= 1) {
        const int64_t t0 = w.first + k * tile;
        if (t0 + tile <= end) turn(t0, std::true_type{});
        else turn(t0, std::false_type{});
    }
    if constexpr (REACH) {
        if (w.wave == 0) leave_segment<V>(carry, all, a, w);
    } else {
        if (a.state_out && w.seg == 0 && w.wave == 0) store_f<V>(a.state_out + sc, carry);
        if (a.part) {      // the waves' sums in order
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v) join[0][w.wave][lane][v] = drate[v];
            __syncthreads();
            if (w.wave == 0) {
                float sum[V] = {};
                for (int q = 0; q < waves; ++q)
#pragma unroll
                    for (int v = 0; v < V; ++v) sum[v] += join[0][q][lane][v];
                store_f<V>(a.part + (w.b * a.nseg + w.seg) * a.C + w.c, sum);
            }
        }
    }
}

template <int IO, int V, bool GATED> hipError_t scan_fwd(const ScanArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.B * a.nseg * a.cblocks);
    if (a.nseg > 1) scan_fwd_kernel<IO, V, GATED, true><<<grid, 64 * a.waves, 0, stream>>>(a);
    scan_fwd_kernel<IO, V, GATED, false><<<grid, 64 * a.waves, 0, stream>>>(a);
    return hipGetLastError();
}
template <int IO> hipError_t scan_fwd(const ScanArgs& a, hipStream_t stream) {
    if (a.vec == 1) return a.i.p ? scan_fwd<IO, 1, true>(a, stream) : scan_fwd<IO, 1, false>(a, stream);
    return a.i.p ? scan_fwd<IO, 2, true>(a, stream) : scan_fwd<IO, 2, false>(a, stream);
}

template <int IO, int V, bool GATED> hipError_t scan_bwd(const ScanArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.B * a.nseg * a.cblocks);
    if (a.nseg > 1) scan_bwd_kernel<IO, V, false, true><<<grid, 64 * a.waves, 0, stream>>>(a);
    scan_bwd_kernel<IO, V, GATED, false><<<grid, 64 * a.waves, 0, stream>>>(a);
    return hipGetLastError();
}
template <int IO> hipError_t scan_bwd(const ScanArgs& a, hipStream_t stream) {
    if (a.vec == 1) return a.i.p ? scan_bwd<IO, 1, true>(a, stream) : scan_bwd<IO, 1, false>(a, stream);
    return a.i.p ? scan_bwd<IO, 2, true>(a, stream) : scan_bwd<IO, 2, false>(a, stream);
}

}  // namespace
}  // namespace lcv
