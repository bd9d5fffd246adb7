// scan_kernels.h -- the gated linear recurrence over prompts, and its gradients.
//
//   h_t = a_t h_{t-1} + u_t,  u = m s x;   gradients: G_t = dy_t + g_{t+1},  g_t = a_t G_t
// A wave takes 64 or 128 channels of 8 tokens, a lane one or two of the channels, so that the recurrence itself never
// crosses lanes.  Of its tokens a wave first needs only their decay and what they add up from zero; the waves of a
// workgroup leave these in LDS, one barrier to a tile, and every wave joins what stands before it and runs its
// tokens from its own first state.  The last wave's last state enters the next tile.  The workgroup walks along the
// sequence with the next tile's loads on their way: one pass over the data.  Calls of few rows are cut into segments along the
// sequence: a first launch finds the segments' decays and sums, the second begins each segment with the join of those
// before it.
// Bound by HBM where a call has rows enough (times of calls in a row, every call on other inputs than the last):
// 8 x 2048 x 4096 in bf16 with every input takes 113 us, 537 MB at 4.8 TB/s (the same reads and writes with no arithmetic 106),
// under 39 vector instructions to a token and channel, 66 us of issue; sigmoid and convex in fp32 164, 805 MB at 4.9 TB/s.  In
// segments 1 x 65536 x 2048, sigmoid and convex, takes 287 us: by a trace, averages, 128 for the segments' sums (537 MB, 4.2 TB/s;
// 21 instructions and two slow ones are 90 us of issue) and 166 for the pass (805 MB, 4.8 TB/s).  Gradients, the rate's sum with
// them: 8 x 2048 x 4096 with every input, two channels to a lane, 209 us for 940 MB, 4.5 TB/s; 8 x 2048 x 2048, whose 256 workgroups
// take one channel to a lane and so 128 bytes of a row at a time, 118 us for 470 MB, 4.0 TB/s (the forward pass's reads and writes
// alone reach 4.4 so); sigmoid and convex in fp32 279 us for 1.34 GB, 4.8 TB/s.
#pragma once
#include "scan_gates.h"

namespace lcv {
namespace {

// A lane's channels, hidden from the optimiser where they are used: it would add them to the operands' pointers outside the
// loop, and then a wave's part of an address to that by 64-bit vector additions, where an instruction adds a lane's 32 bits to a
// wave's address by itself.
__device__ __forceinline__ uint32_t in_place(uint32_t c) {
    asm volatile("" : "+v"(c));
    return c;
}

// tokens of a wave's turn as stored
template <int IO, int V> struct Turn {
    RawV<IO, V> e[kScanTokens];
};
// Tokens t .. of an operand's row.  CLAMP: those from `end` on replaced by the last one that there is (not used then).  No branch:
// where ways meet, a load's register is copied, and the copy waits for the load.
template <int IO, int V, bool CLAMP>
__device__ __forceinline__ void load_turn(Turn<IO, V>& r, const TokOperand& o, int64_t row, int64_t t, int64_t end, uint32_t c) {
    const typename Elem<IO>::T* p = (const typename Elem<IO>::T*)o.p + row + (!CLAMP || t < end ? t : end - 1) * o.n;
    c = in_place(c);
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j) {
        r.e[j] = load_raw_v<IO, V>(p, 0, c);
        p += !CLAMP || t + j + 1 < end ? o.n : 0;
    }
}
template <int IO, int V>
__device__ __forceinline__ void store_turn(void* y, int64_t row, int64_t n, int64_t t, uint32_t c, const Turn<IO, V>& r, int tokens) {
    typename Elem<IO>::T* p = (typename Elem<IO>::T*)y + row + t * n;
    c = in_place(c);
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j, p += n)
        if (j < tokens) store_raw_v<IO, V>(p, 0, c, r.e[j]);
}
// A turn as fp32.  The registers that it was loaded into are free behind this, and the next turn's loads may follow at once.
template <int V> struct Wide {
    float e[kScanTokens][V];
};
template <int IO, int V> __device__ __forceinline__ void widen_turn(Wide<V>& w, const Turn<IO, V>& r) {
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j) widen<IO, V>(r.e[j], w.e[j]);
}
// how many of a turn's tokens come before `end`
__device__ __forceinline__ int tokens_before(int64_t t, int64_t end) {
    return t >= end ? 0 : end - t < kScanTokens ? (int)(end - t) : kScanTokens;
}

// One token's decays and what its input is multiplied with; for the gradients also 1 / m of a norm and the sigmoid behind a rate
template <int V> struct Gate {
    Decay k[V];
    float m[V], inv[V];
    Sigmoid p[V];
};
// The gates of a turn's first n tokens (those behind forget nothing), and the decay of all of them: the logarithms' sum where
// there are logarithms.  rate: -rate log2(e).
template <int V, int GATE, int MIX, bool GRAD>
__device__ __forceinline__ void gates(Gate<V>* g, Decay* run, const Wide<V>& z, const float* rate, int n) {
    float sum[V] = {};
    RunDecay all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) all[v] = RunDecay{1.f, 0.f};
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float x = z.e[j][v];
            Decay k;
            if constexpr (GATE == LCONV_GATE_SIGMOID) {
                k = decay_of_logit(x);
                if (j >= n) k = Decay{1.f, 0.f};
                lengthen(all[v], k);
            } else {
                float l = kLog2e * x;
                if constexpr (GATE == LCONV_GATE_RATE) {
                    if constexpr (GRAD) g[j].p[v] = sloped_sigmoid(x);
                    l = rate[v] * (GRAD ? g[j].p[v].s : sigmoid(x));
                }
                l = j < n ? l : 0.f;
                sum[v] += l;
                k = decay_of_log2(l);
            }
            g[j].k[v] = k;
            if constexpr (MIX == LCONV_MIX_NORM && GRAD) {
                const float e = energy_of(k);
                g[j].inv[v] = inverse_norm(e);
                g[j].m[v] = e * g[j].inv[v];
            } else {
                g[j].m[v] = MIX == LCONV_MIX_NORM ? norm_of(k) : MIX == LCONV_MIX_CONVEX ? loss_of(k) : 1.f;
            }
        }
#pragma unroll
    for (int v = 0; v < V; ++v) run[v] = GATE == LCONV_GATE_SIGMOID ? whole(all[v]) : decay_of_log2(sum[v]);
}
template <int V, bool GATED> __device__ __forceinline__ void inputs(float (*u)[V], const Gate<V>* g, const Wide<V>& x, const Wide<V>& i, int n) {
#pragma unroll
    for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            u[j][v] = g[j].m[v] * x.e[j][v];
            if constexpr (GATED) u[j][v] *= sigmoid(i.e[j][v]);
            u[j][v] = j < n ? u[j][v] : 0.f;
        }
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
    w.c = (uint32_t)(c < a.C - V ? c : a.C - V);
    return w;
}

template <int V> struct LaneF { float v[V]; };
template <int V> __device__ __forceinline__ LaneF<V> load_f(const float* p) {
    LaneF<V> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
template <int V> __device__ __forceinline__ void store_f(float* p, const float* x) { __builtin_memcpy(p, x, 4 * V); }

// The segments before this one (BACK: behind it) for the state h: each [3][C], its decay (two) and what it adds up from zero.  The
// first to join is what enters the row, which stands in the place of the last segment (BACK: of the first).  Eight at a time, so
// that their reads wait together, behind the first tile's (5 x 777 x 333 in fp32, 7 segments: 7.3 us for 8.4 one after another).
// Bound by that chain in long and narrow rows, which have up to 512 segments: 1 x 65536 x 128, sigmoid and convex, 136 us, of which
// the data's share is below 20.
template <int V, bool BACK> __device__ __forceinline__ void join_segments(float* h, const ScanArgs& a, const Place<V>& w) {
    constexpr int BATCH = 8;
    const int count = BACK ? a.nseg - w.seg : w.seg + 1;
    for (int e0 = 0; e0 < count; e0 += BATCH) {
        LaneF<V> c[BATCH], r[BATCH], H[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const int i = e0 + e < count ? e0 + e : 0, k = BACK ? (i ? a.nseg - i : 0) : (i ? i - 1 : a.nseg - 1);
            const float* s = a.seg + (w.b * a.nseg + k) * 3 * a.C + w.c;
            c[e] = load_f<V>(s);
            r[e] = load_f<V>(s + a.C);
            H[e] = load_f<V>(s + 2 * a.C);
        }
#pragma unroll
        for (int e = 0; e < BATCH; ++e)
            if (e0 + e < count) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = moved(Decay{c[e].v[v], r[e].v[v]}, h[v], H[e].v[v]);
            }
    }
}
template <int V> __device__ __forceinline__ void leave_segment(const float* h, const Decay* all, const ScanArgs& a, const Place<V>& w) {
    float* s = a.seg + (w.b * a.nseg + w.seg) * 3 * a.C + w.c;
    float c[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = all[v].c, r[v] = all[v].w;
    store_f<V>(s, c);
    store_f<V>(s + a.C, r);
    store_f<V>(s + 2 * a.C, h);
}

// What a wave leaves for the others: its decay and a sum
template <int V> __device__ __forceinline__ void leave(float* to, const Decay* run, const float* H) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        to[v] = run[v].c;
        to[V + v] = run[v].w;
        to[2 * V + v] = H[v];
    }
}
template <int V> __device__ __forceinline__ void join(float* h, const float* from, const float* sum) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = moved(Decay{from[v], from[V + v]}, h[v], sum[v]);
}
// h past the waves before this one, or (BACK) from the last wave down to the one behind it: four at a time, so that four
// reads from LDS wait together.
template <int V, int W, bool BACK>
__device__ __forceinline__ void join_waves(float* h, const float (*left)[64][W], int lane, int wave, int waves, int sum) {
    const int count = BACK ? waves - 1 - wave : wave;
    for (int e0 = 0; e0 < count; e0 += 4) {
        float from[4][2 * V], add[4][V];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = e0 + e < count ? e0 + e : 0;
            const float* const p = left[BACK ? waves - 1 - k : k][lane];
            __builtin_memcpy(from[e], p, sizeof(from[e]));
            __builtin_memcpy(add[e], p + sum, sizeof(add[e]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e0 + e < count) join<V>(h, from[e], add[e]);
    }
}

template <int IO, int V, bool GATED, int GATE, int MIX> __global__ void __launch_bounds__(64 * scan_waves(V)) scan_fwd_kernel(ScanArgs a) {
    __shared__ float left[2][scan_waves(V)][64][3 * V], edge[2][64][V];
    const Place<V> w = place<V>(a);
    const int lane = threadIdx.x & 63, last = a.waves - 1;
    const int64_t len = row_len(a.lengths, w.b, a.N), end = w.end < len ? w.end : len;
    const int64_t xr = w.b * a.x.b, zr = w.b * a.z.b, ir = GATED ? w.b * a.i.b : 0, yr = w.b * a.yb;
    const int64_t sc = w.b * a.C + w.c;
    float* const marks = a.marks ? a.marks + w.b * ((a.N + kScanMark - 1) / kScanMark) * a.C + w.c : nullptr;
    float rate[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = GATE == LCONV_GATE_RATE ? -kLog2e * a.rate[w.c + v] : 0.f;
        h[v] = a.nseg == 1 && a.state_in ? a.state_in[sc + v] : 0.f;
    }
    const int64_t mine = (int64_t)w.wave * kScanTokens;
    const int tile = a.waves * kScanTokens;
    Turn<IO, V> nx, nz, ni;
    Wide<V> x, z, i;
    const auto load = [&](int64_t t, auto clamp) LCV_INLINE {
        load_turn<IO, V, clamp.value>(nx, a.x, xr, t, end, w.c);
        load_turn<IO, V, clamp.value>(nz, a.z, zr, t, end, w.c);
        if constexpr (GATED) load_turn<IO, V, clamp.value>(ni, a.i, ir, t, end, w.c);
    };
    // A turn's results are stored at the beginning of the next one, in front of the wait for that one's loads: the number of
    // memory operations behind the loads is the same on every way into the loop, so that the wait is for them alone and not
    // for the stores.  The first turn stores zeros where its own results will stand.
    Turn<IO, V> held{};
    if (w.first < end) load(w.first + mine, std::true_type{});
    if (a.nseg > 1) join_segments<V, false>(h, a, w);
    if (w.wave == last) store_f<V>(edge[0][lane], h);
    int buf = 0;
    const auto turn = [&](int64_t t0, auto full, auto clamp) LCV_INLINE {
        const int64_t t = t0 + mine;
        if constexpr (full) store_turn<IO, V>(a.y, yr, a.yn, t0 > w.first ? t - tile : t, w.c, held, kScanTokens);
        widen_turn<IO, V>(z, nz);
        widen_turn<IO, V>(x, nx);
        if constexpr (GATED) widen_turn<IO, V>(i, ni);
        __builtin_amdgcn_sched_barrier(0);
        load(t + tile, clamp);
        const int n = full ? kScanTokens : tokens_before(t, end);
        Gate<V> g[kScanTokens];
        Decay run[V];
        gates<V, GATE, MIX, false>(g, run, z, rate, n);
        float u[kScanTokens][V], H[V] = {};
        inputs<V, GATED>(u, g, x, i, n);
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) H[v] = moved(g[j].k[v], H[v], u[j][v]);
        leave<V>(left[buf][w.wave][lane], run, H);
        __syncthreads();
        LaneF<V> s = load_f<V>(edge[buf][lane]);
        join_waves<V, 3 * V, false>(s.v, left[buf], lane, w.wave, a.waves, 2 * V);
        if (marks && t % kScanMark == 0 && (full || t < end)) store_f<V>(marks + t / kScanMark * a.C, s.v);
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s.v[v] = moved(g[j].k[v], s.v[v], u[j][v]);
                y[v] = j < n ? s.v[v] : 0.f;
            }
            held.e[j] = narrow<IO, V>(y);
        }
        if (w.wave == last) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = s.v[v];
            store_f<V>(edge[buf ^ 1][lane], h);
        }
        buf ^= 1;
    };
    int64_t t0 = w.first;
    for (; t0 + 2 * tile <= end; t0 += tile) turn(t0, std::true_type{}, std::false_type{});
    if (t0 + tile <= end) {
        turn(t0, std::true_type{}, std::true_type{});
        t0 += tile;
    }
    if (t0 > w.first) store_turn<IO, V>(a.y, yr, a.yn, t0 - tile + mine, w.c, held, kScanTokens);
    if (t0 < end) {
        turn(t0, std::false_type{}, std::true_type{});
        store_turn<IO, V>(a.y, yr, a.yn, t0 + mine, w.c, held, tokens_before(t0 + mine, w.end));
        t0 += tile;
    }
    // tokens behind the row's own tiles
    const float zero[V] = {};
    for (int64_t t = t0 + w.wave; t < w.end; t += a.waves) store_v<IO, V>(a.y, yr + t * a.yn, w.c, zero);
    if (a.state_out && w.seg == a.nseg - 1 && w.wave == last) store_f<V>(a.state_out + sc, h);
}

// The gradients, from the last tile to the first: a tile's states again from its mark, G from the first wave's last one.
template <int IO, int V, bool GATED, int GATE, int MIX> __global__ void __launch_bounds__(64 * kScanGradWaves) scan_bwd_kernel(ScanArgs a) {
    __shared__ float left[2][kScanGradWaves][64][4 * V], edge[2][64][V];
    const Place<V> w = place<V>(a);
    const int lane = threadIdx.x & 63, waves = a.waves;
    const int64_t len = row_len(a.lengths, w.b, a.N), end = w.end < len ? w.end : len;
    const int64_t xr = w.b * a.x.b, zr = w.b * a.z.b, ir = GATED ? w.b * a.i.b : 0, dr = w.b * a.dy.b;
    const int64_t sc = w.b * a.C + w.c;
    const float* const marks = a.marks + w.b * ((a.N + kScanMark - 1) / kScanMark) * a.C;
    float rate[V], per_slope[V], carry[V], drate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        per_slope[v] = GATE == LCONV_GATE_RATE ? -a.rate[w.c + v] : 0.f;
        rate[v] = kLog2e * per_slope[v];
        carry[v] = a.nseg == 1 && a.state_in ? a.state_in[sc + v] : 0.f;
        drate[v] = 0.f;
    }
    const int64_t mine = (int64_t)w.wave * kScanTokens;
    const int tile = waves * kScanTokens;
    Turn<IO, V> nx, nz, ni, nd;
    Wide<V> x, z, i, d;
    RawV<CT_F32, V> mark{}, nmark{};
    const auto load = [&](int64_t t0, auto clamp) LCV_INLINE {
        const int64_t t = t0 + mine;
        load_turn<IO, V, clamp.value>(nz, a.z, zr, t, end, w.c);
        load_turn<IO, V, clamp.value>(nx, a.x, xr, t, end, w.c);
        if constexpr (GATED) load_turn<IO, V, clamp.value>(ni, a.i, ir, t, end, w.c);
        load_turn<IO, V, clamp.value>(nd, a.dy, dr, t, end, w.c);
        nmark = load_raw_v<CT_F32, V>(marks, t0 / kScanMark * a.C, in_place(w.c));
    };
    const int64_t tiles = end > w.first ? (end - w.first + tile - 1) / tile : 0;
    {
        const float zero[V] = {};
        for (int64_t t = w.first + tiles * tile + w.wave; t < w.end; t += waves) {
            store_v<IO, V>(a.dx, w.b * a.dxb + t * a.dxn, w.c, zero);
            store_v<IO, V>(a.dz, w.b * a.dzb + t * a.dzn, w.c, zero);
            if constexpr (GATED) store_v<IO, V>(a.di, w.b * a.dib + t * a.din, w.c, zero);
        }
    }
    if (tiles) load(w.first + (tiles - 1) * tile, std::true_type{});
    if (a.nseg > 1) join_segments<V, true>(carry, a, w);
    if (w.wave == 0) store_f<V>(edge[0][lane], carry);
    int buf = 0;
    Turn<IO, V> ox{}, oz{}, oi{};      // a turn's results, stored by the next one as in the forward pass
    const auto store = [&](int64_t t, int there) LCV_INLINE {
        store_turn<IO, V>(a.dx, w.b * a.dxb, a.dxn, t, w.c, ox, there);
        store_turn<IO, V>(a.dz, w.b * a.dzb, a.dzn, t, w.c, oz, there);
        if constexpr (GATED) store_turn<IO, V>(a.di, w.b * a.dib, a.din, t, w.c, oi, there);
    };
    const auto turn = [&](int64_t t0, int64_t before_t0, auto full) LCV_INLINE {
        const int64_t t = t0 + mine;
        if constexpr (full) store(before_t0 + mine, kScanTokens);
        widen_turn<IO, V>(z, nz);
        widen_turn<IO, V>(x, nx);
        if constexpr (GATED) widen_turn<IO, V>(i, ni);
        widen_turn<IO, V>(d, nd);
        mark = nmark;
        __builtin_amdgcn_sched_barrier(0);
        load(t0 > w.first ? t0 - tile : t0, std::integral_constant<bool, !full>{});
        const int n = full ? kScanTokens : tokens_before(t, end);
        Gate<V> g[kScanTokens];
        Decay run[V];
        gates<V, GATE, MIX, true>(g, run, z, rate, n);
        // Within a turn a decay is one number: its rounding meets eight tokens.  From turn to turn runs go by `run`, and so does
        // what the next tile begins with.
        float u[kScanTokens][V], H[V] = {}, R[V] = {}, before[kScanTokens][V], av[kScanTokens][V];
        Sigmoid in[kScanTokens][V];
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                av[j][v] = value_of(g[j].k[v]);
                d.e[j][v] = j < n ? d.e[j][v] : 0.f;
                if constexpr (GATED) {
                    in[j][v] = sloped_sigmoid(i.e[j][v]);
                    x.e[j][v] *= in[j][v].s;
                }
                u[j][v] = g[j].m[v] * x.e[j][v];
                u[j][v] = j < n ? u[j][v] : 0.f;
                H[v] = fmaf(av[j][v], H[v], u[j][v]);
            }
#pragma unroll
        for (int j = kScanTokens - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) R[v] = av[j][v] * (d.e[j][v] + R[v]);
        leave<V>(left[buf][w.wave][lane], run, R);
        store_f<V>(left[buf][w.wave][lane] + 3 * V, H);
        __syncthreads();
        LaneF<V> s = load_f<V>(edge[buf][lane]);
        join_waves<V, 4 * V, true>(s.v, left[buf], lane, w.wave, waves, 2 * V);
        join_waves<V, 4 * V, false>(mark.e, left[buf], lane, w.wave, waves, 3 * V);
        if (w.wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) carry[v] = moved(run[v], s.v[v], R[v]);
            store_f<V>(edge[buf ^ 1][lane], carry);
        }
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                before[j][v] = mark.e[v];
                mark.e[v] = fmaf(av[j][v], mark.e[v], u[j][v]);
            }
#pragma unroll
        for (int j = kScanTokens - 1; j >= 0; --j) {
            const bool on = j < n;
            float gx[V], gz[V], gi[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float G = d.e[j][v] + s.v[v], Gm = G * g[j].m[v];
                s.v[v] = av[j][v] * G;
                gx[v] = on ? (GATED ? Gm * in[j][v].s : Gm) : 0.f;
                if constexpr (GATED) gi[v] = on ? Gm * x.e[j][v] * in[j][v].rest : 0.f;
                // of log a: a G (h_{t-1} + s x dm / da), dm / da = 0, -1, -a / m; a norm that is zero has the gradient zero
                float dl = before[j][v];
                if constexpr (MIX != LCONV_MIX_PLAIN) dl -= MIX == LCONV_MIX_CONVEX ? x.e[j][v] : x.e[j][v] * (av[j][v] * g[j].inv[v]);
                dl *= s.v[v];
                if constexpr (GATE == LCONV_GATE_SIGMOID) dl *= loss_of(g[j].k[v]);
                if constexpr (GATE == LCONV_GATE_RATE) {
                    dl *= g[j].p[v].s;
                    drate[v] -= on ? dl : 0.f;
                    dl *= per_slope[v] * g[j].p[v].rest;
                }
                gz[v] = on ? dl : 0.f;
            }
            ox.e[j] = narrow<IO, V>(gx);
            oz.e[j] = narrow<IO, V>(gz);
            if constexpr (GATED) oi.e[j] = narrow<IO, V>(gi);
        }
        buf ^= 1;
    };
    int64_t t0 = w.first + (tiles - 1) * tile;
    if (tiles && t0 + tile > end) {
        turn(t0, t0, std::false_type{});
        store(t0 + mine, tokens_before(t0 + mine, w.end));
        t0 -= tile;
    }
    if (t0 >= w.first) {
        for (int64_t to = t0; t0 >= w.first; to = t0, t0 -= tile) turn(t0, to, std::true_type{});
        store(w.first + mine, kScanTokens);
    }
    if (a.state_out && w.seg == 0 && w.wave == 0) store_f<V>(a.state_out + sc, carry);
    if (GATE != LCONV_GATE_RATE || !a.part) return;
    __syncthreads();       // the waves' sums in order
    store_f<V>(left[0][w.wave][lane], drate);
    __syncthreads();
    if (w.wave) return;
    float sum[V] = {};
    for (int q = 0; q < waves; ++q)
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] += left[0][q][lane][v];
    store_f<V>(a.part + (w.b * a.nseg + w.seg) * a.C + w.c, sum);
}

// The segments' decays and what they add up from zero (BACK: what they hand to the left).  The waves take a piece of the
// segment each, one after another along the sequence, and join at its end.
// Nothing follows the last segment (BACK: comes before the first): its place in the workspace keeps the state that enters the row,
// which the main pass takes from there, since it may write another one over it before its first segment begins.
template <int IO, int V, bool GATED, int GATE, int MIX, bool BACK> __global__ void __launch_bounds__(512) scan_segments_kernel(ScanArgs a) {
    __shared__ float left[8][64][3 * V];
    const Place<V> w = place<V>(a);
    const int lane = threadIdx.x & 63, waves = a.waves;
    const int64_t len = row_len(a.lengths, w.b, a.N);
    const TokOperand& from = BACK ? a.dy : a.x;
    float rate[V], H[V];
    Decay run[V];
    RunDecay all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = GATE == LCONV_GATE_RATE ? -kLog2e * a.rate[w.c + v] : 0.f;
        H[v] = 0.f;
        run[v] = Decay{1.f, 0.f};
        all[v] = RunDecay{1.f, 0.f};
    }
    if (w.seg == (BACK ? 0 : a.nseg - 1)) {
        if (w.wave) return;
        if (a.state_in) {
            const LaneF<V> s = load_f<V>(a.state_in + w.b * a.C + w.c);
#pragma unroll
            for (int v = 0; v < V; ++v) H[v] = s.v[v];
        }
        leave_segment<V>(H, run, a, w);
        return;
    }
    const int64_t piece = a.seg_len / waves, first = w.first + w.wave * piece;      // whole turns
    const int64_t stop = first + piece < len ? first + piece : len, turns = stop > first ? (stop - first + kScanTokens - 1) / kScanTokens : 0;
    Turn<IO, V> nx, nz, ni;
    Wide<V> x, z, i;
    const auto load = [&](int64_t k) LCV_INLINE {
        const int64_t t = first + (BACK ? turns - 1 - k : k) * kScanTokens;
        load_turn<IO, V, true>(nx, from, w.b * from.b, t, stop, w.c);
        load_turn<IO, V, true>(nz, a.z, w.b * a.z.b, t, stop, w.c);
        if constexpr (GATED) load_turn<IO, V, true>(ni, a.i, w.b * a.i.b, t, stop, w.c);
    };
    const auto turn = [&](int64_t k, auto full) LCV_INLINE {
        const int64_t t = first + (BACK ? turns - 1 - k : k) * kScanTokens;
        widen_turn<IO, V>(z, nz);
        widen_turn<IO, V>(x, nx);
        if constexpr (GATED) widen_turn<IO, V>(i, ni);
        __builtin_amdgcn_sched_barrier(0);
        load(k + 1 < turns ? k + 1 : k);
        const int n = full ? kScanTokens : (int)(stop - t);
        Gate<V> g[kScanTokens];
        gates<V, GATE, MIX, false>(g, run, z, rate, n);
        float u[kScanTokens][V];
        inputs<V, GATED>(u, g, x, i, n);
#pragma unroll
        for (int e = 0; e < kScanTokens; ++e) {
            const int j = BACK ? kScanTokens - 1 - e : e;
#pragma unroll
            for (int v = 0; v < V; ++v) H[v] = BACK ? times(g[j].k[v], u[j][v] + H[v]) : moved(g[j].k[v], H[v], u[j][v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) lengthen(all[v], run[v]);
    };
    if (turns) load(0);
    for (int64_t k = 0; k < turns; ++k) {
        const int64_t t = first + (BACK ? turns - 1 - k : k) * kScanTokens;
        if (t + kScanTokens <= stop) turn(k, std::true_type{});
        else turn(k, std::false_type{});
    }
#pragma unroll
    for (int v = 0; v < V; ++v) run[v] = whole(all[v]);
    leave<V>(left[w.wave][lane], run, H);
    __syncthreads();
    if (w.wave) return;
#pragma unroll
    for (int v = 0; v < V; ++v) all[v] = RunDecay{1.f, 0.f}, H[v] = 0.f;
    for (int e = 0; e < waves; ++e) {
        const float* const k = left[BACK ? waves - 1 - e : e][lane];
        join<V>(H, k, k + 2 * V);
#pragma unroll
        for (int v = 0; v < V; ++v) lengthen(all[v], Decay{k[v], k[V + v]});
    }
#pragma unroll
    for (int v = 0; v < V; ++v) run[v] = whole(all[v]);
    leave_segment<V>(H, run, a, w);
}

// f(gate, mix) for a call's flags
template <typename F> void by_flags(int gate, int mix, F&& f) {
    using std::integral_constant;
    const auto go = [&](auto g) {
        if (mix == LCONV_MIX_NORM) f(g, integral_constant<int, LCONV_MIX_NORM>{});
        else if (mix == LCONV_MIX_CONVEX) f(g, integral_constant<int, LCONV_MIX_CONVEX>{});
        else f(g, integral_constant<int, LCONV_MIX_PLAIN>{});
    };
    if (gate == LCONV_GATE_RATE) go(integral_constant<int, LCONV_GATE_RATE>{});
    else if (gate == LCONV_GATE_SIGMOID) go(integral_constant<int, LCONV_GATE_SIGMOID>{});
    else go(integral_constant<int, LCONV_GATE_LOG>{});
}

template <int IO, int V, bool GATED> hipError_t scan_fwd(const ScanArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.B * a.nseg * a.cblocks);
    by_flags(a.gate, a.mix, [&](auto gate, auto mix) {
        if (a.nseg > 1) scan_segments_kernel<IO, V, GATED, gate.value, mix.value, false><<<grid, 64 * a.waves, 0, stream>>>(a);
        scan_fwd_kernel<IO, V, GATED, gate.value, mix.value><<<grid, 64 * a.waves, 0, stream>>>(a);
    });
    return hipGetLastError();
}
template <int IO> hipError_t scan_fwd(const ScanArgs& a, hipStream_t stream) {
    if constexpr (IO != CT_F32) {
        if (a.vec == 2) return a.i.p ? scan_fwd<IO, 2, true>(a, stream) : scan_fwd<IO, 2, false>(a, stream);
    }
    return a.i.p ? scan_fwd<IO, 1, true>(a, stream) : scan_fwd<IO, 1, false>(a, stream);
}

template <int IO, int V, bool GATED> hipError_t scan_bwd(const ScanArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.B * a.nseg * a.cblocks);
    by_flags(a.gate, a.mix, [&](auto gate, auto mix) {
        if (a.nseg > 1) scan_segments_kernel<IO, V, false, gate.value, LCONV_MIX_PLAIN, true><<<grid, 64 * a.waves, 0, stream>>>(a);
        scan_bwd_kernel<IO, V, GATED, gate.value, mix.value><<<grid, 64 * a.waves, 0, stream>>>(a);
    });
    return hipGetLastError();
}
template <int IO> hipError_t scan_bwd(const ScanArgs& a, hipStream_t stream) {
    if constexpr (IO != CT_F32) {
        if (a.vec == 2) return a.i.p ? scan_bwd<IO, 2, true>(a, stream) : scan_bwd<IO, 2, false>(a, stream);
    }
    return a.i.p ? scan_bwd<IO, 1, true>(a, stream) : scan_bwd<IO, 1, false>(a, stream);
}

}  // namespace
}  // namespace lcv
