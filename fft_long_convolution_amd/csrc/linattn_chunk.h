// linattn_chunk.h -- linear attention with a decay for each head, by chunks on the matrix cores
// (instantiated per type in linattn_f32.hip, linattn_f16.hip and linattn_bf16.hip).
//
// A chunk of C tokens with the state S that enters it (gamma = exp(log_decay), r = 1 for the
// gradients' direction, else 0):
//   O_i = s_q ( s_kv sum_{j<=i} gamma^(i-j) (Q_i . K_j) V_j + gamma^(i+1-r) S^T Q_i )
//   S  <- gamma^c S + s_kv sum_j gamma^(c-1-j+r) K_j V_j^T
// One pass over the data: a workgroup walks its (b, h), or a segment of it, chunk by chunk with S in
// fp32 in the registers of its four waves; a wave owns 16 NW columns of S and of O, and every row.
//
// How the four products follow each other in registers (lane = 16 g + x, tiles of 16 x 16, the
// accumulator holds rows 4 g + r, r < 4, of column x):
//   P^T  = K Q^T      accumulator: tokens j = 4g + r of query i = x, which is what the next product
//   O^T += V^T P^T    takes as its right operand (column i, contraction over j): no lane moves
//   O^T += S^T Q^T    S's accumulators (rows d = 4g + r, column n = x) are the left operand as they are
//   S   += K^T V      both operands stand transposed to their rows in LDS: ds_read_b64_tr_b16 for 16-bit
//                 types, four strided reads for fp32
// The contraction order inside an operand is {16 t + 4 g + s, 16 (t + 1) + 4 g + s} for a step of 32
// (16-bit) and {16 t + 4 g + s} for fp32, alike on both sides.  Every wave forms all of P (4 of about
// 18 matrix steps per tile) rather than share it through LDS and a barrier.
//
// Precision.  S, P and every sum are fp32.  For 16-bit types P and S are rounded to the type once as
// operands, like the result itself.  What S adds up is not: gamma^.. V is split into three bf16 parts
// (two where no state leaves the call, whose error is 2^-17) or two fp16 parts, so that the state keeps fp32's accuracy over any length.
// fp16 operands that may pass its range (P, S, gamma^.. V) are scaled to it by a power of two, per query,
// per 16 columns and per column.  gamma^c S is S + (gamma^c - 1) S, so that a decay near one does not lose by rounding
// its power.
#pragma once
#include "mixer_io.h"
#include "mixer_kernels.h"

namespace lcv {
namespace {

// ---- matrix-core operands -------------------------------------------------------------------

template <int IO> struct Mx {  // bf16, fp16
    using E = uint16_t;
    static constexpr int C = 32;        // tokens of a chunk
    static constexpr int TK = 2;        // 16-wide tiles of one contraction step
    static constexpr int PADR = 8;      // row padding in LDS, elements: rows 4 banks apart (row reads)
    static constexpr int PADT = 16;     // 8 banks apart (transposed reads)
    static constexpr int VEC = 8;       // elements of 16 bytes
    struct Frag { uint32_t w[4]; };
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
        const u32x4 av = {a.w[0], a.w[1], a.w[2], a.w[3]}, bv = {b.w[0], b.w[1], b.w[2], b.w[3]};
        if constexpr (IO == CT_BF16)
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av), __builtin_bit_cast(bf16x8, bv), c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, av), __builtin_bit_cast(f16x8, bv), c, 0, 0, 0);
    }
    // p: the lane's row + 4 g
    static __device__ __forceinline__ Frag load_row(const E* p, int t) {
        const uint2 lo = *(const uint2*)(p + 32 * t), hi = *(const uint2*)(p + 32 * t + 16);
        return Frag{{lo.x, lo.y, hi.x, hi.y}};
    }
    static __device__ __forceinline__ uint2 tr(const E* p) {
        typedef short s16x4 __attribute__((__vector_size__(8)));
        typedef __attribute__((address_space(3))) s16x4* P;
        return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p));
    }
    // the lane's start in a tile [rows][stride] for transposed reads (16 lanes read 4 rows of 16)
    static __device__ __forceinline__ int tr_start(int g, int x, int stride) { return (4 * g + (x >> 2)) * stride + (x & 3) * 4; }
    static __device__ __forceinline__ Frag load_tr(const E* p, int stride, int j) {
        const uint2 lo = tr(p + 32 * j * stride), hi = tr(p + (32 * j + 16) * stride);
        return Frag{{lo.x, lo.y, hi.x, hi.y}};
    }
    static __device__ __forceinline__ Frag pack(const f32x4* t) {
        return Frag{{pack2<IO>(t[0][0], t[0][1]), pack2<IO>(t[0][2], t[0][3]), pack2<IO>(t[1][0], t[1][1]),
                     pack2<IO>(t[1][2], t[1][3])}};
    }
    static __device__ __forceinline__ void unpack(const Frag& f, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = unpack_lo<IO>(f.w[i]);
            v[2 * i + 1] = unpack_hi<IO>(f.w[i]);
        }
    }
    static __device__ __forceinline__ Frag pack(const float* v) {
        return Frag{{pack2<IO>(v[0], v[1]), pack2<IO>(v[2], v[3]), pack2<IO>(v[4], v[5]), pack2<IO>(v[6], v[7])}};
    }
};

template <> struct Mx<CT_F32> {
    using E = float;
    static constexpr int C = 32, TK = 1, PADR = 4, PADT = 4, VEC = 4;
    struct Frag { f32x4 v; };
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag load_row(const E* p, int t) { return Frag{*(const f32x4*)(p + 16 * t)}; }
    static __device__ __forceinline__ int tr_start(int g, int x, int stride) { return 4 * g * stride + x; }
    static __device__ __forceinline__ Frag load_tr(const E* p, int stride, int j) {
        const E* q = p + 16 * j * stride;
        return Frag{{q[0], q[stride], q[2 * stride], q[3 * stride]}};
    }
    static __device__ __forceinline__ Frag pack(const f32x4* t) { return Frag{t[0]}; }
    static __device__ __forceinline__ void unpack(const Frag& f, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f.v[i];
    }
    static __device__ __forceinline__ Frag pack(const float* v) { return Frag{{v[0], v[1], v[2], v[3]}}; }
};

// 2^(14 - e) and its inverse for a magnitude of binade e: brings the magnitude below 2^15
__device__ __forceinline__ float to_f16_range(float m, float* back) {
    int e = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
    e = e < -100 ? -100 : e > 110 ? 110 : e;
    *back = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    return __uint_as_float((uint32_t)(127 + 14 - e) << 23);
}
// the largest of the four lanes x, x + 16, x + 32, x + 48
__device__ __forceinline__ float max_over_g(float m) {
    m = fmaxf(m, __shfl_xor(m, 16));
    return fmaxf(m, __shfl_xor(m, 32));
}

__device__ __forceinline__ float max_over_wave(float m) {
#pragma unroll
    for (int w = 1; w < 16; w *= 2) m = fmaxf(m, __shfl_xor(m, w));
    return max_over_g(m);
}

// ---- one segment of one (b, h), 64 NW columns -------------------------------------------------

// STATE: only the state that the segment adds up from zero, for the segments after it.
template <int IO, int KT, int NW, bool STATE>
__global__ void __launch_bounds__(256, KT > 8 ? 1 : 2) linattn_chunk_kernel(LinJob a) {
    using M = Mx<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    constexpr int C = M::C, TK = M::TK, CT = C / 16, CJ = CT / TK, KS = KT / TK, ES = TK * 4;
    constexpr int DKP = KT * 16, DVB = 64 * NW, RS = DKP + M::PADR, VS = DVB + M::PADT;
    constexpr int VEC = M::VEC, KV_ROW = DKP / VEC, V_ROW = DVB / VEC;   // 16-byte groups of a row
    constexpr int NK = (C * KV_ROW + 255) / 256, NV = C * V_ROW / 256;   // groups per thread
    static_assert(NV >= 1 && C * V_ROW % 256 == 0 && (NK == 1 || C * KV_ROW % 256 == 0), "whole passes");
    __shared__ __attribute__((aligned(16))) E Qs[STATE ? 8 : C * RS];
    __shared__ __attribute__((aligned(16))) E Ks[C * RS];
    __shared__ __attribute__((aligned(16))) E Vs[C * VS];

    const LinRole& r = a.r[blockIdx.y];
    const int ncb = (r.DV + DVB - 1) / DVB;
    int64_t id = blockIdx.x;
    const int cb = (int)(id % a.ncb);
    id /= a.ncb;
    if (cb >= ncb) return;
    const int nseg = STATE ? a.nseg - 1 : a.nseg;
    const int64_t bh = id / nseg;
    const int seg = (int)(id - bh * nseg);
    const int64_t b = bh / a.H;
    const int h = (int)(bh - b * a.H);
    const int64_t len = row_len(a.lengths, b, a.N);
    const int64_t beg = seg * a.seg_len;
    const int64_t end = beg + a.seg_len < len ? beg + a.seg_len : len;
    if (STATE && beg + a.seg_len >= len) return;   // no segment follows

    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, x = lane & 15;
    const int wcol = cb * DVB + wave * 16 * NW;             // the wave's first column
    const int64_t ob = b * r.o.b + (int64_t)h * r.o.h;
    const int osize = r.o_f32 ? 4 : (int)sizeof(E);

    if constexpr (!STATE) {
        // tokens past the row's length: zeros (16-byte groups of this workgroup's columns)
        const int per = 16 / osize;
        const int groups = ((r.DV - cb * DVB < DVB ? r.DV - cb * DVB : DVB)) / per;
        int64_t t0 = beg > len ? beg : len, t1 = beg + a.seg_len < a.N ? beg + a.seg_len : a.N;
        if (r.O && t1 > t0)
            for (int64_t i = tid; i < (t1 - t0) * groups; i += 256) {
                const int64_t t = t0 + i / groups;
                const int c = cb * DVB + (int)(i % groups) * per;
                *(uint4*)((char*)r.O + (ob + t * r.o.n + c) * osize) = make_uint4(0, 0, 0, 0);
            }
        if (end <= beg && !(seg == 0 && r.s_out)) return;
    }

    // ---- weights of the chunk's tokens
    const float lg = log_gamma(a.log_decay, h);
    const int off = r.reverse;
    float wP[CT][4], wI[CT], wU[CJ][ES];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        wI[t] = r.s_q * expf(lg * (float)(16 * t + x + 1 - off));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 16 * t + x - 4 * g - i;
            wP[t][i] = r.s_q * r.s_kv * expf(lg * (float)(e > 0 ? e : 0));
        }
    }

    // ---- the state that enters
    f32x4 S[KT][NW];
    {
        const bool from_ws = !STATE && a.nseg > 1;
        const int64_t size = (int64_t)r.DK * r.DV;
        const float* s = STATE ? nullptr : from_ws ? r.states + (bh * a.nseg + seg) * size : r.s_in ? r.s_in + bh * size : nullptr;
        const int srow = from_ws ? r.DV : r.s_row, scol = from_ws ? 1 : r.s_col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const int d = 16 * t + 4 * g, c = wcol + 16 * n + x;
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
                if (s && d < r.DK && c < r.DV) {
                    if (srow == 1) {
                        v = *(const f32x4*)(s + (int64_t)c * scol + d);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = s[(int64_t)(d + i) * srow + c];
                    }
                }
                S[t][n] = v;
            }
    }

    // ---- global loads of a chunk, one ahead of the arithmetic.  Each thread's groups keep their row in
    // the chunk and their columns, so their pointers only move on.
    const auto first = [&](const LinOperand& o, int row, int c) LCV_INLINE {
        const int64_t p = beg + row;
        return (const E*)o.p + row_base(o, b, h) + (r.reverse ? len - 1 - p : p) * o.s.n + c;
    };
    const int64_t dir = r.reverse ? -(int64_t)C : C;
    const E *pq[STATE ? 1 : NK], *pk[NK], *pv[NV];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int e = tid + 256 * i;
        pk[i] = first(r.K, e / KV_ROW, (e % KV_ROW) * VEC);
        if constexpr (!STATE) pq[i] = first(r.Q, e / KV_ROW, (e % KV_ROW) * VEC);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = tid + 256 * i;
        pv[i] = first(r.V, e / V_ROW, cb * DVB + (e % V_ROW) * VEC);
    }
    const bool kin = C * KV_ROW >= 256 || tid < C * KV_ROW;      // a narrow chunk leaves threads without a group
    const bool kon = kin && tid % KV_ROW * VEC < r.DK, von = cb * DVB + tid % V_ROW * VEC < r.DV;  // 256 is a multiple of both
    uint4 rq[STATE ? 1 : NK], rk[NK], rv[NV];
    const auto fetch = [&](int64_t left) LCV_INLINE {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const bool on = kon && (tid + 256 * i) / KV_ROW < left;
            rk[i] = on ? *(const uint4*)pk[i] : make_uint4(0, 0, 0, 0);
            pk[i] += dir * r.K.s.n;
            if constexpr (!STATE) {
                rq[i] = on ? *(const uint4*)pq[i] : make_uint4(0, 0, 0, 0);
                pq[i] += dir * r.Q.s.n;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool on = von && (tid + 256 * i) / V_ROW < left;
            rv[i] = on ? *(const uint4*)pv[i] : make_uint4(0, 0, 0, 0);
            pv[i] += dir * r.V.s.n;
        }
    };
    const auto stage = [&]() LCV_INLINE {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int e = tid + 256 * i, row = e / KV_ROW, c = (e % KV_ROW) * VEC;
            if (!kin) continue;
            *(uint4*)(Ks + row * RS + c) = rk[i];
            if constexpr (!STATE) *(uint4*)(Qs + row * RS + c) = rq[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + 256 * i, row = e / V_ROW, c = (e % V_ROW) * VEC;
            *(uint4*)(Vs + row * VS + c) = rv[i];
        }
    };

    const E* qrow = Qs + (STATE ? 0 : x * RS + 4 * g);
    const E* krow = Ks + x * RS + 4 * g;
    const E* ktr = Ks + M::tr_start(g, x, RS);
    const E* vtr = Vs + M::tr_start(g, x, VS) + wave * 16 * NW;
    // the lane's place in the output: token x of the chunk, the first of its four columns
    const int64_t odir = r.reverse ? -r.o.n : r.o.n;
    int64_t oat = STATE ? 0 : ob + (r.reverse ? len - 1 - beg : beg) * r.o.n + x * odir + wcol + 4 * g;

    float em1 = 0.f;
    const auto weigh = [&](int c) LCV_INLINE {
        em1 = expm1f(lg * (float)c);
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int s = 0; s < ES; ++s) {
                const int tok = 16 * TK * j + 16 * (s >> 2) + 4 * g + (s & 3);
                const int e = c - 1 - tok + off;     // past the row's end V is zero; the power is kept finite
                wU[j][s] = r.s_kv * expf(lg * (float)(e > 0 ? e : 0));
            }
    };

    const auto chunk = [&](int c) LCV_INLINE {
        Frag vf[CJ][NW];
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int n = 0; n < NW; ++n) vf[j][n] = M::load_tr(vtr + 16 * n, VS, j);

        if constexpr (!STATE) {
            Frag qf[CT][KS], kf[CT][KS], sf[KS][NW];
#pragma unroll
            for (int it = 0; it < CT; ++it)
#pragma unroll
                for (int t = 0; t < KS; ++t) {
                    qf[it][t] = M::load_row(qrow + 16 * it * RS, t);
                    kf[it][t] = M::load_row(krow + 16 * it * RS, t);
                }
            float sback[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                float to = 1.f;
                sback[n] = 1.f;
                if constexpr (IO == CT_F16) {
                    float m = 0.f;
#pragma unroll
                    for (int t = 0; t < KT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[t][n][i]));
                    to = to_f16_range(max_over_wave(m), &sback[n]);
                }
#pragma unroll
                for (int t = 0; t < KS; ++t) {
                    f32x4 u[TK];
#pragma unroll
                    for (int k = 0; k < TK; ++k) u[k] = IO == CT_F16 ? S[TK * t + k][n] * to : S[TK * t + k][n];
                    sf[t][n] = M::pack(u);
                }
            }
            f32x4 acc[CT][NW], p[CT][CT];
#pragma unroll
            for (int it = 0; it < CT; ++it) {
#pragma unroll
                for (int n = 0; n < NW; ++n) acc[it][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int jt = 0; jt < CT; ++jt) p[it][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int it = 0; it < CT; ++it) {
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt) p[it][jt] = M::mma(kf[jt][t], qf[it][t], p[it][jt]);
#pragma unroll
                    for (int n = 0; n < NW; ++n) acc[it][n] = M::mma(sf[t][n], qf[it][t], acc[it][n]);
                }
#pragma unroll
            for (int it = 0; it < CT; ++it) {
#pragma unroll
                for (int n = 0; n < NW; ++n) acc[it][n] *= IO == CT_F16 ? wI[it] * sback[n] : wI[it];
#pragma unroll
                for (int jt = 0; jt <= it; ++jt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // later tokens are left out, not weighed with 0: they may not be finite
                        p[it][jt][i] = jt < it || x >= 4 * g + i ? p[it][jt][i] * wP[it - jt][i] : 0.f;
                if constexpr (IO == CT_F16) {
                    float m = 0.f, back;
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(p[it][jt][i]));
                    const float to = to_f16_range(max_over_g(m), &back);
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt) p[it][jt] *= to;
#pragma unroll
                    for (int n = 0; n < NW; ++n) {
                        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j <= it / TK; ++j) o = M::mma(vf[j][n], M::pack(p[it] + TK * j), o);
                        acc[it][n] += o * back;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j <= it / TK; ++j) {
                        const Frag pf = M::pack(p[it] + TK * j);
#pragma unroll
                        for (int n = 0; n < NW; ++n) acc[it][n] = M::mma(vf[j][n], pf, acc[it][n]);
                    }
                }
            }
#pragma unroll
            for (int it = 0; it < CT; ++it) {
                if (16 * it + x >= c) continue;
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    if (wcol + 16 * n + 4 * g >= r.DV) continue;
                    const int64_t o = oat + 16 * it * odir + 16 * n;
                    const f32x4 y = acc[it][n];
                    if (IO == CT_F32 || r.o_f32) *(f32x4*)((float*)r.O + o) = y;
                    else *(uint2*)((uint16_t*)r.O + o) = make_uint2(pack2<IO == CT_F32 ? CT_BF16 : IO>(y[0], y[1]),
                                                                    pack2<IO == CT_F32 ? CT_BF16 : IO>(y[2], y[3]));
                }
            }
            oat += C * odir;
        }

        // ---- the state moves on
        constexpr int PARTS = IO == CT_F32 ? 1 : IO == CT_F16 ? 2 : 3;
        Frag u[PARTS][CJ][NW];
        float back[NW];
#pragma unroll
        for (int n = 0; n < NW; ++n) {
            float v[CJ][ES], m = 0.f;
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                M::unpack(vf[j][n], v[j]);
#pragma unroll
                for (int s = 0; s < ES; ++s) {
                    v[j][s] *= wU[j][s];
                    if constexpr (IO == CT_F16) m = fmaxf(m, fabsf(v[j][s]));
                }
            }
            if constexpr (IO == CT_F16) {
                const float to = to_f16_range(max_over_g(m), &back[n]);
#pragma unroll
                for (int j = 0; j < CJ; ++j)
#pragma unroll
                    for (int s = 0; s < ES; ++s) v[j][s] *= to;
            }
#pragma unroll
            for (int j = 0; j < CJ; ++j)
#pragma unroll
                for (int k = 0; k < PARTS; ++k) {
                    u[k][j][n] = M::pack(v[j]);
                    if (k + 1 < PARTS) {
                        float q[ES];
                        M::unpack(u[k][j][n], q);
#pragma unroll
                        for (int s = 0; s < ES; ++s) v[j][s] -= q[s];
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            f32x4 d[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) d[n] = IO == CT_F16 ? f32x4{0.f, 0.f, 0.f, 0.f} : S[t][n] + S[t][n] * em1;
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                const Frag kt = M::load_tr(ktr + 16 * t, RS, j);
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
#pragma unroll
                    for (int n = 0; n < NW; ++n) d[n] = M::mma(kt, u[k][j][n], d[n]);
            }
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                if constexpr (IO == CT_F16) S[t][n] += S[t][n] * em1 + d[n] * back[n];
                else S[t][n] = d[n];
            }
        }
    };

    if (beg < end) {
        fetch(end - beg);
        weigh(C);
    }
    int64_t at = beg;
    for (; at + C <= end; at += C) {
        __syncthreads();
        stage();
        __syncthreads();
        if (at + C < end) fetch(end - at - C);
        chunk(C);
    }
    if (at < end) {
        const int c = (int)(end - at);
        __syncthreads();
        stage();
        weigh(c);
        __syncthreads();
        chunk(c);
    }

    // ---- the state that leaves
    float* s = nullptr;
    int srow = r.DV, scol = 1;
    if constexpr (STATE) {
        s = r.states + (bh * a.nseg + seg + 1) * (int64_t)r.DK * r.DV;
    } else if (r.s_out && (end == len || len == 0) && (beg < len || seg == 0)) {
        s = r.s_out + bh * (int64_t)r.DK * r.DV;
        srow = r.s_row;
        scol = r.s_col;
    }
    if (s) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const int d = 16 * t + 4 * g, c = wcol + 16 * n + x;
                if (d >= r.DK || c >= r.DV) continue;
                if (srow == 1) {
                    *(f32x4*)(s + (int64_t)c * scol + d) = S[t][n];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[(int64_t)(d + i) * srow + c] = S[t][n][i];
                }
            }
    }
}

template <int IO, int KT, int NW>
hipError_t launch_chunk(const LinJob& a, hipStream_t stream) {
    const int64_t rows = a.B * a.H;
    if (a.nseg > 1) {
        linattn_chunk_kernel<IO, KT, NW, true><<<dim3((unsigned)(rows * (a.nseg - 1) * a.ncb), a.nroles), 256, 0, stream>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        e = launch_linattn_join(a, stream);
        if (e != hipSuccess) return e;
    }
    linattn_chunk_kernel<IO, KT, NW, false><<<dim3((unsigned)(rows * a.nseg * a.ncb), a.nroles), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <int IO>
hipError_t launch_chunk_io(const LinJob& a, hipStream_t stream) {
    const int k = a.kt, n = a.nw;
    if (k == 2) return n == 1 ? launch_chunk<IO, 2, 1>(a, stream) : launch_chunk<IO, 2, 2>(a, stream);
    if (k == 4) return n == 1 ? launch_chunk<IO, 4, 1>(a, stream) : launch_chunk<IO, 4, 2>(a, stream);
    if (k == 8) return n == 1 ? launch_chunk<IO, 8, 1>(a, stream) : launch_chunk<IO, 8, 2>(a, stream);
    return n == 1 ? launch_chunk<IO, 16, 1>(a, stream) : launch_chunk<IO, 16, 2>(a, stream);
}

}  // namespace
}  // namespace lcv
