// linattn_chunk.h -- linear attention with a decay for each head, by chunks on the matrix cores
// (instantiated per type in linattn_f32.hip, linattn_f16.hip and linattn_bf16.hip).
//
// A chunk of 32 tokens with the state S that enters it (gamma = exp(log_decay), r = 1 for the
// gradients' direction, else 0):
//   O_i = s_q ( s_kv sum_{j<=i} gamma^(i-j) (Q_i . K_j) V_j + gamma^(i+1-r) S^T Q_i )
//   S  <- gamma^c S + s_kv sum_j gamma^(c-1-j+r) K_j V_j^T
// One pass over the data: a workgroup walks its (b, h), or a segment of it, chunk by chunk with S in
// fp32 in the registers of its four waves; a wave owns 16 NW columns of S and of O, and every row.  Chunks come
// straight to LDS two ahead of the arithmetic.  Few long rows are split into segments: a pass that only adds up each
// segment's own state (K and V are read twice), a scan over them, and the main pass.  The segments' states stand in memory
// as they do in registers, 16 bytes to a lane (in rows, 4 bytes at a time, they cost the prompt below 3 us).
//
// How the four products follow each other in registers (lane = 16 g + x, tiles of 16 x 16, the
// accumulator holds rows 4 g + r, r < 4, of column x):
//   P^T  = K Q^T      accumulator: tokens j = 4g + r of query i = x, which is what the next product
//   O^T += V^T P^T    takes as its right operand (column i, contraction over j): no lane moves
//   O^T += S^T Q^T    S's accumulators (rows d = 4g + r, column n = x) are the left operand as they are
//   S   += K^T V      both operands stand transposed to their rows in LDS: ds_read_b64_tr_b16 for 16-bit
//                 types, four strided reads for fp32
// Every wave forms all of P (12 of its 64 matrix products for a bf16 chunk at D = 128 and NW = 2; for fp32 96 of 236 at
// NW = 1 and 96 of 376 at NW = 2) rather than share it through LDS and a barrier.
//
// What bounds it (bf16, D = 128; times of calls back to back, times of single passes from a trace, which runs them one at a
// time).  Enough rows (gradients, 256 rows of 2048 tokens, 285 us): HBM, 4.7 TB/s of what is read after the XCD's L2 has
// served the roles that walk together (7 tensors of the 9 asked for, by counters) and written.  65536 tokens of 16 rows
// (356 us): HBM; on average of 20 traced calls the state pass takes 143 us for 553 MB and the main pass 253 for 1.1 GB, at
// least 116 and 212 (5.2 TB/s).  A prompt of 32 rows of 4096 (66 us): 24 us of state pass, 8 of scan, 40 of main pass, which
// moves 154 MB in it; what is left to HBM's rate is the start and the end of workgroups that all begin at once.  One
// workgroup to a compute unit: a chunk's chain, about 1.25 us at NW = 2 and 0.9 at NW = 1, of some 275 vector instructions
// and 64 matrix products of a wave.  Eight waves that share one 128-column tile took the same time a chunk, since the SIMD's
// instructions add up, and 64 tokens to a chunk spilled registers.
//
// Precision.  S, P and every sum are fp32.  For 16-bit types P and S are rounded to the type once as
// operands, like the result itself.  What S adds up is not: gamma^.. V is split into three bf16 parts
// (two where no state leaves the call: 2^-17) or two fp16 parts, so that the state keeps fp32's accuracy over any length.
// fp16 operands that may pass its range (P, S, gamma^.. V) are scaled to it by a power of two, per query,
// per 16 columns and per column.  The state's factor gamma^c carries its rounding from chunk to chunk (next_decay), so that
// neither a decay near one nor a fast one loses by its power.
#pragma once
#include "linattn_tiles.h"
#include "mixer_plan.h"

namespace lcv {
namespace {

// ---- one segment of one (b, h), 64 NW columns -------------------------------------------------

// STATE: only the state that the segment adds up from zero, for the segments after it.  WIDE: some roles' O leaves in fp32.
// EXACT: the state's sums to fp32's accuracy.
template <int IO, int KT, int NW, bool STATE, bool WIDE, bool EXACT>
__global__ void __launch_bounds__(256, linattn_alone(KT, NW, IO == CT_F32) ? 1 : NW == 1 && KT <= (IO == CT_BF16 ? 8 : IO == CT_F16 ? 6 : 0) ? 3 : 2) linattn_chunk_kernel(LinJob a) {
    using M = Mx<IO>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    constexpr int C = M::C, TK = M::TK, CT = C / 16, CJ = CT / TK, KS = KT / TK, ES = TK * 4;
    constexpr int DKP = KT * 16, DVB = 64 * NW, VEC = M::VEC;
    // 16-byte groups of a row in LDS: a power of two for the swizzle, also where the tiles are 6 or 12
    constexpr int RK = lin_row_groups(DKP / VEC), RV = DVB / VEC;
    constexpr int QB = STATE ? 0 : C * RK * 16, KB = C * RK * 16, STAGE = QB + KB + C * RV * 16;
    constexpr int NK = C * RK / 256, NV = C * RV / 256;         // loads of a chunk: rounds of 4 waves x 64 lanes
    constexpr bool KHALF = NK == 0;                             // a narrow tile takes two waves
    constexpr int NKR = KHALF ? 1 : NK, LOADS = (STATE ? 1 : 2) * NKR + NV;   // of a wave
    // 16-bit data at NW = 2 deals a wave's columns to its two tiles in fours: a lane's accumulators are then 8
    // neighbours of a token, one 16-byte store, of which four lanes make 64 bytes (gradients of 128 rows of 2048
    // tokens 166 us; with stores of 8 bytes, 32 to a token, 182).
    constexpr bool FOURS = IO != CT_F32 && NW == 2;
    constexpr int PUTS = FOURS ? CT : CT * NW, STORES = STATE ? 0 : PUTS;     // of a wave; a wide FOURS put takes two
    static_assert(NV >= 1 && (NK >= 1 || C * RK == 128), "rounds of whole waves");
    constexpr int SURE = KHALF ? NV : LOADS;         // loads of a chunk that every wave issues
    // chunks in LDS: one in hand, and two on their way where a compute unit then still holds the workgroups
    // that its registers allow (NW = 1: three, which hide each other's loads)
    constexpr int STAGES = 3 * STAGE <= (linattn_alone(KT, NW, IO == CT_F32) ? 160 : NW == 1 && KT <= 8 ? 53 : 80) * 1024 ? 3 : 2;
    __shared__ __attribute__((aligned(16))) char lds0[STAGE], lds1[STAGE];
    char* lds2 = nullptr;
    if constexpr (STAGES == 3) {
        __shared__ __attribute__((aligned(16))) char third[STAGE];
        lds2 = third;
    }

    // Workgroups that read the same tokens (a segment's roles and column blocks) go to one XCD, whose L2
    // they share, and next to them the other heads of these tokens, which lie beside them in token-major memory:
    // consecutive ids go round the eight XCDs, each of which takes a row of groups (batch row, segment, head).
    // Measured against groups dealt to the XCDs in turn, heads outermost (us): prompt of 32 rows of 4096 64, 68; gradients
    // of 128 rows of 2048 157, 163 (head-major 149, 153); 16 rows of 65536 head-major 358, 359, token-major 374, 395.
    // Rows of different lengths are dealt out in turn all the same, or the XCDs of short rows would stand idle (30 rows
    // of 0 to 777 tokens 33, else 40).
    const uint32_t per = a.nroles * a.ncb, nseg = STATE ? a.nseg - 1 : a.nseg;    // 64-bit divisions take a microsecond
    const uint32_t slot = blockIdx.x / 8, groups = a.B * a.H * nseg, xcd = blockIdx.x % 8;
    const uint32_t group = a.lengths ? slot / per * 8 + xcd : xcd * ((groups + 7) / 8) + slot / per;
    if (group >= groups) return;
    const int member = (int)(slot % per), cb = member % a.ncb;
    const LinRole r = a.r[member / a.ncb];       // a copy: its fields stay in scalar registers
    if (cb * DVB >= r.DV) return;
    const uint32_t place = group / (uint32_t)a.H, brow = place / nseg;
    const int seg = (int)(place - brow * nseg), h = (int)(group - place * (uint32_t)a.H);
    const int64_t b = brow, bh = b * a.H + h;
    const int64_t len = row_len(a.lengths, b, a.N);
    const int64_t beg = seg * a.seg_len;
    const int64_t end = beg + a.seg_len < len ? beg + a.seg_len : len;
    if (STATE && beg + a.seg_len >= len) return;   // no segment follows

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, x = lane & 15;
    const int wcol = cb * DVB + wave * 16 * NW;             // the wave's first column
    const auto column = [&](int n) LCV_INLINE { return wcol + (FOURS ? 8 * (x >> 2) + 4 * n + (x & 3) : 16 * n + x); };   // tile n's column x
    const int64_t ob = b * r.o.b + (int64_t)h * r.o.h;

    const bool wide = IO == CT_F32 || (WIDE && r.wide);
    const int osz = wide ? 4 : 2;
    if constexpr (!STATE) {
        // tokens past the row's length: zeros (16-byte groups of this workgroup's columns)
        const int per = 16 / osz;
        const int groups = ((r.DV - cb * DVB < DVB ? r.DV - cb * DVB : DVB)) / per;
        int64_t t0 = beg > len ? beg : len, t1 = beg + a.seg_len < a.N ? beg + a.seg_len : a.N;
        if (t1 > t0)
            for (int64_t i = tid; i < (t1 - t0) * groups; i += 256) {
                const int64_t t = t0 + i / groups;
                const int c = cb * DVB + (int)(i % groups) * per;
                *(uint4*)((char*)r.O + (ob + t * r.o.n + c) * osz) = make_uint4(0, 0, 0, 0);
            }
        if (end <= beg && !(seg == 0 && r.s_out)) return;
    }

    // ---- loads of a chunk straight to LDS, two chunks ahead of the arithmetic.  Round i of a tile fills
    // 16-byte slots 256 i + 64 wave + lane; a slot's row and columns stay, so its pointer only moves on.
    // Its address is a scalar that moves on, at the chunk's lowest token, plus the lane's own offset.
    const int64_t low = r.reverse ? len - beg - C : beg, dir = r.reverse ? -(int64_t)C : C;
    const auto start = [&](const LinOperand& o) LCV_INLINE { return (const char*)o.p + (row_base(o, b, h) + low * o.s.n) * (int)sizeof(E); };
    const auto offset = [&](const LinOperand& o, int row, int c) LCV_INLINE {
        return (uint32_t)(r.reverse ? C - 1 - row : row) * (uint32_t)(o.s.n * (int)sizeof(E)) + (uint32_t)(c * (int)sizeof(E));
    };
    const char *pq = STATE ? nullptr : start(r.Q), *pk = start(r.K), *pv = start(r.V);
    const int64_t dq = dir * r.Q.s.n * (int)sizeof(E), dk = dir * r.K.s.n * (int)sizeof(E), dv = dir * r.V.s.n * (int)sizeof(E);
    // A lane without a column has an offset past the buffer's end, where loads give zeros and stores do nothing: every
    // wave issues every load and every store, so that their numbers are known.
    uint32_t oq[NKR], ok[NKR], ov[NV];
    const bool kin = !KHALF || wave < 2;
#pragma unroll
    for (int i = 0; i < NKR; ++i) {
        const int s = 256 * i + tid, row = s / RK % C, c = ((s % RK) ^ swizzle(row, RK)) * VEC;
        ok[i] = c < r.DK ? offset(r.K, row, c) : kNowhere;
        oq[i] = STATE || c >= r.DK ? kNowhere : offset(r.Q, row, c);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int s = 256 * i + tid, row = s / RV, c = cb * DVB + ((s % RV) ^ swizzle(row, RV)) * VEC;
        ov[i] = c < r.DV ? offset(r.V, row, c) : kNowhere;
    }
    if (r.DK < DKP || cb * DVB + DVB > r.DV) {       // columns that the operands do not have are zero
        for (int i = tid; i < STAGE / 16; i += 256) {
            *(uint4*)(lds0 + 16 * i) = make_uint4(0, 0, 0, 0);
            *(uint4*)(lds1 + 16 * i) = make_uint4(0, 0, 0, 0);
            if constexpr (STAGES == 3) *(uint4*)(lds2 + 16 * i) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
    }
    // load i of a whole chunk's LOADS
    const auto piece = [&](auto i, char* to) LCV_INLINE {
        constexpr int I = i.value, Q = STATE ? 0 : NKR;
        char* const t = to + 1024 * wave;
        if constexpr (I < Q + NKR) {
            if (kin) {
                if constexpr (I < Q) to_lds(pq, oq[I], t + 4096 * I);
                else to_lds(pk, ok[I - Q], t + QB + 4096 * (I - Q));
            }
        } else if constexpr (I < LOADS) {
            to_lds(pv, ov[I - Q - NKR], t + QB + KB + 4096 * (I - Q - NKR));
        }
    };
    const auto move_on = [&]() LCV_INLINE {
        if constexpr (!STATE) pq += dq;
        pk += dk;
        pv += dv;
    };
    const auto fetch = [&](char* to, int64_t left) LCV_INLINE {
        if (left >= C) {
            static_for<0, LOADS>([&](auto i) LCV_INLINE { piece(i, to); });
        } else {
            // zeros for the tokens that a last chunk lacks
            char* const t = to + 1024 * wave;
#pragma unroll
            for (int i = 0; i < NKR; ++i) {
                const bool in = (256 * i + tid) / RK % C < left;
                if (kin && in) {
                    if constexpr (!STATE) to_lds(pq, oq[i], t + 4096 * i);
                    to_lds(pk, ok[i], t + QB + 4096 * i);
                }
                if (kin && !in) {
                    if constexpr (!STATE) *(uint4*)(t + 4096 * i + 16 * lane) = make_uint4(0, 0, 0, 0);
                    *(uint4*)(t + QB + 4096 * i + 16 * lane) = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool in = (256 * i + tid) / RV < left;
                if (in) to_lds(pv, ov[i], t + QB + KB + 4096 * i);
                else *(uint4*)(t + QB + KB + 4096 * i + 16 * lane) = make_uint4(0, 0, 0, 0);
            }
        }
        move_on();
    };

    // the first chunks are on their way while the weights are formed and the state comes in
    int64_t left = end - beg;                  // tokens from the chunk in hand on
    if (left > 0) {
        fetch(lds0, left);
        if (STAGES == 3 && left > C) fetch(lds1, left - C);
    }

    // ---- weights of the chunk's tokens
    const float lg = log_gamma(a.log_decay, h);
    const int off = r.reverse;
    float wP[CT][4], wI[CT], wU[CJ][ES];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        wI[t] = r.s_q * decay_power(lg, (float)(16 * t + x + 1 - off));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 16 * t + x - 4 * g - i;
            wP[t][i] = r.s_q * r.s_kv * decay_power(lg, (float)(e > 0 ? e : 0));
        }
    }

    // ---- the state that enters.  The segments' states stand as they are in registers: tiles, 16 bytes to a lane.
    const auto state_tile = [&](int seg, int t, int n) LCV_INLINE {
        const int tiles = KT * 4 * NW * a.ncb, tile = ((cb * 4 + wave) * NW + n) * KT + t;
        return (f32x4*)(r.states + (((int64_t)bh * a.nseg + seg) * tiles + tile) * 256) + lane;
    };
    const auto has_tile = [&](int t, int n) LCV_INLINE { return M::state_row(t, 0) < r.DK && wcol + (FOURS ? 4 : 16) * n < r.DV; };
    f32x4 S[KT][NW];
    {
        const bool from_ws = !STATE && a.nseg > 1;
        const float* s = STATE || from_ws || !r.s_in ? nullptr : r.s_in + bh * ((int64_t)r.DK * r.DV);
        const int srow = r.s_row, scol = r.s_col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const int d = M::state_row(t, g), c = column(n);
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
                if (from_ws) {
                    if (has_tile(t, n)) v = *state_tile(seg, t, n);
                } else if (s && d < r.DK && c < r.DV) {
                    if (srow == 1) {
                        v = *(const f32x4*)(s + (int64_t)c * scol + d);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = s[(int64_t)(d + i) * srow + c];
                    }
                }
                if constexpr (IO == CT_F16) {      // an infinity would scale its 15 neighbours' columns to nothing; a NaN does not
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = fabsf(v[i]) == __builtin_inff() ? __uint_as_float(0x7fc00000u) : v[i];
                }
                S[t][n] = v;
            }
    }

    const typename M::At lk = M::at(g, x, RK), lv = M::at(g, x, RV);
    // the output likewise: lane x's token, the first of its columns; token tiles of 16 and column tiles
    // are steps of the scalar
    char* po = STATE ? nullptr : (char*)r.O + (ob + low * r.o.n) * osz;
    const int64_t d_o = dir * r.o.n * osz, o16 = 16 * r.o.n * osz;
    const int mine = wcol + (FOURS ? 8 : 4) * g;
    uint32_t oo[FOURS ? 1 : NW];
#pragma unroll
    for (int n = 0; n < (FOURS ? 1 : NW); ++n)
        oo[n] = mine + 16 * n < r.DV ? (uint32_t)(r.reverse ? 15 - x : x) * (uint32_t)(r.o.n * osz) + (uint32_t)(mine * osz) : kNowhere;

    float g_hi = 0.f, g_lo = 0.f, g_owed = 0.f;
    const auto weigh = [&](int c) LCV_INLINE {
        g_hi = decay_power(lg, (float)c);
        g_lo = g_owed = 0.f;
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int s = 0; s < ES; ++s) {
                const int tok = 16 * TK * j + 16 * (s >> 2) + 4 * g + (s & 3);
                const int e = c - 1 - tok + off;     // past the row's end V is zero; the power is kept finite
                wU[j][s] = r.s_kv * decay_power(lg, (float)(e > 0 ? e : 0));
            }
    };

    f32x4 acc[CT][NW];
    const auto put = [&](int i) LCV_INLINE {
        const int it = FOURS ? i : i / NW, n = FOURS ? 0 : i % NW;
        char* const at = po + (r.reverse ? CT - 1 - it : it) * o16 + 16 * n * osz;
        const f32x4 y = acc[it][n], y2 = acc[it][NW - 1];
        if (wide) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), buffer_at(at), oo[n], 0, 0);
            if constexpr (FOURS) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y2), buffer_at(at + 16), oo[n], 0, 0);
        } else if constexpr (FOURS) {
            const u32x4 w = {pack2<IO>(y[0], y[1]), pack2<IO>(y[2], y[3]), pack2<IO>(y2[0], y2[1]), pack2<IO>(y2[2], y2[3])};
            __builtin_amdgcn_raw_buffer_store_b128(w, buffer_at(at), oo[n], 0, 0);
        } else if constexpr (IO != CT_F32) {
            typedef uint32_t u32x2 __attribute__((__vector_size__(8)));
            const u32x2 w = {pack2<IO>(y[0], y[1]), pack2<IO>(y[2], y[3])};
            __builtin_amdgcn_raw_buffer_store_b64(w, buffer_at(at), oo[n], 0, 0);
        }
    };
    const auto emit = [&](int c) LCV_INLINE {
        if constexpr (!STATE) {
#pragma unroll
            for (int i = 0; i < PUTS; ++i)
                if (16 * (FOURS ? i : i / NW) + x < c) put(i);
            po += d_o;
        }
    };

    // One chunk.  FULL: a whole chunk with a whole one to fetch; its loads and its stores stand between the
    // products (issued in a row they hold the wave up, some 180 cycles a load).
    const auto chunk = [&](auto full, const char* L, char* then) LCV_INLINE {
        constexpr bool FULL = full.value;
        const char *const Lk = L + QB, *const Lv = L + QB + KB;
        Frag vf[CJ][NW];
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const char* const v = Lv + j * TK * 16 * RV * 16;
                vf[j][n] = FOURS ? M::load_kt(v, lv, wave * NW + n, RV) : M::load_v(v, lv, wave * NW + n, RV);
            }

        // gamma^.. V in parts that add up to its fp32 value
        constexpr int PARTS = IO == CT_F32 ? 1 : IO == CT_F16 || !EXACT ? 2 : 3;
        Frag u[PARTS][CJ][NW];
        float back[NW], none[NW];      // none: 0, or the NaN of a column whose V is not finite
#pragma unroll
        for (int n = 0; n < NW; ++n) none[n] = 0.f;
        const auto split = [&](int n) LCV_INLINE {
            float v[CJ][ES], m = 0.f;
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                M::unpack(vf[j][n], v[j]);
#pragma unroll
                for (int s = 0; s < ES; ++s) {
                    v[j][s] = fmaf(v[j][s], wU[j][s], none[n]);
                    if constexpr (IO == CT_F16) m = fmaxf(m, fabsf(v[j][s]));
                }
            }
            if constexpr (IO == CT_F16) {
                const float up = to_f16_range(max_over_g(m), &back[n]);
#pragma unroll
                for (int j = 0; j < CJ; ++j)
#pragma unroll
                    for (int s = 0; s < ES; ++s) v[j][s] *= up;
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
        };

        if constexpr (!STATE) {
            float to[NW], sback[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                to[n] = sback[n] = 1.f;
                if constexpr (IO == CT_F16) {
                    float m = 0.f;
#pragma unroll
                    for (int t = 0; t < KT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S[t][n][i]));
                    to[n] = to_f16_range(max_over_wave(m), &sback[n]);
                }
            }
            f32x4 p[CT][CT];
#pragma unroll
            for (int it = 0; it < CT; ++it) {
#pragma unroll
                for (int n = 0; n < NW; ++n) acc[it][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int jt = 0; jt < CT; ++jt) p[it][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            static_for<0, KS>([&](auto ti) LCV_INLINE {
                constexpr int t = ti.value;
                Frag qf[CT], kf[CT], sf[NW];
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    qf[it] = M::load_row(L + 16 * it * RK * 16, lk, t);
                    kf[it] = M::load_row(Lk + 16 * it * RK * 16, lk, t);
                }
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    f32x4 w[TK];
#pragma unroll
                    for (int k = 0; k < TK; ++k) w[k] = IO == CT_F16 ? S[TK * t + k][n] * to[n] : S[TK * t + k][n];
                    sf[n] = M::pack(w);
                }
                if constexpr (FULL) static_for<t * LOADS / KS, (t + 1) * LOADS / KS>([&](auto i) LCV_INLINE { piece(i, then); });
#pragma unroll
                for (int it = 0; it < CT; ++it) {
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt) p[it][jt] = M::mma(kf[jt], qf[it], p[it][jt]);
#pragma unroll
                    for (int n = 0; n < NW; ++n) acc[it][n] = M::mma(sf[n], qf[it], acc[it][n]);
                }
            });
            // A V that is not finite must not reach the queries before it, whose 0 in P times V is a NaN: it leaves the product, and
            // the later queries' column and the state's become NaN here.  In all other chunks it costs four vector
            // instructions for 16 bytes of V and a branch: prompt of 32 rows of 4096 66 -> 68 us, gradients of 128 rows of 2048 153 -> 155.
            float sum[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                sum[n] = 0.f;
#pragma unroll
                for (int j = 0; j < CJ; ++j) sum[n] = M::nan_of(vf[j][n], sum[n]);
            }
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(__builtin_isunordered(sum[0], sum[NW - 1])) != 0, 0)) {
                const float nan = __uint_as_float(0x7fc00000u);
                int ahead = 4 * g - x;               // of the lane's first token in a tile to its query
                asm volatile("" : "+v"(ahead));      // nothing of this is to be kept in registers through the other chunks
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    Frag bad[CJ];
                    float any = 0.f;
#pragma unroll
                    for (int j = 0; j < CJ; ++j) {
                        float v[ES], one[ES];
                        M::unpack(vf[j][n], v);
#pragma unroll
                        for (int e = 0; e < ES; ++e) {
                            one[e] = fabsf(v[e]) < __builtin_inff() ? 0.f : 1.f;
                            v[e] = one[e] != 0.f ? 0.f : v[e];
                            any = fmaxf(any, one[e]);
                        }
                        vf[j][n] = M::pack(v);
                        bad[j] = M::pack(one);
                    }
                    none[n] = max_over_g(any) != 0.f ? nan : 0.f;
                    // how many such tokens a query has behind it
#pragma unroll
                    for (int it = 0; it < CT; ++it) {
                        f32x4 behind = {0.f, 0.f, 0.f, 0.f}, w[CT];
#pragma unroll
                        for (int jt = 0; jt < CT; ++jt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[jt][i] = jt < it || (jt == it && ahead + i <= 0) ? 1.f : 0.f;
#pragma unroll
                        for (int j = 0; j < CJ; ++j) behind = M::mma(bad[j], M::pack(w + TK * j), behind);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[it][n][i] = behind[i] != 0.f ? nan : acc[it][n][i];
                    }
                }
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
                    float m = 0.f, pback;
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(p[it][jt][i]));
                    const float up = to_f16_range(max_over_g(m), &pback);
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt) p[it][jt] *= up;
#pragma unroll
                    for (int n = 0; n < NW; ++n) {
                        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j <= it / TK; ++j) o = M::mma(vf[j][n], M::pack(p[it] + TK * j), o);
                        acc[it][n] += o * pback;
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
        }
#pragma unroll
        for (int n = 0; n < NW; ++n) split(n);

        // The waits count on it that this chunk's loads, all issued by now, stay ahead of its stores, which follow: vector
        // memory operations do not cross here, anything else may.  (The built loops are checked for it by a test: without
        // this the compiler had put two stores ahead of four loads in the fp32 kernel of 192 x 128.)
        if constexpr (FULL && !STATE) __builtin_amdgcn_sched_barrier(0x78f);
        // ---- the state moves on
        const float gc = next_decay(g_hi, g_lo, g_owed);
        static_for<0, KT>([&](auto ti) LCV_INLINE {
            constexpr int t = ti.value;
            f32x4 d[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) d[n] = IO == CT_F16 ? f32x4{0.f, 0.f, 0.f, 0.f} : S[t][n] * gc;
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                const Frag kt = M::load_kt(Lk + j * TK * 16 * RK * 16, lk, t, RK);
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
#pragma unroll
                    for (int n = 0; n < NW; ++n) d[n] = M::mma(kt, u[k][j][n], d[n]);
            }
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                if constexpr (IO == CT_F16) S[t][n] = S[t][n] * gc + d[n] * back[n];
                else S[t][n] = d[n];
            }
            if constexpr (FULL && STATE) {
                static_for<t * LOADS / KT, (t + 1) * LOADS / KT>([&](auto i) LCV_INLINE { piece(i, then); });
            } else if constexpr (FULL) {
                static_for<t * PUTS / KT, (t + 1) * PUTS / KT>([&](auto i) LCV_INLINE { put(i.value); });
            }
        });
        if constexpr (FULL) {
            move_on();
            if constexpr (!STATE) po += d_o;
        }
    };

    // ---- the chunks.  A chunk's loads have to be in when it begins.
    if (left > 0) weigh(left < C ? (int)left : C);
    if (left >= C) {      // a last, shorter chunk has a factor of its own
        const DecayPair gc = decay_pair(lg, (float)C);
        g_hi = uniform(gc.hi);
        g_lo = uniform(gc.lo);
    }
    // STAGES chunks a turn, each stage by its own name: then the compiler knows which loads a read waits for.
    // Operations are counted in their order.  With three stages a chunk's loads are older than the stores of the two
    // chunks before it and the next chunk's loads, which may all be outstanding; with two stages older than the last
    // chunk's stores.  The first two chunks' loads have no such stores behind them and are waited for ahead of the loop.
    constexpr int LAST = STAGES == 3 ? 5 : 3;
    bool stored = false, ahead = false;        // a whole chunk's stores, and after them nothing; a whole fetch before them
    if (left >= LAST * C) {
        std::integral_constant<bool, true> full;
        wait_for_all_but<0>();
        const auto turn = [&](char* now, char* then) LCV_INLINE {
            wait_for_all_but<STAGES == 3 ? SURE + 2 * STORES : STORES>();
            barrier_only();
            chunk(full, now, then);
        };
        do {
            if constexpr (STAGES == 3) {
                turn(lds0, lds2);
                turn(lds1, lds0);
                turn(lds2, lds1);
            } else {
                turn(lds0, lds1);
                turn(lds1, lds0);
            }
            left -= STAGES * C;
        } while (left >= LAST * C);
        stored = true;
        ahead = STAGES == 3;
    }
    // the last chunks
    // (what a whole chunk issued after the next one's loads, its own stores and perhaps a whole fetch, is known and may
    // be outstanding)
    for (int t = 0; left > 0; left -= C) {
        char *now = lds0, *then = lds1;
        if constexpr (STAGES == 3) {
            if (t == 0) then = lds2;
            if (t == 1) { now = lds1; then = lds0; }
            if (t == 2) now = lds2;
        } else if (t == 1) {
            now = lds1;
            then = lds0;
        }
        if (ahead) wait_for_all_but<STAGES == 3 ? SURE + STORES : STORES>();
        else if (stored) wait_for_all_but<STORES>();
        else wait_for_all_but<0>();
        barrier_only();
        stored = true;
        ahead = STAGES == 3 && left >= STAGES * C;
        if (left > (STAGES - 1) * C) fetch(then, left - (STAGES - 1) * C);
        if (left < C && end - beg > C) weigh((int)left);
        chunk(std::integral_constant<bool, false>{}, now, nullptr);
        emit(left < C ? (int)left : C);
        t = t + 1 == STAGES ? 0 : t + 1;
    }

    // ---- the state that leaves
    if constexpr (STATE) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n)
                if (has_tile(t, n)) *state_tile(seg + 1, t, n) = S[t][n];
    } else if (r.s_out && (end == len || len == 0) && (beg < len || seg == 0)) {
        float* const s = r.s_out + bh * (int64_t)r.DK * r.DV;
        const int srow = r.s_row, scol = r.s_col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const int d = M::state_row(t, g), c = column(n);
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

template <int IO, int KT, int NW, bool WIDE, bool EXACT>
hipError_t launch_chunk_as(const LinJob& a, hipStream_t stream) {
    const int64_t rows = a.B * a.H;
    const auto grid = [&](int nseg) { return (unsigned)linattn_workgroups(LinPlan{a.kt, a.nw, a.ncb, nseg, a.seg_len}, rows, a.nroles); };
    if (a.nseg > 1) {
        linattn_chunk_kernel<IO, KT, NW, true, false, EXACT><<<grid(a.nseg - 1), 256, 0, stream>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        e = launch_linattn_join(a, IO == CT_F32, stream);
        if (e != hipSuccess) return e;
    }
    linattn_chunk_kernel<IO, KT, NW, false, WIDE, EXACT><<<grid(a.nseg), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <int IO, int KT, int NW>
hipError_t launch_chunk(const LinJob& a, hipStream_t stream) {
    // fp32 is wide as it is, and only bf16 has a third part to leave out
    constexpr bool W = IO != CT_F32, X = IO == CT_BF16;
    bool wide = false;
    for (int i = 0; i < a.nroles; ++i) wide |= W && a.r[i].wide;
    if (a.exact || !X) return wide ? launch_chunk_as<IO, KT, NW, W, true>(a, stream) : launch_chunk_as<IO, KT, NW, false, true>(a, stream);
    return wide ? launch_chunk_as<IO, KT, NW, W, !X>(a, stream) : launch_chunk_as<IO, KT, NW, false, !X>(a, stream);
}

template <int IO, int NW>
hipError_t launch_chunk_nw(const LinJob& a, hipStream_t stream) {
    if (a.kt == 2) return launch_chunk<IO, 2, NW>(a, stream);
    if (a.kt == 4) return launch_chunk<IO, 4, NW>(a, stream);
    if (a.kt == 6) return launch_chunk<IO, 6, NW>(a, stream);
    if (a.kt == 8) return launch_chunk<IO, 8, NW>(a, stream);
    if (a.kt == 12) return launch_chunk<IO, 12, NW>(a, stream);
    return launch_chunk<IO, 16, NW>(a, stream);
}

template <int IO> hipError_t launch_chunk_io(const LinJob& a, hipStream_t stream) {
    return a.nw == 1 ? launch_chunk_nw<IO, 1>(a, stream) : launch_chunk_nw<IO, 2>(a, stream);
}

}  // namespace
}  // namespace lcv
