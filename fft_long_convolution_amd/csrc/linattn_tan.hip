// linattn_tan.hip -- the gradient of linear attention's decay.
//
// With T_t = dS_t / dlog(gamma) = gamma (T_{t-1} + S_{t-1}) the gradient is scale sum_t (T_t^T q_t) . dy_t + <T_L, dstate_out>.
// For a chunk of C tokens with S and T entering it, i and j counted from its first token:
//   sum_{j < i} (i - j) gamma^(i-j) (q_i . k_j) (v_j . dy_i)  +  sum_i gamma^(i+1) (T^T q_i + (i + 1) S^T q_i) . dy_i
//   S <- gamma^c S + sum_j gamma^(c-1-j) k_j v_j^T
//   T <- gamma^c (T + c S) + sum_j (c-1-j) gamma^(c-1-j) k_j v_j^T
// The first sum is an element by element product of two score matrices, K Q^T and V dY^T, whose accumulators have the same
// layout, so it takes no third product.  A workgroup of four waves holds 64 columns of S and T in registers and walks a
// (b, h), or a segment of it; what it adds is linear in its columns of V and dY.  Long rows are split into segments as in the
// forward: a pass over the segments' own S and T, a scan, and the main pass.
// The sum's terms have either sign, so that one 16-bit rounding of its operands would show in the fp32 result: bf16 data
// multiplies as it is, S, T and the weighted V in two bf16 parts (2^-17); fp16 and fp32 data go through fp32 products.
// Bound by the chain of a chunk's products and waits, two waves to a SIMD (bf16 at one wave, with the accumulators moved
// between register files, took a third longer).  Measured beside the other gradients, D = 128 (us more): 128 rows of 2048
// tokens in bf16 132, in fp16 546, in fp32 573; 32 rows of 4096 92, 334, 359 -- fp32 products take sixteen times bf16's time.
#include "linattn_tiles.h"
#include "mixer_plan.h"

namespace lcv {
namespace {

template <int IO, int KT, bool STATE>
__global__ void __launch_bounds__(256, KT <= (IO == CT_BF16 ? 8 : 4) ? 2 : 1) linattn_tan_kernel(LinTanArgs a) {
    using M = Mx<IO == CT_BF16 ? CT_BF16 : CT_F32>;
    using E = typename M::E;
    using Frag = typename M::Frag;
    constexpr int C = M::C, TK = M::TK, VEC = M::VEC, CT = C / 16, CJ = CT / TK, KS = KT / TK, ES = 4 * TK;
    constexpr int RK = KT * 16 / VEC, RV = 64 / VEC, RS = 4 / TK;     // 16-byte groups of a row; contraction steps of 64 columns
    constexpr int NK = (C * RK + 255) / 256, NV = C * RV / 256, PARTS = IO == CT_BF16 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) char Lq[STATE ? 16 : C * RK * 16], Lk[C * RK * 16], Lv[C * RV * 16], Ly[STATE ? 16 : C * RV * 16];
    __shared__ float red[4];

    // 32-bit divisions, which stay in scalar registers like the addresses that come from them
    const uint32_t ncb = linattn_tan_blocks(a.DV), nseg = STATE ? a.nseg - 1 : a.nseg;
    const uint32_t group = blockIdx.x / ncb, row = group / nseg, brow = row / (uint32_t)a.H;
    const int cb = (int)(blockIdx.x - group * ncb), seg = (int)(group - row * nseg), h = (int)(row - brow * (uint32_t)a.H);
    const int64_t b = brow, bh = row;
    const int64_t len = row_len(a.lengths, b, a.N), beg = seg * a.seg_len;
    const int64_t end = beg + a.seg_len < len ? beg + a.seg_len : len;
    if (STATE && beg + a.seg_len >= len) return;   // no segment follows
    float* const part = a.part + (((int64_t)h * a.B + b) * a.nseg + seg) * ncb + cb;
    if (end <= beg) {                              // T is zero where there are no tokens at all
        if (!STATE && threadIdx.x == 0) *part = 0.f;
        return;
    }
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, x = lane & 15;
    const int col = cb * 64 + wave * 16 + x;       // the lane's column of S and T
    const float lg = log_gamma(a.log_decay, h);
    const int64_t size = (int64_t)a.DK * a.DV;
    // byte offset of the lane's row i of tile k in a state
    const auto at = [&](int k, int i) LCV_INLINE {
        const int d = M::state_row(k, g);
        return only_if(d < a.DK & col < a.DV, (uint32_t)((d + i) * a.DV + col) * 4);
    };

    f32x4 S[KT], T[KT];
    {
        const float* s = STATE ? nullptr : a.nseg > 1 ? a.states + (bh * a.nseg + seg) * 2 * size : a.s_in ? a.s_in + bh * size : nullptr;
        const float* t = !STATE && a.nseg > 1 ? s + size : nullptr;
#pragma unroll
        for (int k = 0; k < KT; ++k) S[k] = T[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (s)
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[k][i] = load_f32(s, at(k, i));
        if (t)
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) T[k][i] = load_f32(t, at(k, i));
    }
    // weights: (i - j) gamma^(i-j) of a pair, the token's place and gamma^place against the state that enters
    float wD[CT][4], nI[CT], wI[CT], wU[CJ][ES], nU[CJ][ES], cgc = 0.f;
    float g_hi = 0.f, g_lo = 0.f, g_owed = 0.f;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        nI[t] = (float)(16 * t + x + 1);
        wI[t] = decay_power(lg, nI[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 16 * t + x - 4 * g - i;
            wD[t][i] = e > 0 ? (float)e * decay_power(lg, (float)e) : 0.f;
        }
    }
    const auto weigh = [&](int c) LCV_INLINE {
        g_hi = decay_power(lg, (float)c);
        g_lo = g_owed = 0.f;
        cgc = (float)c * decay_power(lg, (float)c);
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int s = 0; s < ES; ++s) {
                const int e = c - 1 - (16 * TK * j + 16 * (s >> 2) + 4 * g + (s & 3));    // past the row's end V is zero
                nU[j][s] = (float)(e > 0 ? e : 0);
                wU[j][s] = decay_power(lg, nU[j][s]);
            }
    };

    // A chunk on its way in registers, as stored (fp16: 8 bytes to a group of 4).  A lane without a row or a column loads
    // from past the buffer's end, which gives zeros: no lane leaves the wave, here as for the states.  (With branches
    // round these loads the widest heads' kernel, its registers all taken, had a value that every lane needs later moved
    // to another register inside a branch, for the branch's lanes alone.)
    typedef typename std::conditional<IO == CT_F16, uint2, uint4>::type Raw;
    struct Chunk { Raw q[STATE ? 1 : NK], k[NK], v[NV], y[STATE ? 1 : NV]; };
    const auto get = [&](const LinOperand& o, int slot, int R, int rows, int c0, int D, int64_t t0) LCV_INLINE {
        constexpr uint32_t es = IO == CT_F32 ? 4 : 2;
        const int row = slot / R, c = c0 + slot % R * VEC;
        const char* const base = (const char*)o.p + (row_base(o, b, h) + t0 * o.s.n) * es;
        const uint32_t off = only_if(row < rows & c < D, (uint32_t)row * (uint32_t)(o.s.n * es) + (uint32_t)c * es);
        if constexpr (IO == CT_F16) return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b64(buffer_at(base), off, 0, 0));
        else return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b128(buffer_at(base), off, 0, 0));
    };
    const auto load = [&](Chunk& f, int64_t t0) LCV_INLINE {
        const int rows = (int)(end - t0 < C ? end - t0 : C);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            f.k[i] = get(a.k, 256 * i + tid, RK, rows, 0, a.DK, t0);
            if constexpr (!STATE) f.q[i] = get(a.q, 256 * i + tid, RK, rows, 0, a.DK, t0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f.v[i] = get(a.v, 256 * i + tid, RV, rows, cb * 64, a.DV, t0);
            if constexpr (!STATE) f.y[i] = get(a.dy, 256 * i + tid, RV, rows, cb * 64, a.DV, t0);
        }
    };
    const auto put = [&](char* tile, int slot, int R, const Raw& r) LCV_INLINE {
        const int row = slot / R;
        if (C * R % 256 != 0 && row >= C) return;      // a narrow tile takes fewer lanes
        char* const p = tile + row * R * 16 + ((slot % R) ^ swizzle(row, R)) * 16;
        if constexpr (IO == CT_F16)
            *(f32x4*)p = f32x4{unpack_lo<CT_F16>(r.x), unpack_hi<CT_F16>(r.x), unpack_lo<CT_F16>(r.y), unpack_hi<CT_F16>(r.y)};
        else
            *(uint4*)p = r;
    };
    const auto store = [&](const Chunk& f) LCV_INLINE {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            put(Lk, 256 * i + tid, RK, f.k[i]);
            if constexpr (!STATE) put(Lq, 256 * i + tid, RK, f.q[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            put(Lv, 256 * i + tid, RV, f.v[i]);
            if constexpr (!STATE) put(Ly, 256 * i + tid, RV, f.y[i]);
        }
    };

    const typename M::At lk = M::at(g, x, RK), lv = M::at(g, x, RV);
    float tan = 0.f;
    Chunk f;
    load(f, beg);
    weigh(end - beg < C ? (int)(end - beg) : C);
    if (end - beg >= C) {      // a last, shorter chunk has a factor of its own
        const DecayPair gc = decay_pair(lg, (float)C);
        g_hi = uniform(gc.hi);
        g_lo = uniform(gc.lo);
    }
    for (int64_t t0 = beg; t0 < end; t0 += C) {
        const int c = (int)(end - t0 < C ? end - t0 : C);
        if (c < C) weigh(c);
        __syncthreads();                           // the last chunk has been read
        store(f);
        __syncthreads();
        if (t0 + C < end) load(f, t0 + C);

        if constexpr (!STATE) {
            f32x4 aS[CT], aT[CT], p[CT][CT];
#pragma unroll
            for (int it = 0; it < CT; ++it) {
                aS[it] = aT[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int jt = 0; jt < CT; ++jt) p[it][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                Frag qf[CT];
#pragma unroll
                for (int it = 0; it < CT; ++it) qf[it] = M::load_row(Lq + 16 * it * RK * 16, lk, t);
                const auto state = [&](const f32x4* s, f32x4* acc) LCV_INLINE {
                    float v[ES];
#pragma unroll
                    for (int e = 0; e < ES; ++e) v[e] = s[e >> 2][e & 3];
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        const Frag w = M::pack(v);
#pragma unroll
                        for (int it = 0; it < CT; ++it) acc[it] = M::mma(w, qf[it], acc[it]);
                        if (k + 1 < PARTS) {
                            float q[ES];
                            M::unpack(w, q);
#pragma unroll
                            for (int e = 0; e < ES; ++e) v[e] -= q[e];
                        }
                    }
                };
                state(S + TK * t, aS);
                state(T + TK * t, aT);
                if (wave < RS) {                   // a wave's step of V dY^T's columns; the others have none
#pragma unroll
                    for (int jt = 0; jt < CT; ++jt) {
                        const Frag kf = M::load_row(Lk + 16 * jt * RK * 16, lk, t);
#pragma unroll
                        for (int it = jt; it < CT; ++it) p[it][jt] = M::mma(kf, qf[it], p[it][jt]);
                    }
                }
            }
            if (wave < RS) {
                const char *const lvw = Lv, *const lyw = Ly;
                Frag vf[CT], yf[CT];
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    vf[it] = M::load_row(lvw + 16 * it * RV * 16, lv, wave);
                    yf[it] = M::load_row(lyw + 16 * it * RV * 16, lv, wave);
                }
#pragma unroll
                for (int it = 0; it < CT; ++it)
#pragma unroll
                    for (int jt = 0; jt <= it; ++jt) {
                        const f32x4 r = M::mma(vf[jt], yf[it], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tan += jt < it || x > 4 * g + i ? p[it][jt][i] * r[i] * wD[it - jt][i] : 0.f;
                    }
            }
            // dy of token x of the tile, columns 4 g .. 4 g + 3 of the wave's 16
#pragma unroll
            for (int it = 0; it < CT; ++it) {
                const int row = 16 * it + x, e = 16 * wave + 4 * g;
                const char* const at = Ly + row * RV * 16 + ((e / VEC) ^ swizzle(row, RV)) * 16 + e % VEC * (int)sizeof(E);
                float y[4];
                if constexpr (IO == CT_BF16) {
                    const uint2 w = *(const uint2*)at;
                    y[0] = unpack_lo<IO>(w.x); y[1] = unpack_hi<IO>(w.x); y[2] = unpack_lo<IO>(w.y); y[3] = unpack_hi<IO>(w.y);
                } else {
                    *(f32x4*)y = *(const f32x4*)at;
                }
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) s += (aT[it][i] + nI[it] * aS[it][i]) * y[i];
                tan += wI[it] * s;
            }
        }

        // ---- S and T move on
        Frag u[2][PARTS][CJ];
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            float v[ES], w[ES];
            M::unpack(M::load_v(Lv + j * TK * 16 * RV * 16, lv, wave, RV), v);
#pragma unroll
            for (int s = 0; s < ES; ++s) {
                v[s] *= wU[j][s];
                w[s] = v[s] * nU[j][s];
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                u[0][k][j] = M::pack(v);
                u[1][k][j] = M::pack(w);
                if (k + 1 < PARTS) {
                    float q[ES];
                    M::unpack(u[0][k][j], q);
#pragma unroll
                    for (int s = 0; s < ES; ++s) v[s] -= q[s];
                    M::unpack(u[1][k][j], q);
#pragma unroll
                    for (int s = 0; s < ES; ++s) w[s] -= q[s];
                }
            }
        }
        const float gc = next_decay(g_hi, g_lo, g_owed);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            T[t] = T[t] * gc + S[t] * cgc;
            S[t] = S[t] * gc;
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                const Frag kt = M::load_kt(Lk + j * TK * 16 * RK * 16, lk, t, RK);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) {
                    S[t] = M::mma(kt, u[0][k][j], S[t]);
                    T[t] = M::mma(kt, u[1][k][j], T[t]);
                }
            }
        }
    }

    if constexpr (STATE) {
        float* const s = a.states + (bh * a.nseg + seg + 1) * 2 * size;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                store_f32(s, at(t, i), S[t][i]);
                store_f32(s + size, at(t, i), T[t][i]);
            }
    } else {
        tan *= a.scale;
        if (a.ds_out && end == len) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) tan += T[t][i] * load_f32(a.ds_out + bh * size, at(t, i));
        }
        for (int w = 32; w; w >>= 1) tan += __shfl_xor(tan, w);
        if (lane == 0) red[wave] = tan;
        __syncthreads();
        if (tid == 0) *part = red[0] + red[1] + red[2] + red[3];
    }
}

// Slot s of a row's pairs (S, T) holds what segment s - 1 added up from zero; it becomes the pair that enters segment s.
__global__ void __launch_bounds__(256) linattn_tan_join_kernel(LinTanArgs a) {
    const int64_t size = (int64_t)a.DK * a.DV, i = (int64_t)blockIdx.x * 256 + threadIdx.x, bh = i / (size / 4);
    if (bh >= a.B * a.H) return;
    const int64_t e = (i - bh * (size / 4)) * 4, len = row_len(a.lengths, bh / a.H, a.N);
    f32x4 S = {0.f, 0.f, 0.f, 0.f}, T = S;
    if (a.s_in) S = *(const f32x4*)(a.s_in + bh * size + e);
    float* const st = a.states + bh * a.nseg * 2 * size + e;
    *(f32x4*)st = S;
    *(f32x4*)(st + size) = T;
    const float lg = log_gamma(a.log_decay, (int)(bh % a.H)), n = (float)a.seg_len, cgc = n * decay_power(lg, n);
    const DecayPair gamma = decay_pair(lg, n);
    for (int s = 1; s < a.nseg && s * a.seg_len < len; ++s) {
        float* const p = st + s * 2 * size;
        T = decayed(T, gamma, S * cgc + *(const f32x4*)(p + size));
        S = decayed(S, gamma, *(const f32x4*)p);
        *(f32x4*)p = S;
        *(f32x4*)(p + size) = T;
    }
}

__global__ void __launch_bounds__(64) linattn_tan_sum_kernel(const float* part, float* dlog, int64_t n) {
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < n; i += 64) s += part[blockIdx.x * n + i];
    for (int w = 32; w; w >>= 1) s += __shfl_xor(s, w);
    if (threadIdx.x == 0) dlog[blockIdx.x] = s;
}

template <int IO, int KT> hipError_t go(const LinTanArgs& a, hipStream_t stream) {
    const int64_t rows = a.B * a.H, ncb = linattn_tan_blocks(a.DV);
    if (a.nseg > 1) {
        linattn_tan_kernel<IO, KT, true><<<(unsigned)(rows * (a.nseg - 1) * ncb), 256, 0, stream>>>(a);
        const int64_t threads = rows * ((int64_t)a.DK * a.DV / 4);
        linattn_tan_join_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(a);
    }
    linattn_tan_kernel<IO, KT, false><<<(unsigned)(rows * a.nseg * ncb), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <int IO> hipError_t go(const LinTanArgs& a, hipStream_t stream) {
    const int kt = linattn_kt(a.DK);
    return kt == 2 ? go<IO, 2>(a, stream) : kt == 4 ? go<IO, 4>(a, stream) : kt <= 8 ? go<IO, 8>(a, stream) : go<IO, 16>(a, stream);
}

}  // namespace

hipError_t launch_linattn_tan(int dtype, const LinTanArgs& a, float* dlog, hipStream_t stream) {
    const hipError_t e = dtype == LCONV_F32 ? go<CT_F32>(a, stream) : dtype == LCONV_F16 ? go<CT_F16>(a, stream) : go<CT_BF16>(a, stream);
    if (e != hipSuccess) return e;
    linattn_tan_sum_kernel<<<(unsigned)a.H, 64, 0, stream>>>(a.part, dlog, a.B * a.nseg * linattn_tan_blocks(a.DV));
    return hipGetLastError();
}

}  // namespace lcv
