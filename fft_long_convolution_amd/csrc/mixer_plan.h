// mixer_plan.h -- how a call of the mixer operators is cut into workgroups (host arithmetic only).
#pragma once
#include <stdint.h>

#include "lconv.h"

namespace lcv {

// Linear attention: tiles of the contraction (16 wide, padded to 2, 4, 6, 8, 12 or 16), 16-column tiles per
// wave, column blocks of 64 nw, and segments of seg_len tokens that a (b, h) is split into.
struct LinPlan {
    int kt, nw, ncb, nseg;
    int64_t seg_len;
};

inline int linattn_kt(int64_t DK) { return DK <= 32 ? 2 : DK <= 64 ? 4 : DK <= 96 ? 6 : DK <= 128 ? 8 : DK <= 192 ? 12 : 16; }

// Microseconds that a workgroup alone on its compute unit takes for a chunk of 32 tokens, measured: a chunk's chain of waits
// is much the same for narrow heads; fp16 scales its operands; fp32's matrix products take sixteen times as long.
inline double linattn_chunk_us(int kt, int nw, lconv_dtype_t dtype) {
    static const double us[3][5][2] = {     // contraction of 32, 64, 96 and 128, 192, 256; 64 and 128 columns
        {{2.0, 3.0}, {3.0, 4.5}, {3.9, 6.4}, {6.0, 10.0}, {7.8, 12.8}},       // fp32
        {{0.7, 0.9}, {1.25, 1.75}, {1.5, 2.4}, {2.1, 3.1}, {2.5, 4.0}},       // fp16
        {{0.45, 0.6}, {0.9, 1.2}, {0.95, 1.25}, {1.2, 2.0}, {1.55, 2.45}}};   // bf16
    return us[dtype == LCONV_F32 ? 0 : dtype == LCONV_F16 ? 1 : 2][kt == 2 ? 0 : kt == 4 ? 1 : kt <= 8 ? 2 : kt == 12 ? 3 : 4][nw - 1];
}

// Whether a compute unit holds one workgroup at most: the widest heads and fp32 at 128 columns fill its registers and LDS.
constexpr bool linattn_alone(int kt, int nw, bool f32) { return kt == 16 || (kt == 12 && (nw == 2 || f32)) || (nw == 2 && f32); }

// Chosen by estimated time over the two tile widths and powers of two of segments.  With n chunks in a segment and L
// workgroups on a compute unit (256 of them),
//   main pass   2 us and n chunks of linattn_chunk_us, 1 + 0.35 (L - 1) as long where they share the unit (L where they
//               cannot), but no less than the tokens' bytes at 4.8 TB/s (4.2 where several column blocks read Q and K,
//               less 8 % for a single workgroup to a unit); three roles share some of what they read in the L2
//   more than one segment adds the state pass, 0.65 of that, 12 us for its two launches, and the segments'
//   states, written and read twice, at 8 TB/s.
// Both sides measured (us): bf16 D = 128, 32 rows N 4096: one segment 128, 4: 76, 8: 70, 16: 76; 128 rows N 2048: 1: 82, 2: 111;
// gradients of 256 rows N 2048: 64 columns 340, 128 columns 302; of 16 rows N 1024: 33 in one segment, 39 in two; 16 rows
// N 65536: 64 columns 384, 128 columns 365; fp16 gradients D = 64 of 32 rows N 1001: one segment 52, 8: 38;
// D = 192 bf16, 32 rows N 4096: 64 columns 122 in 8 segments, 128 columns 146 in 4; D = 24: 8 segments 31, 16: 28, 128: 41.
inline LinPlan linattn_plan(int64_t rows, int nroles, int64_t N, int64_t DK, int64_t DV, lconv_dtype_t dtype) {
    const int64_t chunks = (N + 31) / 32;
    const int kt = linattn_kt(DK);
    const double bytes = (double)rows * nroles * (double)N * (double)(DK + DV) * (dtype == LCONV_F32 ? 4 : 2) * (nroles == 3 ? 0.85 : 1.0);
    LinPlan best{};
    double least = 0.0;
    for (int nw = 1; nw <= (DV > 64 ? 2 : 1); ++nw) {
        const int64_t ncb = (DV + 64 * nw - 1) / (64 * nw), wgs = rows * nroles * ncb;
        for (int64_t nseg = 1; nseg == 1 || (nseg <= 1024 && nseg * 2 <= chunks && wgs * nseg <= 4096); nseg *= 2) {
            const int64_t per = (chunks + nseg - 1) / nseg, load = (wgs * nseg + 255) / 256;
            const double shared = linattn_alone(kt, nw, dtype == LCONV_F32) ? (double)load : 1.0 + 0.35 * (double)(load - 1);
            const double pass = (2.0 + (double)per * linattn_chunk_us(kt, nw, dtype)) * shared;
            const double floor = bytes / (nw == 1 && ncb > 1 ? 4.2e6 : 4.8e6) * (load == 1 ? 1.08 : 1.0);  // two of the four operands
            double t = pass > 2 * floor ? pass : 2 * floor;
            if (nseg > 1)
                t += (0.65 * pass > floor ? 0.65 * pass : floor) + 12.0 +
                     (double)(rows * nroles) * (double)nseg * (double)(DK * DV) * 16.0 / 8e6;
            if (best.kt == 0 || t < least) {
                least = t;
                const int64_t len = per * 32;
                best = LinPlan{kt, nw, (int)ncb, (int)((N + len - 1) / len), len};
                if (best.nseg < 1) best.nseg = 1;
            }
        }
    }
    return best;
}

// workspace of one role's segment states (whole tiles)
inline size_t linattn_states_bytes(const LinPlan& p, int64_t rows) {
    return p.nseg > 1 ? (size_t)rows * (size_t)p.nseg * (size_t)(p.kt * 16 * p.ncb * 64 * p.nw) * 4 : 0;
}

// The gradients' roles by launch: dq and dk contract over Dv and have Dk columns, dv the other way round.
// Roles of the same tiles go together: all three, or dq and dk.
struct LinBwdPlan {
    int launches, first[2], roles[2];   // roles first .. first + roles - 1 of (dq, dk, dv)
    LinPlan plan[2];
    size_t states[2];                   // bytes of one role's segment states
    size_t total;
};
inline LinBwdPlan linattn_bwd_plan(int64_t rows, int64_t N, int64_t Dk, int64_t Dv, lconv_dtype_t dtype) {
    LinBwdPlan p{};
    const bool alike = linattn_kt(Dk) == linattn_kt(Dv);
    const int64_t wide = Dk > Dv ? Dk : Dv;
    p.launches = alike ? 1 : 2;
    for (int i = 0; i < p.launches; ++i) {
        p.first[i] = 2 * i;
        p.roles[i] = alike ? 3 : 2 - i;
        p.plan[i] = linattn_plan(rows, p.roles[i], N, alike ? wide : i ? Dk : Dv, alike ? wide : i ? Dv : Dk, dtype);
        p.states[i] = linattn_states_bytes(p.plan[i], rows);
        p.total += (size_t)p.roles[i] * p.states[i];
    }
    return p;
}

// Threads along a launch's grid have to stay below 2^32: so many workgroups of 256.
constexpr int64_t kMaxWorkgroups = ((int64_t)1 << 24) - 1;

// Workgroups of the chunk kernel's main pass (the state pass has fewer): groups rounded up to the XCDs.
inline int64_t linattn_workgroups(const LinPlan& p, int64_t rows, int nroles) { return (rows * p.nseg + 7) / 8 * 8 * nroles * p.ncb; }

// The decay's gradient: column blocks, and segments of at least four chunks until two workgroups to a compute unit.
// Measured (bf16, us beside the other gradients): 32 rows of 4096 tokens, D = 128, one segment 240, 4: 97, 8: 81, 16: 104;
// 16 rows of 65536: 8: 722, 16: 599, 32: 615; 8 rows of 1000, D = 64, 1: 32, 4: 17, 8: 15, 16: 12; 128 rows of 2048: 1: 110, 4: 152.
#ifdef __HIPCC__
__host__ __device__
#endif
inline int linattn_tan_blocks(int64_t DV) { return (int)((DV + 63) / 64); }
struct LinTanPlan { int nseg; int64_t seg_len; };
inline LinTanPlan linattn_tan_plan(int64_t rows, int64_t N, int64_t DV) {
    const int64_t chunks = (N + 31) / 32, wgs = rows * linattn_tan_blocks(DV);
    int64_t nseg = 1;
    while (nseg * 8 <= chunks && wgs * nseg * 2 <= 512) nseg *= 2;
    const int64_t len = (chunks + nseg - 1) / nseg * 32;
    return LinTanPlan{(int)((N + len - 1) / len), len};
}

inline int64_t linattn_tan_workgroups(int64_t rows, int64_t N, int64_t DV) { return rows * linattn_tan_plan(rows, N, DV).nseg * linattn_tan_blocks(DV); }

// Single tokens: columns to a workgroup (see launch_linattn_step).
inline int linattn_step_columns(int64_t rows, int64_t DV) { return rows * ((DV + 127) / 128) < 128 ? 32 : 128; }
inline int64_t linattn_step_workgroups(int64_t rows, int64_t DV) {
    const int cb = linattn_step_columns(rows, DV);
    return rows * ((DV + cb - 1) / cb);
}

// Rotary: units of a token (8 pairs, or 16 copied elements), four heads to a thread where that leaves eight waves to a
// compute unit.
struct RotaryPlan {
    int turns, units, per, hgroups;
    int64_t threads;
};
inline RotaryPlan rotary_plan(int64_t tokens, int64_t D, int64_t rot, int heads) {
    RotaryPlan p{};
    p.turns = (int)((rot / 2 + 7) / 8);
    p.units = p.turns + (int)((D - rot + 15) / 16);
    const int64_t each = tokens * p.units;
    p.per = 4;
    while (p.per > 1 && each * ((heads + p.per - 1) / p.per) < 256 * 512) p.per /= 2;
    p.hgroups = (heads + p.per - 1) / p.per;
    p.threads = each * p.hgroups;
    return p;
}

// Layer norm: rows up to this width are held in registers.
constexpr int64_t kNormRegisterC = 8192;

// Workgroups of the gradient call, each with a partial sum of dweight and dbias over its rows: enough to
// fill the chip (three of 256 threads or two of 512 to each of 256 compute units), no more than turns of
// rows, since every one costs 8 C bytes written and read.  Measured (bf16, us, at 256, 512, 768 and 1024): 32768 rows of
// 768: 75, 48, 42, 41; 16384 of 2048: 64, 47, 46, 47; 16384 of 4096: 111, 82, 97, 88; 8192 of 8192: 102, 90, 103, 105.
// Three turns or fewer go to one workgroup, which leaves the sums itself and saves their launch.
inline int64_t layernorm_parts(int64_t rows, int64_t C) {
    const int64_t per = C <= 128 ? 16 : C <= 1024 ? 4 : C <= 2048 ? 2 : 1;   // rows a workgroup has in hand
    const int64_t turns = (rows + per - 1) / per, most = C <= 2048 ? 768 : 512;
    if (C <= kNormRegisterC && turns > 0 && turns <= 3) return 1;
    return turns < most ? turns : most;
}

}  // namespace lcv
