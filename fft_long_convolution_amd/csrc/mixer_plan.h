// mixer_plan.h -- how a call of the mixer operators is cut into workgroups (host arithmetic only).
#pragma once
#include <stdint.h>

#include "lconv.h"

namespace lcv {

// Linear attention: tiles of the contraction (16 wide, padded to 2, 4, 8 or 16), 16-column tiles per
// wave, column blocks of 64 nw, and segments of seg_len tokens that a (b, h) is split into.
struct LinPlan {
    int kt, nw, ncb, nseg;
    int64_t seg_len;
};

inline int linattn_kt(int64_t DK) { return DK <= 32 ? 2 : DK <= 64 ? 4 : DK <= 128 ? 8 : 16; }

inline LinPlan linattn_plan(int64_t rows, int nroles, int64_t N, int64_t DK, int64_t DV, lconv_dtype_t dtype) {
    LinPlan p;
    p.kt = linattn_kt(DK);
    p.nw = DV > 64 ? 2 : 1;
    p.ncb = (int)((DV + 64 * p.nw - 1) / (64 * p.nw));
    const int64_t C = 64;                       // a multiple of the kernels' chunk
    (void)dtype;
    const int64_t wgs = rows * nroles * p.ncb;
    int64_t nseg = 1;
    if (wgs < 256) {
        nseg = 512 / wgs;
        const int64_t most = N / (4 * C);       // at least four chunks of a segment
        if (nseg > most) nseg = most;
        if (nseg < 1) nseg = 1;
    }
    p.seg_len = ((N + nseg - 1) / nseg + C - 1) / C * C;
    if (p.seg_len < C) p.seg_len = C;
    p.nseg = (int)((N + p.seg_len - 1) / p.seg_len);
    if (p.nseg < 1) p.nseg = 1;
    return p;
}

// workspace of one role's segment states
inline size_t linattn_states_bytes(const LinPlan& p, int64_t rows, int64_t DK, int64_t DV) {
    return p.nseg > 1 ? ((size_t)rows * (size_t)p.nseg * (size_t)(DK * DV) * 4 + 255) / 256 * 256 : 0;
}

// column blocks of the decay's gradient
inline int linattn_tan_blocks(int64_t DV) { return (int)((DV + 63) / 64); }

// Layer norm: rows up to this width are held in registers.
constexpr int64_t kNormRegisterC = 8192;

// Workgroups of the gradient call, each with a partial sum of dweight and dbias over its rows: enough to
// fill the chip (two to four on each of 256 compute units, by their registers), no more than turns of
// rows, since every one costs 8 C bytes written and read.
inline int64_t layernorm_parts(int64_t rows, int64_t C) {
    const int64_t per = C <= 128 ? 16 : C <= 2048 ? 4 : 1;   // rows a workgroup has in hand
    const int64_t turns = (rows + per - 1) / per, most = C <= 2048 ? 512 : 768;
    return turns < most ? turns : most;
}

}  // namespace lcv
