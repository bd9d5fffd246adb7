// block_kernels.h -- launchers of the gated recurrence, the q/k norms with rotary positions and the short convolution
// (host-callable, defined in scan*.hip, qknorm.hip and shortconv.hip), and how their calls are cut into workgroups.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lconv.h"

namespace lcv {

// An operand [B][N][C] whose channels are contiguous: element strides of its rows (the strides' h unused).
struct TokOperand {
    const void* p;
    int64_t b, n;
};

// ---- gated linear recurrence ------------------------------------------------------------------------

// Tokens of a wave's turn; the most waves of a workgroup (one or two channels to a lane; the gradient's registers leave room
// for eight); tokens from one mark to the next, a tile of eight waves.
constexpr int kScanTokens = 8, kScanMark = 64;
constexpr int scan_waves(int vec) { return vec == 2 ? 8 : 16; }
constexpr int kScanGradWaves = 8;

struct ScanArgs {
    TokOperand x, z, i, dy;       // i.p NULL: no input gate; dy: gradients only
    const float* rate;            // [C], LCONV_SCAN_RATE only
    const float* state_in;        // [B][C] or NULL; gradients: dL/dstate_out
    const int32_t* lengths;       // [B] or NULL
    void* y;
    int64_t yb, yn;
    void *dx, *dz, *di;           // gradients
    int64_t dxb, dxn, dzb, dzn, dib, din;
    float* state_out;             // [B][C] or NULL; gradients: dL/dstate_in
    float* marks;                 // [B][tiles][C]: forward written or NULL, gradients read
    float* seg;                   // [B][nseg][3][C]: decays (in two) and sums of the segments (nseg > 1)
    float* part;                  // [B nseg][C]: the rate's gradient, partial sums
    float* drate;
    int64_t B, N, C, seg_len;
    int nseg, cblocks, waves, vec, gate, mix;
};

// How a call is cut: channels to a lane, blocks of 64 vec channels, segments of seg_len tokens (a multiple of a tile),
// waves to a workgroup.
struct ScanPlan {
    int vec, cblocks, nseg, waves;
    int64_t seg_len;
};
// Two channels to a lane move 256 bytes of a 16-bit row at a time, which memory gives 10 % faster than 128, but leave half as many
// workgroups; sixteen waves fill a compute unit that has one workgroup.  Calls of few rows go by segments, which read everything
// twice but for y.  Measured (bf16, every input, us; channels to a lane, waves, segments):
//   8 x 2048 x 4096    2, 8, 1: 114    1, 8, 1: 126    1, 16, 1: 123    2, 8, 16: 95 + 132
//   10 x 2048 x 2048   2, 8, 1: 95     1, 16, 1: 107 (a second round of 256 workgroups)
//   8 x 2048 x 2048    1, 16, 1: 64    2, 8, 1: 94
//   16 x 2048 x 1024   1, 16, 1: 53    1, 8, 1: 63     2, 8, 4: 88
//   4 x 2048 x 2048    1, 16, 1: 52    2, 8, 8: 52     2, 8, 1: 98
//   2 x 2048 x 2048    2, 8, 8: 34     1, 16, 1: 51
//   1 x 65536 x 4096   2, 8, 16: 638   1, 8, 16: 700   1, 16, 1: 1464
//   1 x 777 x 333      1, 8, 8: 15     1, 16, 1: 24
//   16 x 300 x 2048    1, 8, 1: 20     1, 16, 1: 26
//   600 x 512 x 64     1, 8, 1: 27     2, 8, 1: 40 (sigmoid, convex: half the lanes without channels)
// With two channels to a lane a compute unit holds one workgroup of the gradients (of log or sigmoid, plain, without an input gate:
// two); with one channel one of those with an input gate and rate and norm, rate and convex, or sigmoid and norm (130 to 144
// registers), two of the others.  They go by rounds of 256, and a round of two channels takes 7/4 of one, as measured where one
// workgroup is all there is, for the others too (every input, one / two channels): 8 x 2048 x 4096 237 / 211, 9 x 2048 x 2048 206 / 176, 64 x 512 x 1024 128 / 116, but
// 300 x 512 x 128 89 / 94; in segments 1 x 65536 x 2048 601 / 519, 4 x 2048 x 2048 76 / 65, 3 x 1001 x 1000 30 / 27, but 2 x 700 x 64
// 24 / 25.  Segments (one channel): 4 x 2048 x 2048 in 1, 2, 4 95, 77, 78; 3 x 1001 x 1000 in 1, 4, 8 53, 28, 31; 1 x 65536 x 4096 in
// 1, 4, 8, 16 2870, 1140, 1043, 1050.
inline ScanPlan scan_plan(int64_t B, int64_t N, int64_t C, lconv_dtype_t dtype, bool grad) {
    ScanPlan p{};
    const int64_t ones = B * ((C + 63) / 64), twos = B * ((C + 127) / 128);      // rows of one and of two channels to a lane
    const bool pairs = dtype != LCONV_F32 && C % 2 == 0 && C > 64, cut = ones <= (grad ? 128 : 96) && N > 256;
    const auto rounds = [](int64_t rows) { return (rows + 255) / 256; };
    p.vec = pairs && (cut || (grad ? 7 * rounds(twos) < 4 * rounds(ones) : ones > 256)) ? 2 : 1;
    p.cblocks = (int)((C + 64 * p.vec - 1) / (64 * p.vec));
    const int64_t rows = B * p.cblocks;
    p.waves = p.vec == 2 || grad || cut || rows >= 512 ? 8 : 16;
    const int64_t tile = p.waves * kScanTokens, tiles = (N + tile - 1) / tile;
    int64_t nseg = 1;
    if (cut)
        while (nseg * 2 * rows <= (grad ? 256 : 512) && nseg * 2 <= tiles) nseg *= 2;
    const int64_t per = (tiles + nseg - 1) / nseg;
    p.seg_len = per * tile;
    p.nseg = (int)((N + p.seg_len - 1) / p.seg_len);
    if (N < tile) p.waves = (int)((N + kScanTokens - 1) / kScanTokens);
    return p;
}

struct ScanStepArgs {
    TokOperand x, z, i;           // rows b apart
    const float* rate;
    float* state;                 // [nslots][C]
    const int32_t* slots;         // [B] or NULL
    void* y;
    int64_t yb;
    int64_t B, C, nslots;
    int gate, mix;
};

hipError_t launch_scan_fwd(int dtype, const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_bwd(int dtype, const ScanArgs& a, hipStream_t stream);
hipError_t launch_scan_step(int dtype, const ScanStepArgs& a, hipStream_t stream);
// out = in (or zeros) for calls without tokens
hipError_t launch_row_state(const float* in, float* out, int64_t n, hipStream_t stream);

// ---- norms of q and k with rotary positions -----------------------------------------------------------

// Lanes to a head: a power of two that holds its units (8 pairs, or 16 elements that are only scaled).  An item is one token
// of `per` heads, which share the token's sines.
struct QkPlan {
    int turns, units, lanes, per, hgroups;
    int64_t items;
};
inline QkPlan qk_plan(int64_t tokens, int64_t D, int64_t rot, int heads) {
    QkPlan p{};
    p.turns = (int)((rot / 2 + 7) / 8);
    p.units = p.turns + (int)((D - rot + 15) / 16);
    p.lanes = 1;
    while (p.lanes < p.units) p.lanes *= 2;
    p.per = 4;
    while (p.per > 1 && tokens * ((heads + p.per - 1) / p.per) * p.lanes < 256 * 512) p.per /= 2;
    p.hgroups = (heads + p.per - 1) / p.per;
    p.items = tokens * p.hgroups;
    return p;
}
// The gradients' workgroups keep to q or to k, each with a partial sum of that weight's gradient over its items; at most as
// many for both as the chip holds at once in 16 bits (three to a compute unit; of fp32, with 176 registers, two, so that a third of
// its workgroups begin when others have ended), shared out by heads.  Measured (bf16, D = 128, 16 + 16 heads of 4 x 4096 tokens, us,
// at most 512, 768, 1024): 90, 86, 97; workgroups that take q and k in turn, 1024: 114.
struct QkGradPlan {
    QkPlan p[2];
    int parts[2];
};
inline QkGradPlan qk_grad_plan(int64_t tokens, int64_t D, int64_t rot, int64_t H, int64_t G) {
    QkGradPlan g{};
    const int64_t heads[2] = {H, G}, most = 768;
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        g.p[i] = qk_plan(tokens, D, rot, (int)heads[i]);
        const int64_t wgs = (g.p[i].items * g.p[i].lanes + 255) / 256, share = most * heads[i] / (H + G) > 0 ? most * heads[i] / (H + G) : 1;
        g.parts[i] = (int)(wgs < share ? wgs : share);
    }
    return g;
}

struct QkArgs {
    const void *x[2], *dy[2], *w[2];      // q and k; w NULL: ones
    lconv_strides_t xs[2], dys[2], ys[2];
    void* y[2];                           // forward: the results; gradients: dq, dk
    float* dw[2];                         // [D] or NULL
    float* part;                          // [parts of q, then of k][D]
    const int32_t* positions;
    int64_t pos_stride;
    const float* inv_freq;
    float magnitude, eps;
    int64_t B, N;
    int heads[2], D, rot, flags;
};
hipError_t launch_qknorm_fwd(int dtype, const QkArgs& a, hipStream_t stream);
hipError_t launch_qknorm_bwd(int dtype, const QkArgs& a, hipStream_t stream);

// ---- short causal convolution ---------------------------------------------------------------------------

constexpr int kConvMaxTaps = 8;

struct ConvArgs {
    TokOperand x, dy;             // dy: gradients only
    const void *w, *bias;         // [C][K]; [C] or NULL
    const void* state_in;         // [B][K-1][C] or NULL: the inputs before the first token, oldest first
    const void* dstate_out;       // gradients: of the inputs that the call left, or NULL
    const int32_t* lengths;
    void* y;                      // gradients: dx
    int64_t yb, yn;
    void* state_out;              // [B][K-1][C] or NULL; gradients: dL/dstate_in
    float *dw, *db;               // [C][K], [C] or NULL
    float* part;                  // [groups][K + 1][C]: taps, then the bias
    int64_t B, N, C, run;
    int K, silu, vec, cgroups, runs, groups;
};

// How a call is cut: channels to a lane, groups of 64 vec channels, runs of tokens to a wave (never shorter than the K - 1
// inputs before a run, so that only a row's first run meets its state), workgroups of four runs (gradients: each with a
// partial sum over the runs that it takes in turn).
struct ConvPlan {
    int vec, cgroups, runs, groups;
    int64_t run;
};
// The last lane of a width that four does not divide shares channels with the one before it; inplace (one buffer for both
// states) forbids that, since the two may be in different workgroups, one of which would read what the other has written.
// Runs: every wave reads K - 1 tokens of its neighbours again, and few calls have waves to spare.  The gradients' waves take
// runs in turn: 768 workgroups, or 512 of more than four taps, as measured at 4 and 8 taps in bf16.  By their registers a compute
// unit holds three workgroups of 3 or 4 taps and two of 6 to 8; of 2 taps it would hold four, of 5 in 16 bits three.  Measured
// (bf16, us, forward / gradients): 8 x 2048 x 4096, K = 4: runs of 16 49 / 108, 32 48 / 94, 64 49 / 99, in 512,
// 768, 1024 workgroups 103, 94, 107; 1 x 65536 x 2048, K = 8: 32 119 / 256, 64 114 / 232, 128 116 / 206, in 512, 768, 1024
// workgroups 206, 215, 213; 2 x 2048 x 2048, K = 4: 16 10 / 20, 32 11 / 23; 3 x 1001 x 1000, K = 3: 16 6.5 / 16, 32 8.8 / 21.
inline ConvPlan conv_plan(int64_t B, int64_t N, int64_t C, int64_t K, bool grad, bool inplace) {
    ConvPlan p{};
    p.vec = C % 4 == 0 || (C > 4 && !inplace) ? 4 : 1;
    p.cgroups = (int)((C + 64 * p.vec - 1) / (64 * p.vec));
    p.run = K <= 4 ? 32 : grad ? 128 : 64;
    while (p.run > kConvMaxTaps && B * ((N + p.run - 1) / p.run) * p.cgroups < 256 * 8) p.run /= 2;
    const int64_t runs = (N + p.run - 1) / p.run, groups = (B * runs + 3) / 4, most = ((K <= 4 ? 768 : 512) + p.cgroups - 1) / p.cgroups;
    p.runs = (int)runs;
    p.groups = (int)(grad && groups > most ? most : groups);
    return p;
}

struct ConvStepArgs {
    TokOperand x;
    const void *w, *bias;
    void* state;                  // [nslots][K-1][C]
    const int32_t* slots;
    void* y;
    int64_t yb, B, C, nslots;
    int K, silu;
};

hipError_t launch_conv_fwd(int dtype, const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_bwd(int dtype, const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_step(int dtype, const ConvStepArgs& a, hipStream_t stream);
// out = in (or zeros), n elements, for calls without tokens
hipError_t launch_conv_state(int dtype, const void* in, void* out, int64_t n, hipStream_t stream);

}  // namespace lcv
