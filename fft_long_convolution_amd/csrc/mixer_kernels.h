// mixer_kernels.h -- launchers of the linear-attention, rotary and layer-norm kernels
// (host-callable, defined in linattn*.hip, rotary.hip and layernorm.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lconv.h"

namespace lcv {

// An operand [B][H][N][D] with element strides; the head of row h is h / share (heads that
// several query heads share).
struct LinOperand {
    const void* p;
    lconv_strides_t s;
    int share;
};

// One linear attention
//   O_i = s_q ( s_kv sum_{j<=i} gamma^(i-j) (Q_i . K_j) V_j + gamma^(i+1-r) S^T Q_i ),
//   S' = gamma^L S + s_kv sum_j gamma^(L-1-j+r) K_j V_j^T
// over the tokens 0 .. L-1 in order (r = 0) or from the last to the first (r = 1: the gradients'
// direction, where the state that enters is dL/dS of the last token's state, which no decay
// precedes).  Q, K are DK wide, V and O DV wide, S is DK x DV.
struct LinRole {
    LinOperand Q, K, V;
    void* O;
    lconv_strides_t o;
    int DK, DV;
    const float* s_in;        // [B][H] states, element (d, n) at d * s_row + n * s_col; NULL: zeros
    float* s_out;             // the same layout; NULL: not wanted
    int s_row, s_col;
    float* states;            // [B][H][nseg][column tiles][kt][256]: the states that enter the segments (nseg > 1)
    float s_q, s_kv;
    int reverse;
    int wide;                 // O in fp32 (a sum over shared heads follows), else in the dtype
};

// Up to three linear attentions over the same tokens in one launch, with one plan (linattn_plan).
struct LinJob {
    LinRole r[3];
    int nroles;
    const float* log_decay;   // [H]
    const int32_t* lengths;   // [B] or NULL
    int64_t B;
    int H;
    int64_t N, seg_len;
    int kt, nw, ncb, nseg;
    int exact;                // a state leaves the call
};

struct LinStepArgs {
    LinOperand q, k, v;       // strides' n unused
    void* y;
    lconv_strides_t ys;
    const float* log_decay;
    float* state;
    const int32_t* slots;
    float scale;
    int64_t B, nslots;
    int H, DK, DV;
};

// The decay's gradient: see linattn_tan.hip.  nseg and seg_len from linattn_tan_plan.
struct LinTanArgs {
    LinOperand q, k, v, dy;
    const float *s_in, *ds_out;   // [B][H][DK][DV] or NULL
    const float* log_decay;       // [H]
    const int32_t* lengths;       // [B] or NULL
    float* states;                // [B][H][nseg][2][DK][DV] (nseg > 1)
    float* part;                  // [H][B][nseg][column blocks]
    float scale;
    int64_t B, N, seg_len;
    int H, DK, DV, nseg;
};

hipError_t launch_linattn(int dtype, const LinJob& a, hipStream_t stream);
hipError_t launch_linattn_f32(const LinJob& a, hipStream_t stream);
hipError_t launch_linattn_f16(const LinJob& a, hipStream_t stream);
hipError_t launch_linattn_bf16(const LinJob& a, hipStream_t stream);
hipError_t launch_linattn_bf16_wide(const LinJob& a, hipStream_t stream);   // nw = 2
// the segments' own states to the states that enter them
hipError_t launch_linattn_join(const LinJob& a, bool f32, hipStream_t stream);
hipError_t launch_linattn_step(int dtype, const LinStepArgs& a, hipStream_t stream);
hipError_t launch_linattn_tan(int dtype, const LinTanArgs& a, float* dlog, hipStream_t stream);
// For both of two tensors: out[b][g][n][:] = sum over the `share` heads of g of the fp32 rows in[b][h][n][:] (dense)
struct HeadSumArgs {
    const float* in[2];
    void* out[2];
    lconv_strides_t os[2];
    int D[2];
    int64_t B, N;
    int G, share;
};
hipError_t launch_head_sum(int dtype, const HeadSumArgs& a, hipStream_t stream);
// state_out = state_in (or zeros) for calls without tokens
hipError_t launch_copy_state(const float* in, float* out, int64_t n, hipStream_t stream);

struct RotaryArgs {
    LinOperand q, k;
    void *yq, *yk;
    lconv_strides_t yqs, yks;
    const int32_t* positions;
    int64_t pos_stride;
    const float* inv_freq;
    float magnitude;
    int64_t B, N;
    int H, G, D, rot, flags;
};
hipError_t launch_rotary(int dtype, const RotaryArgs& a, hipStream_t stream);

struct NormArgs {
    const void *x, *dy, *weight, *bias;
    int64_t xs, dys, ys;
    void* y;                  // forward: y; gradient: dx
    float *mean, *rstd;       // forward: written (nullable); gradient: read
    float *dweight, *dbias, *part;
    int64_t rows, C;
    float eps;
};
hipError_t launch_layernorm_fwd(int dtype, const NormArgs& a, hipStream_t stream);
hipError_t launch_layernorm_bwd(int dtype, const NormArgs& a, hipStream_t stream);

}  // namespace lcv
