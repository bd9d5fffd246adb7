// linattn.hip -- linear attention with a decay for each head: prompts, gradients, single tokens.
#include "mixer_kernels.h"
#include "mixer_io.h"
#include "mixer_plan.h"

namespace lcv {
namespace {

// Slot s of a row's states holds what segment s - 1 added up from zero; it becomes the state that
// enters segment s, slot 0 the state that enters the row.  Slots are the chunk kernel's registers: tiles of 16 x 16, 4 rows
// to a lane.  Eight segments' loads in flight (one load at a time took nearly twice as long).
__global__ void __launch_bounds__(256) linattn_join_kernel(LinJob a, int f32) {
    const LinRole& r = a.r[blockIdx.y];
    const uint32_t per = a.kt * a.ncb * 4 * a.nw * 64, i = blockIdx.x * 256 + threadIdx.x;   // lanes of a slot
    const uint32_t bh = i / per, e = i - bh * per;
    if (bh >= a.B * a.H) return;
    const int64_t size = 4 * (int64_t)per;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    const bool fours = !f32 && a.nw == 2;
    const int lane = e & 63, g = lane >> 4, x = lane & 15, m = (int)((e >> 6) / (uint32_t)a.kt), t = (int)(e >> 6) - m * a.kt;
    const int d0 = f32 ? 16 * t : 32 * (t >> 1) + 4 * (t & 1), n0 = fours ? 32 * (m >> 1) + 4 * (m & 1) : 16 * m;
    if (d0 >= r.DK || n0 >= r.DV) return;      // a tile that there is not
    if (r.s_in) {
        const int d = d0 + (f32 ? 4 : 8) * g, n = n0 + (fours ? 8 * (x >> 2) + (x & 3) : x);
        if (d < r.DK && n < r.DV) {
            const float* s = r.s_in + (int64_t)bh * (r.DK * r.DV) + d * r.s_row + n * r.s_col;
            for (int j = 0; j < 4; ++j) S[j] = s[j * r.s_row];
        }
    }
    float* st = r.states + (int64_t)bh * a.nseg * size + 4 * e;
    *(f32x4*)st = S;
    const uint32_t b = bh / (uint32_t)a.H;
    const int64_t len = row_len(a.lengths, b, a.N);
    const DecayPair gamma = decay_pair(log_gamma(a.log_decay, (int)(bh - b * (uint32_t)a.H)), (float)a.seg_len);
    // a row's segments are in a chain of their own, but their sums are not: eight loads in flight
    int last = a.nseg;
    while (last > 1 && (last - 1) * a.seg_len >= len) --last;
    for (int s = 1; s < last; s += 8) {
        f32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s + j < last) v[j] = *(const f32x4*)(st + (s + j) * size);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s + j < last) {
                S = decayed(S, gamma, v[j]);
                *(f32x4*)(st + (s + j) * size) = S;
            }
    }
}

// One token: S = gamma S + k v^T in place, y = scale S^T q, gamma as two floats so that thousands of tokens drift no more than
// a prompt's chunks.  The state's 8 Dk Dv bytes are read and
// written once, all else is small: bound by HBM, or by latency for few rows.  A workgroup takes CB columns
// of one (b, h): 16-byte loads along a row, up to 16 of them in flight per thread, q and k as floats
// through LDS while the state is on its way, y's sum over the rows through LDS.  Measured, D = 128: 256 sequences of 16
// heads (537 MB) 108 us, 5.0 TB/s (one load at a time 179 us); one sequence of 16 heads 5.3 us.
template <int IO, int CB>
__global__ void __launch_bounds__(256) linattn_step_kernel(LinStepArgs a) {
    constexpr int LPR = CB / 4, RPP = 256 / LPR, BATCH = 16;   // lanes to a row, rows to a pass
    __shared__ float qk[2][256];
    __shared__ __attribute__((aligned(16))) f32x4 red[256];
    const int ncb = (a.DV + CB - 1) / CB;
    const int64_t bh = blockIdx.x / ncb;
    const int cb = (int)(blockIdx.x - bh * ncb);
    const int64_t b = bh / a.H;
    const int h = (int)(bh - b * a.H), tid = threadIdx.x;
    const int n = cb * CB + tid % LPR * 4, d0 = tid / LPR;
    const bool on = n < a.DV;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    const int64_t yo = b * a.ys.b + (int64_t)h * a.ys.h;
    if (slot < 0 || slot >= a.nslots) {
        if (d0 == 0 && on)
            for (int i = 0; i < 4; ++i) store1<IO>(a.y, yo + n + i, 0.f);
        return;
    }
    float* S = a.state + (slot * a.H + h) * (int64_t)a.DK * a.DV + n;
    f32x4 s[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
        if (on && d0 + i * RPP < a.DK) s[i] = *(const f32x4*)(S + (int64_t)(d0 + i * RPP) * a.DV);
    if (tid < a.DK) {
        qk[0][tid] = load1<IO>(a.q.p, row_base(a.q, b, h) + tid) * a.scale;
        qk[1][tid] = load1<IO>(a.k.p, row_base(a.k, b, h) + tid);
    }
    f32x4 v = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
    if (on)
        for (int i = 0; i < 4; ++i) v[i] = load1<IO>(a.v.p, row_base(a.v, b, h) + n + i);
    const DecayPair gamma = decay_pair(log_gamma(a.log_decay, h), 1.f);
    __syncthreads();
    for (int base = 0; base < a.DK; base += BATCH * RPP) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int d = base + d0 + i * RPP;
            if (!on || d >= a.DK) continue;
            if (base) s[i] = *(const f32x4*)(S + (int64_t)d * a.DV);
            s[i] = decayed(s[i], gamma, v * qk[1][d]);
            y += s[i] * qk[0][d];
            *(f32x4*)(S + (int64_t)d * a.DV) = s[i];
        }
    }
    red[tid] = y;
    __syncthreads();
    if (tid < CB && cb * CB + tid < a.DV) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < RPP; ++i) t += ((const float*)red)[i * CB + tid];
        store1<IO>(a.y, yo + cb * CB + tid, t);
    }
}

template <int IO>
__global__ void __launch_bounds__(256) head_sum_kernel(HeadSumArgs a) {
    const int which = blockIdx.y, D = a.D[which], share = a.share, G = a.G;
    const float* const in = a.in[which];
    const lconv_strides_t os = a.os[which];
    const int64_t N = a.N, total = a.B * G * N * (D / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / (D / 8);
        const int d = (int)(i - row * (D / 8)) * 8;
        const int64_t bg = row / N, t = row - bg * N;
        const int64_t b = bg / G, g = bg - b * G;
        float x[8] = {0.f};
        for (int s = 0; s < share; ++s) {
            const float* p = in + ((bg * share + s) * N + t) * D + d;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] += p[j];
        }
        store8<IO>(a.out[which], b * os.b + g * os.h + t * os.n + d, x);
    }
}

__global__ void __launch_bounds__(256) copy_state_kernel(const float* in, float* out, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        out[i] = in ? in[i] : 0.f;
}

unsigned grid_1d(int64_t threads) {
    const int64_t g = (threads + 255) / 256;
    return (unsigned)(g < 8192 ? (g > 0 ? g : 1) : 8192);
}

template <typename F> hipError_t by_dtype(int dtype, F&& f) {
    if (dtype == LCONV_F32) f(std::integral_constant<int, CT_F32>{});
    else if (dtype == LCONV_F16) f(std::integral_constant<int, CT_F16>{});
    else f(std::integral_constant<int, CT_BF16>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn(int dtype, const LinJob& a, hipStream_t stream) {
    return dtype == LCONV_F32 ? launch_linattn_f32(a, stream) : dtype == LCONV_F16 ? launch_linattn_f16(a, stream)
                                                                                   : launch_linattn_bf16(a, stream);
}

hipError_t launch_linattn_join(const LinJob& a, bool f32, hipStream_t stream) {
    const int64_t lanes = a.B * a.H * ((int64_t)a.kt * a.ncb * 4 * a.nw * 64);
    linattn_join_kernel<<<dim3((unsigned)((lanes + 255) / 256), a.nroles), 256, 0, stream>>>(a, f32);
    return hipGetLastError();
}

hipError_t launch_linattn_step(int dtype, const LinStepArgs& a, hipStream_t stream) {
    // few rows: 32 columns to a workgroup, four times the workgroups to share the latency.  Measured (D = 128, us, at 32
    // and 128 columns): 16 rows 4.7, 5.9; 64 rows 5.2, 6.3; 256 rows 8.2, 7.6; 1024 rows 28, 21; 4096 rows 91, 82
    const int64_t rows = a.B * a.H;
    const bool narrow = linattn_step_columns(rows, a.DV) == 32;
    const unsigned grid = (unsigned)linattn_step_workgroups(rows, a.DV);
    return by_dtype(dtype, [&](auto io) {
        if (narrow) linattn_step_kernel<io.value, 32><<<grid, 256, 0, stream>>>(a);
        else linattn_step_kernel<io.value, 128><<<grid, 256, 0, stream>>>(a);
    });
}

hipError_t launch_head_sum(int dtype, const HeadSumArgs& a, hipStream_t stream) {
    const int64_t total = a.B * a.G * a.N * ((a.D[0] > a.D[1] ? a.D[0] : a.D[1]) / 8);
    return by_dtype(dtype, [&](auto io) { head_sum_kernel<io.value><<<dim3(grid_1d(total), 2), 256, 0, stream>>>(a); });
}

hipError_t launch_copy_state(const float* in, float* out, int64_t n, hipStream_t stream) {
    copy_state_kernel<<<grid_1d(n), 256, 0, stream>>>(in, out, n);
    return hipGetLastError();
}

}  // namespace lcv
