// scan.hip -- the gated linear recurrence: dispatch, the rate's sum, single tokens.
#include "scan_gates.h"
#include "scan_launch.h"

namespace lcv {
namespace {

// drate from the partial sums of rows and segments, in their order: a workgroup takes 32 channels, its 8 groups of lanes every
// eighth part, and joins the groups in order.  4 us at 8 rows; at many rows bound by the latency of its loads, one after another:
// 4096 x 64 x 512 218 us beside 608 for the gradients themselves.
__global__ void __launch_bounds__(256) scan_rate_kernel(const float* part, float* drate, int64_t parts, int64_t C) {
    __shared__ float join[8][32];
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + l;
    float u = 0.f;
    if (c < C)
        for (int64_t p = q; p < parts; p += 8) u += part[p * C + c];
    join[q][l] = u;
    __syncthreads();
    if (q || c >= C) return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += join[i][l];
    drate[c] = s;
}

// One token: h = a h + u in place, y = h.  Each element is read and written once: latency for few rows (64 x 2048 in bf16, 2.1 MB:
// 3.3 us, about what an empty launch takes), HBM for many.
template <int IO, int V, bool GATED> __global__ void __launch_bounds__(256) scan_step_kernel(ScanStepArgs a) {
    const int64_t per = a.C / V, i = (int64_t)blockIdx.x * 256 + threadIdx.x, b = i / per;
    const uint32_t c = (uint32_t)(i - b * per) * V;
    if (b >= a.B) return;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    float y[V] = {};
    if (slot >= 0 && slot < a.nslots) {
        float* const state = a.state + slot * a.C + c;
        float x[V], z[V], g[V], h[V];
        widen<IO, V>(load_raw_v<IO, V>(a.x.p, b * a.x.b, c), x);
        widen<IO, V>(load_raw_v<IO, V>(a.z.p, b * a.z.b, c), z);
        if constexpr (GATED) widen<IO, V>(load_raw_v<IO, V>(a.i.p, b * a.i.b, c), g);
        __builtin_memcpy(h, state, sizeof(h));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Decay k = a.gate == LCONV_GATE_SIGMOID ? decay_of_logit(z[v])
                          : a.gate == LCONV_GATE_LOG     ? decay_of_log2(kLog2e * z[v])
                                                         : decay_of_log2(-kLog2e * a.rate[c + v] * sigmoid(z[v]));
            const float m = a.mix == LCONV_MIX_NORM ? norm_of(k) : a.mix == LCONV_MIX_CONVEX ? loss_of(k) : 1.f;
            float u = m * x[v];
            if constexpr (GATED) u *= sigmoid(g[v]);
            y[v] = moved(k, h[v], u);
        }
        __builtin_memcpy(state, y, sizeof(y));
    }
    store_v<IO, V>(a.y, b * a.yb, c, y);
}

__global__ void __launch_bounds__(256) row_state_kernel(const float* in, float* out, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) out[i] = in ? in[i] : 0.f;
}

template <int IO, int V> void go(const ScanStepArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.B * (a.C / V) + 255) / 256);
    if (a.i.p) scan_step_kernel<IO, V, true><<<grid, 256, 0, stream>>>(a);
    else scan_step_kernel<IO, V, false><<<grid, 256, 0, stream>>>(a);
}
template <int IO> void go(const ScanStepArgs& a, hipStream_t stream) {
    if (a.C % 2) go<IO, 1>(a, stream);
    else go<IO, 2>(a, stream);
}

}  // namespace

hipError_t launch_scan_fwd(int dtype, const ScanArgs& a, hipStream_t stream) {
    return dtype == LCONV_F32 ? launch_scan_fwd_f32(a, stream) : dtype == LCONV_F16 ? launch_scan_fwd_f16(a, stream)
                                                                                    : launch_scan_fwd_bf16(a, stream);
}

hipError_t launch_scan_bwd(int dtype, const ScanArgs& a, hipStream_t stream) {
    const hipError_t e = dtype == LCONV_F32 ? launch_scan_bwd_f32(a, stream) : dtype == LCONV_F16 ? launch_scan_bwd_f16(a, stream)
                                                                                                  : launch_scan_bwd_bf16(a, stream);
    if (e != hipSuccess || !a.part) return e;
    scan_rate_kernel<<<(unsigned)((a.C + 31) / 32), 256, 0, stream>>>(a.part, a.drate, a.B * a.nseg, a.C);
    return hipGetLastError();
}

hipError_t launch_scan_step(int dtype, const ScanStepArgs& a, hipStream_t stream) {
    if (dtype == LCONV_F32) go<CT_F32>(a, stream);
    else if (dtype == LCONV_F16) go<CT_F16>(a, stream);
    else go<CT_BF16>(a, stream);
    return hipGetLastError();
}

hipError_t launch_row_state(const float* in, float* out, int64_t n, hipStream_t stream) {
    const int64_t grid = (n + 255) / 256;
    row_state_kernel<<<(unsigned)(grid < 8192 ? grid : 8192), 256, 0, stream>>>(in, out, n);
    return hipGetLastError();
}

}  // namespace lcv
