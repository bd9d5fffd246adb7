// The host code of the recurrence, the q/k norms and the short convolution under the address and undefined-behaviour
// sanitizers: plans over many shapes, size queries, and calls whose launchers record what they were given: a call launches
// within a grid's reach and with a plan that covers it, or is refused before its first launch.  Addresses are never
// dereferenced.  Exit status 0 when all holds.
#include <cstdint>
#include <cstdio>

#include "block_kernels.h"
#include "lconv.h"

static int failures = 0, launches = 0;

static void need(bool ok, const char* what, int64_t a, int64_t b, int64_t c, int64_t d = 0) {
    if (ok) return;
    std::fprintf(stderr, "%s: %lld %lld %lld %lld\n", what, (long long)a, (long long)b, (long long)c, (long long)d);
    ++failures;
}
static hipError_t grid(const char* what, int64_t workgroups, int threads) {
    ++launches;
    need(workgroups > 0 && workgroups * threads < (int64_t)1 << 32, what, workgroups, threads, 0);
    return hipSuccess;
}

namespace lcv {
static void covers(const ScanArgs& a, bool grad) {
    const int64_t tile = (int64_t)a.waves * kScanTokens;
    need(a.waves >= 1 && a.waves <= (grad ? kScanGradWaves : scan_waves(a.vec)), "waves", a.waves, a.vec, grad);
    need((int64_t)a.cblocks * 64 * a.vec >= a.C && (a.vec == 1 || a.C % 2 == 0), "blocks", a.C, a.cblocks, a.vec);
    need(a.nseg >= 1 && a.nseg * a.seg_len >= a.N && (a.nseg - 1) * a.seg_len < a.N, "segments", a.N, a.nseg, a.seg_len);
    need(a.nseg == 1 || (a.waves == 8 && a.seg_len % tile == 0 && a.seg_len % kScanMark == 0), "segment", a.waves, a.seg_len, tile);
    need(tile % kScanMark == 0 || (a.nseg == 1 && a.N <= tile), "marks", a.N, tile, a.nseg);
    need((a.seg != nullptr) || a.nseg == 1, "workspace", a.N, a.nseg, 0);
}
hipError_t launch_scan_fwd(int, const ScanArgs& a, hipStream_t) {
    covers(a, false);
    return grid("scan", a.B * a.nseg * a.cblocks, 64 * a.waves);
}
hipError_t launch_scan_bwd(int, const ScanArgs& a, hipStream_t) {
    covers(a, true);
    return grid("scan gradients", a.B * a.nseg * a.cblocks, 64 * a.waves);
}
hipError_t launch_scan_step(int, const ScanStepArgs& a, hipStream_t) { return grid("scan token", (a.B * a.C + 255) / 256, 256); }
hipError_t launch_row_state(const float*, float*, int64_t, hipStream_t) { return grid("state", 1, 256); }
hipError_t launch_qknorm_fwd(int, const QkArgs& a, hipStream_t) {
    const QkPlan p = qk_plan(a.B * a.N, a.D, a.rot, a.heads[0] + a.heads[1]);
    need(p.lanes >= p.units && p.lanes <= 64 && p.per * p.hgroups >= a.heads[0] + a.heads[1], "units", p.units, p.lanes, p.per);
    return grid("norm", (p.items * p.lanes + 255) / 256, 256);
}
hipError_t launch_qknorm_bwd(int, const QkArgs& a, hipStream_t) {
    if (a.B * a.N == 0) return grid("norm sums", 1, 1024);
    const QkGradPlan g = qk_grad_plan(a.B * a.N, a.D, a.rot, a.heads[0], a.heads[1]);
    need(g.parts[0] + g.parts[1] <= 770 && (g.parts[0] > 0) == (a.heads[0] > 0) && (g.parts[1] > 0) == (a.heads[1] > 0), "parts", g.parts[0],
         g.parts[1], a.heads[0], a.heads[1]);
    need(a.heads[0] == 0 || a.heads[1] == 0 || g.p[0].lanes == g.p[1].lanes, "lanes", g.p[0].lanes, g.p[1].lanes, 0);
    return grid("norm gradients", g.parts[0] + g.parts[1], 256);
}
static void covers(const ConvArgs& a, bool grad) {
    need(a.run >= kConvMaxTaps && a.runs * a.run >= a.N && (a.runs - 1) * a.run < a.N, "runs", a.N, a.run, a.runs);
    need((int64_t)a.cgroups * 64 * a.vec >= a.C && a.C >= a.vec, "groups", a.C, a.cgroups, a.vec);
    need(grad || (int64_t)a.groups * 4 >= a.B * a.runs, "workgroups", a.B, a.runs, a.groups);
    // one buffer for both states: no two lanes share a channel
    need(grad || a.C % a.vec == 0 || !a.state_in || a.state_in != a.state_out, "state in place", a.C, a.vec, 0);
}
hipError_t launch_conv_fwd(int, const ConvArgs& a, hipStream_t) {
    covers(a, false);
    return grid("conv", (int64_t)a.cgroups * a.groups, 256);
}
hipError_t launch_conv_bwd(int, const ConvArgs& a, hipStream_t) {
    if (a.groups == 0) return grid("conv sums", 1, 256);
    covers(a, true);
    return grid("conv gradients", (int64_t)a.cgroups * a.groups, 256);
}
hipError_t launch_conv_step(int, const ConvStepArgs& a, hipStream_t) { return grid("conv token", (a.B * a.C + 255) / 256, 256); }
hipError_t launch_conv_state(int, const void*, void*, int64_t, hipStream_t) { return grid("state", 1, 256); }
}  // namespace lcv

// a call launches or is refused and launches nothing
template <typename F> static bool taken(F&& call) {
    launches = 0;
    const int st = call();
    if (!(st == LCONV_SUCCESS && launches == 1) && !(st == LCONV_ERR_UNSUPPORTED && launches == 0)) {
        std::fprintf(stderr, "status %d after %d launches\n", st, launches);
        ++failures;
    }
    return st == LCONV_SUCCESS;
}

static void* at(uint64_t a) { return (void*)(uintptr_t)(a << 57); }     // 2^57 bytes apart: the largest operand here
static float* fat(uint64_t a) { return (float*)at(a); }

int main() {
    const size_t much = (size_t)1 << 60;
    const int64_t Bs[] = {1, 2, 7, 64, 300, 1 << 14, 1 << 20, 1 << 24}, Ns[] = {1, 7, 8, 63, 64, 65, 255, 257, 1001, 4096, 65536, 1 << 20, 2147483647};
    const int64_t Cs[] = {1, 2, 3, 5, 63, 64, 65, 130, 333, 1000, 4096, 1 << 17, 1 << 24};
    for (int64_t B : Bs)
        for (int64_t N : Ns)
            for (int64_t C : Cs) {
                if ((double)B * (double)N * (double)C > 1e16) continue;
                for (lconv_dtype_t dt : {LCONV_F32, LCONV_F16, LCONV_BF16}) {
                    for (int flags : {LCONV_GATE_SIGMOID | LCONV_MIX_CONVEX, LCONV_GATE_RATE | LCONV_MIX_NORM}) {
                        const bool f = taken([&] {
                            return lconv_gated_scan_fwd(at(1), nullptr, at(2), nullptr, at(3), nullptr, fat(4), fat(5), nullptr, at(6), nullptr,
                                                        fat(5), fat(7), B, N, C, flags, dt, at(8), much, nullptr);
                        });
                        const bool b = taken([&] {
                            return lconv_gated_scan_bwd(at(1), nullptr, at(2), nullptr, at(3), nullptr, at(4), nullptr, fat(5), fat(6), fat(7),
                                                        nullptr, at(8), nullptr, at(9), nullptr, at(10), nullptr, fat(11), fat(7), B, N, C, flags,
                                                        dt, at(12), much, nullptr);
                        });
                        if (B <= (1 << 20) && B * C <= (1 << 24) && !(f && b)) need(false, "refused", B, N, C);
                        // queries give nothing for what is refused, and room for every segment for what is taken
                        if (!f) need(lconv_gated_scan_workspace_bytes(B, N, C, dt) == 0, "query", B, N, C);
                        if (f) need(lconv_gated_scan_marks_bytes(B, N, C) >= (size_t)(B * C) * 4 * (size_t)((N + 63) / 64), "marks", B, N, C);
                        const lcv::ScanPlan p = lcv::scan_plan(B, N, C, dt, false), g = lcv::scan_plan(B, N, C, dt, true);
                        if (f && p.nseg > 1) need(lconv_gated_scan_workspace_bytes(B, N, C, dt) >= (size_t)(B * p.nseg * C) * 12, "room", B, N, C);
                        const size_t parts = (flags & 3) == LCONV_GATE_RATE ? (size_t)(B * g.nseg * C) * 4 : 0;
                        if (b) need(lconv_gated_scan_bwd_workspace_bytes(B, N, C, flags, dt) >= parts + (g.nseg > 1 ? (size_t)(B * g.nseg * C) * 12 : 0),
                                    "room of gradients", B, N, C);
                    }
                    for (int64_t K : {2, 4, 8}) {
                        for (bool inplace : {false, true}) {
                            const bool f = taken([&] {
                                return lconv_shortconv_fwd(at(1), nullptr, at(2), at(3), at(4), nullptr, at(5), nullptr, at(inplace ? 4 : 6), B, N, C, K,
                                                           LCONV_SHORTCONV_SILU, dt, nullptr);
                            });
                            if (B <= (1 << 20) && B * N * C <= (1 << 28) && !f) need(false, "conv refused", B, N, C);
                        }
                        const bool b = taken([&] {
                            return lconv_shortconv_bwd(at(1), nullptr, at(2), nullptr, at(3), at(4), at(5), at(6), nullptr, at(7), nullptr, fat(8), fat(9),
                                                       at(10), B, N, C, K, 0, dt, at(11), much, nullptr);
                        });
                        if (b)
                            need(lconv_shortconv_bwd_workspace_bytes(B, N, C, K) ==
                                     (size_t)lcv::conv_plan(B, N, C, K, true, false).groups * (size_t)(K + 1) * (size_t)C * 4,
                                 "conv room", B, N, C, K);
                    }
                }
                if (N == 1) {
                    taken([&] {
                        return lconv_gated_scan_step(at(1), C, at(2), C, at(3), C, fat(4), fat(5), nullptr, at(6), C, B, C, B, LCONV_GATE_RATE, LCONV_F16, nullptr);
                    });
                    taken([&] { return lconv_shortconv_step(at(1), C, at(2), at(3), at(4), nullptr, at(5), C, B, C, 4, B, 0, LCONV_F16, nullptr); });
                }
            }
    for (int64_t B : {(int64_t)1, (int64_t)64, (int64_t)1 << 20})
        for (int64_t N : {(int64_t)1, (int64_t)1023, (int64_t)1 << 16, (int64_t)1 << 24})
            for (int64_t H : {0, 1, 5, 64})
                for (int64_t G : {0, 1, 8})
                    for (int64_t D : {8, 24, 96, 128, 512})
                        for (int64_t rot : {(int64_t)0, (int64_t)2, D / 4 * 2, D}) {
                            if (H + G == 0) continue;
                            const bool f = taken([&] {
                                return lconv_qknorm_rotary_fwd(at(1), nullptr, G ? at(2) : nullptr, nullptr, at(3), at(4), nullptr, 0, fat(5), 1.f, 1e-6f, at(6),
                                                               nullptr, G ? at(7) : nullptr, nullptr, B, H, G, N, D, rot, 0, LCONV_BF16, nullptr);
                            });
                            const bool b = taken([&] {
                                return lconv_qknorm_rotary_bwd(at(1), nullptr, G ? at(2) : nullptr, nullptr, at(3), nullptr, G ? at(4) : nullptr, nullptr, at(5),
                                                               at(6), nullptr, 0, fat(7), 1.f, 1e-6f, at(8), nullptr, G ? at(9) : nullptr, nullptr, fat(10),
                                                               fat(11), B, H, G, N, D, rot, LCONV_QKNORM_CENTRED, LCONV_BF16, at(12), much, nullptr);
                            });
                            if (B * N * (H + G) <= (1 << 20) && !(f && b)) need(false, "norm refused", B, N, H, G);
                            need(!b || lconv_qknorm_rotary_bwd_workspace_bytes(B, H, G, N, D, rot) > 0, "norm room", B, N, H, G);
                        }
    if (failures) return 1;
    std::printf("BLOCK_SANITIZED_OK\n");
    return 0;
}
