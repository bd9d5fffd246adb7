// Which variant of a kernel each call takes, from its plan: lines of "scan type B N C", "conv B N C K" or "norm B N H G D rot"
// on the standard input; the variants, one a line, on the output.
#include <cstdio>
#include <cstring>

#include "block_kernels.h"

int main() {
    char kind[16];
    while (std::scanf("%15s", kind) == 1) {
        long long n[6] = {};
        const int want = !std::strcmp(kind, "norm") ? 6 : 4;
        for (int i = 0; i < want; ++i)
            if (std::scanf("%lld", &n[i]) != 1) return 1;
        if (!std::strcmp(kind, "scan")) {
            for (bool grad : {false, true}) {
                const lcv::ScanPlan p = lcv::scan_plan(n[1], n[2], n[3], (lconv_dtype_t)n[0], grad);
                const bool part = n[2] < p.waves * lcv::kScanTokens || p.waves < 8;
                std::printf("scan %lld %s: channels %d, waves %s%d, %s\n", n[0], grad ? "gradients" : "forward", p.vec, part ? "below " : "",
                            part ? 8 : p.waves, p.nseg > 1 ? "segments" : "rows");
            }
        } else if (!std::strcmp(kind, "conv")) {
            for (bool grad : {false, true}) {
                const lcv::ConvPlan p = lcv::conv_plan(n[0], n[1], n[2], n[3], grad, false);
                const bool again = grad && n[0] * p.runs > 4 * (long long)p.groups;
                std::printf("conv %s: taps %lld, channels %d\nconv %s: %s%s\n", grad ? "gradients" : "forward", n[3], p.vec,
                            grad ? "gradients" : "forward", p.runs > 1 ? "runs" : "rows", again ? ", several to a wave" : "");
            }
        } else {
            const long long tokens = n[0] * n[1];
            const lcv::QkPlan f = lcv::qk_plan(tokens, n[4], n[5], (int)(n[2] + n[3]));
            const bool full = n[5] % 16 == 0 && (n[4] - n[5]) % 16 == 0 && f.lanes == f.units;
            std::printf("norm: lanes %d, %s groups\nnorm forward: heads %d\n", f.lanes, full ? "whole" : "parts of", f.per);
            const lcv::QkGradPlan g = lcv::qk_grad_plan(tokens, n[4], n[5], n[2], n[3]);
            for (int i = 0; i < 2; ++i)
                if (n[2 + i])
                    std::printf("norm gradients: heads %d\nnorm gradients: items %s\n", g.p[i].per,
                                g.p[i].items * g.p[i].lanes > 256ll * g.parts[i] ? "in turn" : "once");
        }
    }
    return 0;
}
