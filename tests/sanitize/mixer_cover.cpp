// Which chunk kernels of linear attention the plans choose, over a wide range of calls, and which of them a list of test
// cases reaches: standard input holds "dtype rows N Dk Dv" lines; standard output one line for each kernel that plans choose
// and no case reaches, then the two counts.  A kernel is (type, contraction tiles, column tiles, whole rows or segments,
// forward or gradients), counted only where a segment is long enough for the pipelined loop (five chunks).
#include <cstdio>
#include <map>
#include <string>
#include <tuple>

#include "mixer_plan.h"

using Kernel = std::tuple<int, int, int, int, int>;
using Seen = std::map<Kernel, std::string>;

static void see(Seen& s, const lcv::LinPlan& p, lconv_dtype_t dt, bool grad, const char* call, int64_t N) {
    if ((p.nseg > 1 ? p.seg_len : N) < 161) return;
    s.emplace(Kernel{(int)dt, p.kt, p.nw, p.nseg > 1, grad}, call);
}

static void call(Seen& s, int64_t rows, int64_t N, int64_t Dk, int64_t Dv, lconv_dtype_t dt) {
    char text[120];
    std::snprintf(text, sizeof text, "%d %ld %ld %ld %ld", (int)dt, (long)rows, (long)N, (long)Dk, (long)Dv);
    see(s, lcv::linattn_plan(rows, 1, N, Dk, Dv, dt), dt, false, text, N);
    const lcv::LinBwdPlan b = lcv::linattn_bwd_plan(rows, N, Dk, Dv, dt);
    for (int i = 0; i < b.launches; ++i) see(s, b.plan[i], dt, true, text, N);
}

int main() {
    Seen chosen, tested;
    for (int64_t rows : {1, 2, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 144, 192, 256, 400, 512, 1024})
        for (int64_t N : {161, 170, 200, 256, 330, 512, 700, 1001, 1500, 2048, 4096, 8192, 16384, 65536, 262144})
            for (int64_t Dk : {8, 24, 32, 40, 64, 72, 96, 104, 128, 136, 160, 192, 200, 256})
                for (int64_t Dv : {8, 24, 32, 40, 64, 72, 96, 104, 128, 136, 160, 192, 200, 256})
                    for (lconv_dtype_t dt : {LCONV_F32, LCONV_F16, LCONV_BF16}) call(chosen, rows, N, Dk, Dv, dt);
    long dt, rows, N, Dk, Dv;
    while (std::scanf("%ld %ld %ld %ld %ld", &dt, &rows, &N, &Dk, &Dv) == 5) call(tested, rows, N, Dk, Dv, (lconv_dtype_t)dt);
    int missing = 0;
    for (const auto& [k, text] : chosen)
        if (!tested.count(k)) {
            std::printf("type %d tiles %d columns %d %s %s: chosen for %s\n", std::get<0>(k), std::get<1>(k), 64 * std::get<2>(k),
                        std::get<3>(k) ? "segments" : "whole rows", std::get<4>(k) ? "gradients" : "forward", text.c_str());
            ++missing;
        }
    std::printf("chosen %zu missing %d\n", chosen.size(), missing);
    return 0;
}
