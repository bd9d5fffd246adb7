// mixer_checks.h -- host-side checks of strided operands, shared by mixer_api.cpp and block_api.cpp.
#pragma once
#include <initializer_list>

#include "api_checks.h"

namespace lcv {
namespace {

// The address range of one buffer; with a token-major footprint where it is a strided operand.
struct Range {
    const void* p;
    size_t bytes;
    // strided operands: the elements of one token lie within `foot` bytes, tokens are `step` bytes
    // apart and batch rows a multiple of that (step 0: not of this form)
    size_t foot, step;
};

Range buffer(const void* p, int64_t n, size_t es) { return Range{p, (size_t)n * es, 0, 0}; }

bool overlap(const Range& a, const Range& b) {
    if (!lcv::overlap(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.step == 0 || a.step != b.step) return true;
    // slices of one token-major buffer: b's footprint modulo the token step, seen from a's start
    const intptr_t d = (intptr_t)((uintptr_t)b.p - (uintptr_t)a.p);
    const intptr_t st = (intptr_t)a.step;
    const size_t at = (size_t)(((d % st) + st) % st);
    return !(at >= a.foot && at + b.foot <= a.step);
}

// no output meets an input or another output
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* a = outs.begin(); a != outs.end(); ++a) {
        for (const Range& b : ins)
            if (overlap(*a, b)) return true;
        for (const Range* b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return true;
    }
    return false;
}

// Strides of an operand [B][H][N][D]: resolves NULL to dense and checks them; `r` gets its range.
// B, H, N > 0 here.  A dimension of length one may come with any stride; it leaves with 0, since the kernels also form
// addresses a chunk away from a row's ends (the gradients' 31 tokens before a single one, which no lane then reads).
lconv_status_t operand(const void* p, const lconv_strides_t* given, int64_t B, int64_t H, int64_t N, int64_t D,
                       lconv_dtype_t dt, bool written, lconv_strides_t* s, Range* r) {
    const int64_t es = (int64_t)dtype_size(dt);
    if (given) {
        *s = *given;
    } else {
        int64_t t;
        s->n = D;
        if (!mul_ok(N, D, &s->h) || !mul_ok(H, s->h, &s->b) || !mul_ok(B, s->b, &t)) return LCONV_ERR_INVALID_SHAPE;
    }
    if (B == 1) s->b = 0;
    if (H == 1) s->h = 0;
    if (N == 1) s->n = 0;
    struct Dim { int64_t n, st; } dim[3] = {{B, s->b}, {H, s->h}, {N, s->n}};
    int64_t last = D, t;                 // elements from the start to the end of the last row
    for (const Dim& d : dim) {
        if (d.n == 1) continue;
        if (d.st < 0 || !mul_ok(d.n - 1, d.st, &t) || t > INT64_MAX / 8 - last) return LCONV_ERR_INVALID_SHAPE;
        last += t;
        if (d.st * es % 16) return LCONV_ERR_MISALIGNED;
    }
    if (written) {
        // rows must be apart: taken from the smallest stride up, each step clears what lies below it
        int64_t span = D;
        bool used[3] = {false, false, false};
        for (int k = 0; k < 3; ++k) {
            int m = -1;
            for (int i = 0; i < 3; ++i)
                if (!used[i] && (m < 0 || dim[i].st < dim[m].st || (dim[i].st == dim[m].st && dim[i].n < dim[m].n))) m = i;
            used[m] = true;
            if (dim[m].n == 1) continue;
            if (dim[m].st < span) return LCONV_ERR_INVALID_SHAPE;
            span += (dim[m].n - 1) * dim[m].st;
        }
    }
    if (!p) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(p)) return LCONV_ERR_MISALIGNED;
    *r = Range{p, (size_t)last * (size_t)es, 0, 0};
    const int64_t foot = (H == 1 ? 0 : (H - 1) * s->h) + D;
    // one token's step: the n stride, or for single tokens the batch row's
    const int64_t step = N > 1 ? s->n : s->b;
    if ((N > 1 || B > 1) && step >= foot && (B == 1 || s->b % step == 0)) {
        r->foot = (size_t)(foot * es);
        r->step = (size_t)(step * es);
    }
    return LCONV_SUCCESS;
}

}  // namespace
}  // namespace lcv
