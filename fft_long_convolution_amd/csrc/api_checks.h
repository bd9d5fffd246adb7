// api_checks.h -- host-side argument checks shared by the C ABI's entry points.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "lconv.h"

namespace lcv {
namespace {

size_t dtype_size(lconv_dtype_t dt) { return dt == LCONV_F32 ? 4 : 2; }
bool dtype_ok(int dt) { return dt == LCONV_F32 || dt == LCONV_F16 || dt == LCONV_BF16; }

bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

lconv_status_t hip_status(hipError_t e) { return e == hipSuccess ? LCONV_SUCCESS : LCONV_ERR_HIP; }

}  // namespace
}  // namespace lcv
