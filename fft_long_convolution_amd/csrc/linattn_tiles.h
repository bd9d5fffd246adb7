// linattn_tiles.h -- LDS tiles, matrix-core operands and waits of linear attention's chunk kernels.
// Matrix products are 16 x 16 tiles of a wave: lane = 16 g + x holds rows 4 g + r, r < 4, of column x.
#pragma once
#include "mixer_io.h"
#include "mixer_kernels.h"

namespace lcv {
namespace {

// ---- matrix-core operands -------------------------------------------------------------------

// A tile in LDS is [rows][R groups of 16 bytes], no padding; logical group c of a row stands at c ^ f(row),
// so that the 16 rows of a row read, and the rows of a transposed read, fall on all banks.  (Rows of less
// than 256 bytes share a line of banks: f takes the row's place beyond it.)
__device__ __forceinline__ constexpr int swizzle(int row, int R) {
    const int s = R >= 16 ? row : R == 8 ? row >> 1 : row >> 2, h = R >= 16 ? 8 : R / 2;
    const int top = R >= 16 ? s >> 3 : R == 8 ? s >> 2 : s >> 1;
    return 2 * (s & (h - 1)) | (top & 1);
}

constexpr int lin_row_groups(int groups) {
    int r = 4;
    while (r < groups) r *= 2;
    return r;
}

typedef short s16x2 __attribute__((__vector_size__(4)));

template <int IO> struct Mx {  // bf16, fp16
    using E = uint16_t;
    static constexpr int C = 32;        // tokens of a chunk
    static constexpr int TK = 2;        // 16-wide tiles of one contraction step
    static constexpr int VEC = 8;       // elements of 16 bytes
    struct Frag { uint32_t w[4]; };
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
        const u32x4 av = {a.w[0], a.w[1], a.w[2], a.w[3]}, bv = {b.w[0], b.w[1], b.w[2], b.w[3]};
        if constexpr (IO == CT_BF16)
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av), __builtin_bit_cast(bf16x8, bv), c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, av), __builtin_bit_cast(f16x8, bv), c, 0, 0, 0);
    }
    // A state tile's row m is the contraction index of step t / 2, place 8 (m / 4) + 4 (t & 1) + m % 4: two
    // tiles' accumulators are then 8 neighbours, the 16 bytes that a row read takes at once.
    static __device__ __forceinline__ int state_row(int t, int g) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1); }
    // The lane's places in a tile: row x for row reads; for transposed reads (16 lanes read 4 rows of four
    // 8-byte pieces, and each gets a column of 4) K's pieces stand 16 bytes apart, V's side by side.
    // Step t is an exclusive or away.
    struct At { int row, tr, col; };
    static __device__ __forceinline__ At at(int g, int x, int R) {
        const int r = 4 * g + (x >> 2), f = swizzle(r, R);
        return At{x * R * 16 + (g ^ swizzle(x, R)) * 16, r * R * 16 + ((x & 3) ^ f) * 16,
                  r * R * 16 + (((x & 3) >> 1) ^ f) * 16 + (x & 1) * 8};
    }
    static __device__ __forceinline__ Frag load_row(const char* p, const At& l, int t) {
        const uint4 w = *(const uint4*)(p + (l.row ^ (64 * t)));
        return Frag{{w.x, w.y, w.z, w.w}};
    }
    static __device__ __forceinline__ uint2 tr(const char* p) {
        typedef short s16x4 __attribute__((__vector_size__(8)));
        typedef __attribute__((address_space(3))) s16x4* P;
        return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p));
    }
    // the state's tile t of K^T, and the 16 columns from 16 t of V, over the tokens of a step
    static __device__ __forceinline__ Frag load_kt(const char* p, const At& l, int t, int R) {
        const char* q = p + (l.tr ^ (64 * (t >> 1))) + 8 * (t & 1);
        const uint2 lo = tr(q), hi = tr(q + 16 * R * 16);
        return Frag{{lo.x, lo.y, hi.x, hi.y}};
    }
    static __device__ __forceinline__ Frag load_v(const char* p, const At& l, int t, int R) {
        const char* q = p + (l.col ^ (32 * t));
        const uint2 lo = tr(q), hi = tr(q + 16 * R * 16);
        return Frag{{lo.x, lo.y, hi.x, hi.y}};
    }
    static __device__ __forceinline__ Frag pack(const f32x4* t) {
        return Frag{{pack2<IO>(t[0][0], t[0][1]), pack2<IO>(t[0][2], t[0][3]), pack2<IO>(t[1][0], t[1][1]),
                     pack2<IO>(t[1][2], t[1][3])}};
    }
    static __device__ __forceinline__ void unpack(const Frag& f, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = unpack_lo<IO>(f.w[i]);
            v[2 * i + 1] = unpack_hi<IO>(f.w[i]);
        }
    }
    static __device__ __forceinline__ Frag pack(const float* v) {
        return Frag{{pack2<IO>(v[0], v[1]), pack2<IO>(v[2], v[3]), pack2<IO>(v[4], v[5]), pack2<IO>(v[6], v[7])}};
    }
    // m, or a NaN if one of the elements is not finite
    static __device__ __forceinline__ float nan_of(const Frag& f, float m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (IO == CT_BF16) m = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(s16x2, f.w[i]), s16x2{0, 0}, m, false);
            else m = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, f.w[i]), f16x2{0, 0}, m, false);
        }
        return m;
    }
};

template <> struct Mx<CT_F32> {
    using E = float;
    static constexpr int C = 32, TK = 1, VEC = 4;
    struct Frag { f32x4 v; };
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ int state_row(int t, int g) { return 16 * t + 4 * g; }
    struct At { int row, tr[4]; };
    static __device__ __forceinline__ At at(int g, int x, int R) {
        At l;
        l.row = x * R * 16 + (g ^ swizzle(x, R)) * 16;
        for (int s = 0; s < 4; ++s) {
            const int r = 4 * g + s;
            l.tr[s] = r * R * 16 + ((x >> 2) ^ swizzle(r, R)) * 16 + (x & 3) * 4;
        }
        return l;
    }
    static __device__ __forceinline__ Frag load_row(const char* p, const At& l, int t) {
        return Frag{*(const f32x4*)(p + (l.row ^ (64 * t)))};
    }
    static __device__ __forceinline__ Frag load_v(const char* p, const At& l, int t, int R) { return load_kt(p, l, t, R); }
    static __device__ __forceinline__ Frag load_kt(const char* p, const At& l, int t, int R) {
        Frag f;
#pragma unroll
        for (int s = 0; s < 4; ++s) f.v[s] = *(const float*)(p + (l.tr[s] ^ (64 * t)));
        return f;
    }
    static __device__ __forceinline__ Frag pack(const f32x4* t) { return Frag{t[0]}; }
    static __device__ __forceinline__ void unpack(const Frag& f, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f.v[i];
    }
    static __device__ __forceinline__ Frag pack(const float* v) { return Frag{{v[0], v[1], v[2], v[3]}}; }
    static __device__ __forceinline__ float nan_of(const Frag& f, float m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaf(f.v[i], 0.f, m);
        return m;
    }
};

// Global memory from a scalar address on, by 32-bit offsets of the lanes: raw buffer accesses, whose address
// takes no vector arithmetic.  Every offset lies within the buffer's size by the host's limit on token strides
// (31 of at most 2^27 bytes); kNowhere does not.
constexpr uint32_t kBufferBytes = 0xfc000000u, kNowhere = 0xfffffff0u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const char* base) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)kBufferBytes, 0x00020000);
}
// An offset, or past the buffer's end; as a maximum, which the compiler does not turn into a branch.
__device__ __forceinline__ uint32_t only_if(bool in, uint32_t off) {
    const uint32_t least = in ? 0u : kNowhere;
    return off > least ? off : least;
}
__device__ __forceinline__ float load_f32(const float* base, uint32_t off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buffer_at((const char*)base), off, 0, 0));
}
__device__ __forceinline__ void store_f32(float* base, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), buffer_at((const char*)base), off, 0, 0);
}
// 64 lanes' 16 bytes each to 1 KB of LDS in lane order, without registers for the data
__device__ __forceinline__ void to_lds(const char* base, uint32_t off, char* dst) {
    typedef __attribute__((address_space(3))) void* L;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_at(base), (L)dst, 16, off, 0, 0, 0);
}
// Barrier of a workgroup whose waves have waited for what they wrote: a fence would also wait for the
// loads to LDS of the chunks ahead.
__device__ __forceinline__ void barrier_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// at most `vm` vector memory operations outstanding, no LDS operation
template <int vm> __device__ __forceinline__ void wait_for_all_but() {
    static_assert(vm < 64, "six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((vm & 15) | ((vm >> 4) << 14) | (7 << 4));
}

// The state's factor from chunk to chunk, in one multiplication: gamma^c rounded, with what each rounding left out
// carried into the next chunk's, so that the product of any number of them is gamma^(c n) to one rounding.  (A pair of
// floats costs a second operation for every element of the state; one rounded factor drifts.)
__device__ __forceinline__ float uniform(float v) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v))); }
__device__ __forceinline__ float next_decay(float hi, float lo, float& owed) {
    const float t = lo + owed, g = hi + t;
    owed = t - (g - hi);
    return g;
}

// 2^(14 - e) and its inverse for a magnitude of binade e: brings the magnitude below 2^15
__device__ __forceinline__ float to_f16_range(float m, float* back) {
    int e = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
    e = e < -100 ? -100 : e > 110 ? 110 : e;
    *back = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    return __uint_as_float((uint32_t)(127 + 14 - e) << 23);
}
// the largest of the four lanes x, x + 16, x + 32, x + 48
__device__ __forceinline__ float max_over_g(float m) {
    m = fmaxf(m, __shfl_xor(m, 16));
    return fmaxf(m, __shfl_xor(m, 32));
}

__device__ __forceinline__ float max_over_wave(float m) {
#pragma unroll
    for (int w = 1; w < 16; w *= 2) m = fmaxf(m, __shfl_xor(m, w));
    return max_over_g(m);
}

}  // namespace
}  // namespace lcv
