// cache_common.cuh -- what the kernels of the paged cache share: the e4m3 cache
// format, 16-byte global access and the type conversions.
//
// An e4m3 cache holds codes and one power-of-two exponent per block of 16
// tokens and KV head: value = code * 2^exp.  A floating 8-bit code has the same
// relative step at every exponent, so a power-of-two scale loses nothing
// against an arbitrary one, and moving a code to a larger exponent is exact
// until it becomes subnormal: a block can take a larger token, and rows can
// change blocks, without rounding the rows that are there twice.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "internal.h"

namespace plx {

constexpr int KV_BLOCK = 16;        // tokens that share an exponent (== a page's smallest size)
constexpr int KV_EMIN = -120, KV_EMAX = 120;

__device__ __forceinline__ uint4 ldg_nc16(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// 4 packed e4m3 -> 2 packed fp16x2 (exact)
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// 2 packed fp16x2 -> 4 packed e4m3, round to nearest even
__device__ __forceinline__ uint32_t f16x2_to_e4m3x4(uint32_t lo, uint32_t hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\tmov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "r"(lo), "r"(hi));
    return r;
}

// 2^e for whole e; below 2^-126 it is 2^-126 (stored exponents are in [-120, 120])
__device__ __forceinline__ float exp2_whole(int e) { return __int_as_float((max(e, -126) + 127) << 23); }

// Codes of one 16-byte chunk moved from exponent e to exponent e + k, k >= 0:
// code 2^-k rounded to nearest even.  fp16 holds code 2^-k exactly while it is
// at least half of the smallest code (2^-10), and what is below that is 0 in
// either format, so the intermediate fp16 rounding never shows.
__device__ __forceinline__ uint4 e4m3_shift_down(uint4 c, int k) {
    // 2^-k as fp16: normal to 2^-14, subnormal to 2^-24, 0 beyond
    const unsigned short h = k <= 14 ? (unsigned short)((15 - k) << 10) : (k <= 24 ? (unsigned short)(1 << (24 - k)) : 0);
    const __half2 f = __halves2half2(__ushort_as_half(h), __ushort_as_half(h));
    uint32_t *w = &c.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(w[i], lo, hi);
        const __half2 l2 = __hmul2(*reinterpret_cast<__half2 *>(&lo), f), h2 = __hmul2(*reinterpret_cast<__half2 *>(&hi), f);
        w[i] = f16x2_to_e4m3x4(*reinterpret_cast<const uint32_t *>(&l2), *reinterpret_cast<const uint32_t *>(&h2));
    }
    return c;
}

}  // namespace plx
