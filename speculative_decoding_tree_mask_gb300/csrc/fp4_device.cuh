// Device helpers of the 4-bit cache: e2m1 codes under e4m3 block scales. Internal.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "spec_device.cuh"

namespace specv {

// Two e2m1 codes of a byte as a pair of halves (exact); the low nibble is the low half.
// All four bytes of a word at once.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// Two e4m3 scales as a pair of halves (exact: 448 is the largest, 2^-9 the smallest).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes of eight floats, the first in the low nibble: nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float *y) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]),
          "f"(y[7]));
    return r;
}

// The e4m3 nearest to x >= 0 (ties to even, at most 448; NaN gives the NaN code).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

// Row (token, head) of a 4-bit cache in units of one head's D elements.
__device__ __forceinline__ uint32_t fp4_row(const spec_fp4_cache &c, int blk, int off, int head) {
    return c.layout == SPEC_KV_NHD
               ? ((uint32_t)blk * c.block_size + off) * (uint32_t)c.H + head
               : ((uint32_t)blk * c.H + head) * (uint32_t)c.block_size + off;
}

// The cache block of position p of request b, or -1 when it lies outside the table or cache.
__device__ __forceinline__ int fp4_block(const spec_fp4_cache &c, const FastDiv &by_page, int b,
                                         int64_t p, int *off) {
    if (p < 0 || p > INT32_MAX) return -1;   // the table holds at most INT32_MAX positions
    const int bi = (int)by_page((uint32_t)p);
    if (bi >= c.max_blocks) return -1;
    *off = (int)p - bi * c.block_size;
    const int blk = __ldg(c.block_table + (int64_t)b * c.max_blocks + bi);
    return blk >= 0 && blk < c.num_blocks ? blk : -1;
}

}  // namespace specv
