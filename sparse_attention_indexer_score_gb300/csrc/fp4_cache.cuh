// The 4-bit key/value cache: the layout of a section (one head of one page) and
// the conversions of its codes and scales.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dsa {

// Scale bytes of a token's key (and of its value): dim / 16, padded so that a
// token's row of both is a multiple of 8 bytes.
__host__ __device__ __forceinline__ int fp4_scale_row(int dim) { return (dim + 63) / 64 * 4; }
__host__ __device__ __forceinline__ int fp4_section_bytes(int dim) { return kPage * (dim + 2 * fp4_scale_row(dim)); }

// Offsets of a token's rows in a section.
__host__ __device__ __forceinline__ int fp4_k_row(int dim, int t) { return t * (dim / 2); }
__host__ __device__ __forceinline__ int fp4_v_row(int dim, int t) { return (kPage + t) * (dim / 2); }
__host__ __device__ __forceinline__ int fp4_scales(int dim, int t) { return kPage * dim + t * 2 * fp4_scale_row(dim); }

constexpr int kFp4MaxDim = 128;

// Eight codes (a word, column i at bits 4i) as FP16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two E4M3 scales (the low 16 bits) as an FP16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float2 half2_float2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

int check_kv_cache_fp4(const dsa_kv_cache_fp4* c);

}  // namespace dsa
