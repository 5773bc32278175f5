// gdn_kv4.cuh -- the 4-bit number format of the paged K/V cache and its conversions (sm_103a).
//
// A group of 16 consecutive dimensions of one cached key or value head is 16 e2m1 codes (8 bytes; dimension 2j in the
// lower half of byte j) and one e4m3 scale byte; a number is code * scale * (the cache's k_scale or v_scale, a power of
// two).  code * scale has at most 6 significant bits and magnitude 2^-10 .. 2688 (or 0): exact in fp16 and in bf16.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "gdn_common.cuh"

namespace gdn {

// Two e2m1 codes (one byte) -> f16x2, for the four bytes of a word (byte j -> out[j])
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&out)[4]) {
    asm("{\n\t.reg .b8 x, y, z, w;\n\tmov.b32 {x, y, z, w}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, x;\n\tcvt.rn.f16x2.e2m1x2 %1, y;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, z;\n\tcvt.rn.f16x2.e2m1x2 %3, w;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}

// Two e4m3 numbers (the lower 16 bits) -> f16x2
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// e4m3 byte of x >= 0, to nearest even, saturating at 448 (0x7e)
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %1;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "f"(x));
    return r & 0xffu;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
    const uint32_t h = e4m3x2_to_f16(b & 0xffu);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// e2m1 codes of (lo, hi), to nearest even, saturating at 6: one byte, lo in its lower half
__device__ __forceinline__ uint32_t f32x2_to_e2m1(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r & 0xffu;
}

// The tensor-core product on registers: D (16 x 8, fp32) += A (16 x 16) B (16 x 8), f16
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Two f16 numbers, a NaN as 0
__device__ __forceinline__ uint32_t nan_as_zero(uint32_t a) {
    const __half2 h = *reinterpret_cast<const __half2*>(&a);
    return a & __heq2_mask(h, h);
}

__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp; 0 for -inf
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- two fp32 numbers an instruction -----------------------------------------------------------------------
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Programmatic dependent launch: wait for the launch before this one in the stream to be complete and visible
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace gdn
