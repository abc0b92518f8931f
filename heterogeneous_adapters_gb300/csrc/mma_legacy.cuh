// Warp-level matrix pieces of the 4-bit kernels: ldmatrix, mma.sync on bf16, and the step
// from packed 4-bit codes to bf16 operands.
#pragma once
#include <stdint.h>

namespace lora {

// Four 8 x 8 matrices of 16-bit elements; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held one register a lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// c += a b, a 16 x 16 (row), b 16 x 8 (column), bf16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles I and I + 4 of a word of eight codes, as the bf16 pair (code - bias): 0x4300 is
// 128.0 in bf16, whose last seven bits count in ones, so 0x4300 | c = 128 + c, and
// `minus` = (128 + bias) twice is taken off exactly.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t minus) {
    uint32_t t, r;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(t) : "r"(I ? w >> (4 * I) : w));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(minus));
    return r;
}
constexpr uint32_t kMinus8 = 0x43084308u;   // 136.0 twice: codes as -8 .. 7

// The same in f16, whose ten bits after the point hold a second nibble in place: 0x6400 is
// 1024.0, 0x6400 | c = 1024 + c, and 0x6400 | c << 4 = 1024 + 16 c, of which
// (1024 + 16 c) / 16 - 72 = c - 8.  Word w of eight codes: pairs (0, 4), (1, 5) of `w` and
// (2, 6), (3, 7) of `w >> 8`, nine instructions where bf16 takes eleven.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&out)[4]) {
    const uint32_t h = w >> 8;
    uint32_t t[4];
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(t[0]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(t[1]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(t[2]) : "r"(h));
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(t[3]) : "r"(h));
    constexpr uint32_t k1032 = 0x64086408u, kSixteenth = 0x2C002C00u, kMinus72 = 0xD480D480u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[0]) : "r"(t[0]), "r"(k1032));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out[1]) : "r"(t[1]), "r"(kSixteenth), "r"(kMinus72));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[2]) : "r"(t[2]), "r"(k1032));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out[3]) : "r"(t[3]), "r"(kSixteenth), "r"(kMinus72));
}

// c += a b as mma16816, f16 operands.
__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^x to about 2 ulp; 2^-inf = 0.
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float log2_approx(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 1 / x to about 1 ulp.
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace lora
