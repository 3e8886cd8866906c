// The 4-bit KV cache: its layout, the encoding of a row and the widening of codes, shared by
// the kernels that write, read back and attend over it.
//
// A row (one token of one KV head) is head_dim / 2 bytes of codes and one f16 scale per 32
// dims; codes are [num_blocks, Hkv, block_size, d / 2], scales [num_blocks, Hkv, block_size,
// d / 32], so that what an attention kernel reads of a (block, head) is contiguous.  A nibble
// u stands for scale * (u - 8), u = 1 .. 15.  A 32-bit word holds eight dims, nibbles from the
// lowest: 0 2 4 6 1 3 5 7.  Then (w >> 4 j) & 0x000f000f is the pair of dims 2 j, 2 j + 1 in
// the two halves of a register, and OR-ed with 0x6400 each half is the f16 1024 + u: eight
// codes widen in nine operations, none of them a conversion.  (The interleaved order and these
// steps are a published method: Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run:
// Bringing Large Scale MoE Models into Cloud Scale Production", 2022.)
//
// The scale is max|x| / 7 rounded to bf16, then to f16, at most 9344.  Its eight significant
// bits make scale * code exact in f16 (three bits more), so that attention over the cache, the
// rows read back and the definition agree to the bit; 7 * 9344 is the largest such value f16
// holds.  The rounding of the scale costs nothing: codes are rounded under the stored scale.
// Scales are multiples of 2^-24: below 2^-17 they have fewer bits, and at the first few multiples
// the largest value may be 7.5 scales and more, which code 7 stands for.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {
namespace {

constexpr int kInt4Group = 32;         // dims that share a scale
constexpr float kInt4TopScale = 9344.f;
constexpr float kInt4TopInput = 3e38f;  // larger maxima are taken as this; both have the largest scale

// The bf16 nearest to top / 7 (ties to even) for top >= 0, exactly: the remainder of a midpoint
// says on which side of it the quotient is, and an f32 product off by a few 2^-24 always finds
// the midpoint that matters.
__device__ __forceinline__ float int4_seventh_bf16(float top, float &mid) {
    const uint32_t lo = __float_as_uint(top * 0.14285714924335479736328125f) & 0xffff0000u;
    mid = __uint_as_float(lo | 0x8000u);
    const float side = fmaf(-7.f, mid, top);
    const bool up = side > 0.f || (side == 0.f && (lo & 0x10000u));
    return __uint_as_float(up ? lo + 0x10000u : lo);
}

// The stored scale of a group whose largest magnitude is `top` (NaN left out by the caller), and
// the midpoint of two bf16 values nearest to top / 7.
__device__ __forceinline__ __half int4_scale(float top, float &mid) {
    const float s = int4_seventh_bf16(fminf(top, kInt4TopInput), mid);
    return __float2half_rn(fminf(s, kInt4TopScale));
}

// Code of x under the scale s > 0: the integer nearest to x / s, ties to even, within +-7,
// decided by the exact remainder (inv = 1 / s is rounded).  NaN gives 0.
__device__ __forceinline__ int int4_code(float x, float s, float inv) {
    float c = rintf(fminf(fmaxf(x * inv, -8.f), 8.f));
    const float r = fmaf(-c, s, x), h = 0.5f * s;
    if (fabsf(r) > h || (fabsf(r) == h && (static_cast<int>(c) & 1))) c += r > 0.f ? 1.f : -1.f;
    return x == x ? static_cast<int>(fminf(fmaxf(c, -7.f), 7.f)) : 0;
}

// The place of dim j's nibble in its word.
__device__ __forceinline__ constexpr int int4_shift(int j) { return 4 * (j >> 1) + 16 * (j & 1); }

// One word -> the f16 pairs (0, 1), (2, 3), (4, 5), (6, 7) of u - 8, exactly.
__device__ __forceinline__ void int4_widen(uint32_t w, uint32_t (&p)[4]) {
    const uint32_t v = w >> 8;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(p[0]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(p[1]) : "r"(w));
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(p[2]) : "r"(v));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(p[3]) : "r"(v));
    // 1024 + u - 1032, and (1024 + 16 u) / 16 - 72
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(p[0]) : "r"(0x64086408u));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(p[1]) : "r"(0x2c002c00u), "r"(0xd480d480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(p[2]) : "r"(0x64086408u));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(p[3]) : "r"(0x2c002c00u), "r"(0xd480d480u));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace
}  // namespace pkv
