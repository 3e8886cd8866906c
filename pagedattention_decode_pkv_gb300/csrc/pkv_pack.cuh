// Packed and mixed-precision arithmetic of the prefill kernels' softmax
// (two f32 values in one 64-bit register, or a pair of 16-bit ones).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace pkv {
namespace {

// acc + the low 16-bit value of w (lo) and acc2 + the high one, in f32: the
// mixed-precision adds take the 16-bit operand as it is (exact widening).
template <typename T> __device__ __forceinline__ void pair_acc(uint32_t w, float &acc, float &acc2);
template <> __device__ __forceinline__ void pair_acc<__nv_bfloat16>(uint32_t w, float &acc, float &acc2) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
        : "+f"(acc), "+f"(acc2)
        : "r"(w));
}
template <> __device__ __forceinline__ void pair_acc<__half>(uint32_t w, float &acc, float &acc2) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "add.rn.f32.f16 %0, lo, %0;\n\tadd.rn.f32.f16 %1, hi, %1;\n\t}"
        : "+f"(acc), "+f"(acc2)
        : "r"(w));
}

// tanh(u) = u (f0 + f1 u^2 + .. + f4 u^8) for |u| <= kTanhLimit: the minimax fit in relative error, 3e-7
constexpr float kTanhLimit = 0.7f;
constexpr double kTanhFit[5] = {0.9999996973, -0.3333021287, 0.1328111218, -0.05083622068, 0.0137736928};

// max(a, b, c) in one instruction (three-input max; NaN operands are ignored
// as by fmaxf).
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// (x0, x1) * s + c per lane, both fused and rounded once (one packed f32x2 FMA);
// s2 / c2 hold the same value in both halves.
__device__ __forceinline__ void fma_x2(float x0, float x1, uint64_t s2, uint64_t c2, float &e0, float &e1) {
    asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\t"
        "fma.rn.f32x2 d, a, %4, %5;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(e0), "=f"(e1)
        : "f"(x0), "f"(x1), "l"(s2), "l"(c2));
}

__device__ __forceinline__ uint64_t splat2(float v) {
    const uint64_t u = __float_as_uint(v);
    return u | u << 32;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace
}  // namespace pkv
