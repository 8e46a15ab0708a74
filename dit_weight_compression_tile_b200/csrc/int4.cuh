// The 4-bit group-scaled weight and the 8-bit activation checkpoint: storage and element arithmetic
// shared by their kernels (int4.cu, int4_gemm.cu).
//
// Weight: W[o, k] = s[o, k / group] q[o, k], q in -8 .. 7, group 32, 64 or 128, s BF16 or FP16 (the type
// of the activations).  Codes: row o holds words(k) 32-bit words of eight codes each; word w holds inputs
// 8 w .. 8 w + 7 as q + 8 in four bits, inputs 0, 2, 4, 6 of the eight in bits 0, 4, 8, 12 and inputs
// 1, 3, 5, 7 in bits 16, 20, 24, 28, so that (word >> 4 i) & 0x000f000f is the pair of inputs 2 i, 2 i + 1
// in the two halves of a register.  Rows are padded with q = 0 to a multiple of 32 inputs (16 bytes).
//
// Checkpoint: x[t, k] ~ a[t, k / 128] c[t, k], c in -127 .. 127, a fp32; rows of codes padded with 0 to a
// multiple of 16 features.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/eptile_int4.h"

namespace ep {

constexpr uint32_t kActGroup = 128;

__host__ __device__ constexpr int64_t int4_row_bytes(int64_t k) { return (k + 31) / 32 * 16; }
__host__ __device__ constexpr int64_t act8_row_bytes(int64_t k) { return (k + 15) / 16 * 16; }

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    using Pair = __nv_bfloat162;
    static constexpr uint32_t kMagic = 0x43004300u;  // 128 + c for c < 128
    static constexpr uint32_t kInf = 0x7f80u;
    __device__ static float f(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
    __device__ static uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <>
struct Elem<__half> {
    using Pair = __half2;
    static constexpr uint32_t kMagic = 0x64006400u;  // 1024 + c for c < 1024
    static constexpr uint32_t kInf = 0x7c00u;
    __device__ static float f(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    __device__ static uint16_t bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

// The code of x for scale s: the integer nearest the exact quotient x / s, ties to even, in -top .. top.
// `inv` is 1 / s rounded; t = x inv is off by less than 2^-22 top, so rint(t) can only be wrong next to a
// half; there the sign of x - s h (h the half, an exact product and sum under fma, which keeps the sign)
// decides.  s and x scaled by `quotient_unit` so that the difference does not underflow.
__device__ __forceinline__ float quotient_unit(float s) { return s < 0x1p-100f ? 0x1p64f : 1.0f; }
__device__ __forceinline__ int quotient_code(float x, float s, float inv, float top) {
    const float t = x * inv;
    float q = rintf(t);
    const float d = t - q;
    if (fabsf(d) > 0.498f) {
        const float h = q + (d > 0.0f ? 0.5f : -0.5f), lo = h - 0.5f, hi = h + 0.5f;
        const float e = __fmaf_rn(-s, h, x);
        q = e > 0.0f ? hi : e < 0.0f ? lo : 2.0f * rintf(0.5f * h);  // a tie: the even one of lo and hi
    }
    return __float2int_rn(fminf(fmaxf(q, -top), top));
}

}  // namespace ep
