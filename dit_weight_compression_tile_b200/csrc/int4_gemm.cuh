// What the products with a 4-bit group-scaled weight share (int4_gemm.cu, int4_gemv.cu).
#pragma once
#include <cuda.h>

#include "device_util.cuh"
#include "int4.cuh"

namespace ep {

struct Int4Args {
    const uint32_t *codes;   // the weight's codes, `words` per row
    const uint16_t *scales;  // n x groups
    const uint16_t *x;       // activations (m x k) or the output's gradient (m x n), rows ldx apart
    const int8_t *act;       // checkpoint codes and scales
    const float *act_scales;
    const uint16_t *bias;
    uint16_t *out;           // m x n, m x k or n x groups
    uint32_t *status;
    int64_t ldx;
    int64_t m;
    uint32_t n, k, group, groups, words, act_groups;
};

// the current device's SM count (0: no device), looked up once per device
int device_sms();

// ep_int4_linear: up to so many tokens (two token tiles) int4_gemv.cu, above it the tcgen05 kernel.  Measured with
// 16 tokens, the former against the latter: 1024 x 1024 2.7 us against 6.6, 4096 x 4096 6.9 against 11.0,
// 8192 x 28672 48.6 against 82.0, 8192 x 8192 in groups of 32 22.6 against 32.0 (17 tokens, 57 us at 8192 x 28672, would
// need a third tile)
constexpr int64_t kGemvTokens = 16;
int int4_gemv(const Int4Args &a, int32_t dtype, int sms, cudaStream_t s);

// The eight codes of a word as four pairs of exact 16-bit numbers q / 4 (BF16) or q (FP16): pair i holds
// inputs 2 i, 2 i + 1.  Two shiftless masks, one shift, two masks, each followed by one fused
// multiply-add:
//   bits 0-3 under the exponent of 128 (BF16) or 1024 (FP16), where they count ones: (128 + c) / 4 - 34,
//     1024 + c - 1032;
//   bits 4-7: FP16 under 1024, counting 16: (1024 + 16 c) / 16 - 72.  BF16's mantissa ends at bit 6, but
//     with a zero exponent above, bit 7 is the exponent's last place, and the subnormals and the first
//     binade have the same spacing: the bits are the number c 2^-129; c 2^-129 2^127 - 2 = (c - 8) / 4.
// (One shift per pair instead costs 7 integer instructions per word against 5, on the pipe that is the
// busiest here.)
template <typename T>
struct Codes;
template <>
struct Codes<__nv_bfloat16> {
    static constexpr float kUnit = 4.0f;  // times this is q
    __device__ static uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t d;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
        return d;
    }
    __device__ static uint32_t low(uint32_t w) { return fma2((w & 0x000f000fu) | 0x43004300u, 0x3e803e80u, 0xc208c208u); }
    __device__ static uint32_t high(uint32_t w) { return fma2(w & 0x00f000f0u, 0x7f007f00u, 0xc000c000u); }
};
template <>
struct Codes<__half> {
    static constexpr float kUnit = 1.0f;
    __device__ static uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
        return d;
    }
    __device__ static uint32_t low(uint32_t w) { return fma2((w & 0x000f000fu) | 0x64006400u, 0x3c003c00u, 0xe408e408u); }
    __device__ static uint32_t high(uint32_t w) { return fma2((w & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd480d480u); }
};
template <typename T>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&d)[4]) {
    const uint32_t v = w >> 8;
    d[0] = Codes<T>::low(w);
    d[1] = Codes<T>::high(w);
    d[2] = Codes<T>::low(v);
    d[3] = Codes<T>::high(v);
}

// Tensor maps (encoded by the driver on the host, passed to kernels as parameters) of a row-major matrix
// with rows `pitch` bytes apart (a multiple of 16, as the base address): boxes of box_cols x box_rows
// elements with the 32-, 64- or 128-byte swizzle that fits a box's row, zeros outside the matrix.
bool tensor_map(CUtensorMap *map, const void *base, CUtensorMapDataType type, uint32_t elt, uint64_t cols, uint64_t rows,
                uint64_t pitch, uint32_t box_cols, uint32_t box_rows);

// the box at (col, row) into shared memory, completing on an mbarrier
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint32_t col, uint32_t row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(col), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&v)[4], uint32_t a) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
}

// all threads of the cluster's CTAs; shared memory written before it is visible to the others after it
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// a float of the shared memory of the cluster's CTA `rank`, at the place of this CTA's `p`
__device__ __forceinline__ float ld_cluster(const float *p, uint32_t rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
}

}  // namespace ep
