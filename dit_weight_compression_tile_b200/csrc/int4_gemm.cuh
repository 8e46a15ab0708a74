// What the products with a 4-bit group-scaled weight share (int4_gemm.cu, int4_gemv.cu).
#pragma once
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

constexpr int64_t kGemvTokens = 16;  // ep_int4_linear: up to here the weights' stream bounds it (int4_gemv.cu)
int int4_gemv(const Int4Args &a, int32_t dtype, int sms, cudaStream_t s);

// codes 2 i, 2 i + 1 of a word as a pair of exact 16-bit integers: the code's four bits below the bits of
// 128 (BF16) or 1024 (FP16), whose last place is 1, minus 136 or 1032
template <typename T>
__device__ __forceinline__ uint32_t code_pair(uint32_t word, uint32_t i) {
    using Pair = typename Elem<T>::Pair;
    const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | Elem<T>::kMagic;
    const uint32_t off = Elem<T>::kMagic | 0x00080008u;
    const Pair d = __hsub2(*reinterpret_cast<const Pair *>(&v), *reinterpret_cast<const Pair *>(&off));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// all threads of the cluster's CTAs; shared memory written before it is visible to the others after it
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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
