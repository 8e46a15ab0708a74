// The 4-bit group-scaled weight: its quantizer and its reconstruction, and 8-bit activation checkpoints
// (ep_int4_quantize, ep_int4_dequantize, ep_act8_pack, ep_act8_unpack).  All four read and write each
// element once: HBM's time is the floor.  None reaches it: instructions bound them, as stands beside each.
#include <algorithm>

#include "int4_gemm.cuh"

namespace ep {
namespace {

// a load of eight consecutive elements (valid ones; the others 0) as fp32
template <typename T>
__device__ __forceinline__ void load8(const T *p, int64_t valid, bool aligned, float (&v)[8]) {
    if (aligned && valid >= 8) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
            const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = Elem<T>::f(uint16_t(r[i]));
                v[2 * i + 1] = Elem<T>::f(uint16_t(r[i] >> 16));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4)
                v[i] = i < valid ? __ldg(reinterpret_cast<const float *>(p) + i) : 0.0f;
            else
                v[i] = i < valid ? Elem<T>::f(__ldg(reinterpret_cast<const uint16_t *>(p) + i)) : 0.0f;
        }
    }
}

// the largest magnitude of a group as bits (a NaN or infinity gives at least 0x7f800000): `lanes`
// neighbouring lanes share it
__device__ __forceinline__ uint32_t group_top(const float (&v)[8], int lanes) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) u = max(u, __float_as_uint(v[i]) & 0x7fffffffu);
    for (int d = lanes / 2; d > 0; d >>= 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, d));
    return u;
}

// 16 elements of a row as they are stored (beyond `valid`: 0)
template <typename T>
struct Raw16 {
    static constexpr int kWords = 4 * int(sizeof(T));
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p, int64_t valid, bool aligned) {
        if (aligned && valid >= 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = i < valid ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0u;
                } else {
                    const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
                    const uint32_t lo = 2 * i < valid ? __ldg(h + 2 * i) : 0u, hi = 2 * i + 1 < valid ? __ldg(h + 2 * i + 1) : 0u;
                    w[i] = lo | (hi << 16);
                }
            }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return Elem<T>::f(uint16_t(w[i / 2] >> (16 * (i & 1))));
    }
    // the largest magnitude as fp32 bits, at least those of infinity where there is a NaN or an infinity:
    // magnitudes order as integers, two at a time in 16-bit halves
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) m = max(m, w[i] & 0x7fffffffu);
            else m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        }
        if constexpr (sizeof(T) == 4) {
            return m;
        } else {
            const uint32_t h = max(m & 0xffffu, m >> 16);
            return __float_as_uint(Elem<T>::f(uint16_t(h))) | (h >= Elem<T>::kInf ? 0x7f800000u : 0u);
        }
    }
};

__device__ __forceinline__ float fma_sat(float a, float b, float c) {
    float d;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Whether x / a can be an exact half that the first rounding does not already send to the even integer.  An
// odd multiple of a / 2 has at least a's digits, so a must be no longer than x; a = m 2^e / 127 with m an integer of
// x's length is an integer times 2^e, or periodic and as long as an fp32 can be; and for a power of two the
// reciprocal and the rounding are exact.  BF16's m, below 256, leave 127 and 254: powers of two.
template <typename T>
constexpr bool kHalves = true;
template <>
constexpr bool kHalves<__nv_bfloat16> = false;

// the exact way, for the groups that need it (a call: written in place it cost every group 4 us in 27)
struct Slow16 {
    float x[16];
    uint32_t w[4];
};
__device__ __noinline__ void act8_codes_slow(Slow16 *p, bool bad, float a) {
    const float up = quotient_unit(a), s = a * up, inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w |= (uint32_t(bad ? 0 : quotient_code(p->x[4 * i + e] * up, s, inv, 127.0f)) & 0xffu) << (8 * e);
        p->w[i] = w;
    }
}

struct PackArgs {
    int64_t ldx, total;  // groups of all tokens
    int64_t step_t;      // a CTA's next 32 groups are step_t tokens and step_g groups on
    uint32_t k, groups, step_g;
    bool aligned;
};

// Checkpoint: 8 lanes hold one group of 128 features, 16 each.  Scale a = max / 127 (rounded; 1 where
// that is 0, NaN where the group has a NaN or an infinity, whose codes are 0).  q = x (1 / a) + 1.5 2^23 in
// one fused multiply-add has the nearest integer in its low bits, wrong at most next to a half; the
// remainder x - q a is exact (a multiple of a's last place, at most about a / 2) and says whether the next
// integer is nearer, or (kHalves) as near and even: two saturated multiply-adds give the 0 or 1 to add and to
// subtract, on the pipe that has room.  Tiny a go by quotient_code.  With BF16 activations the quotients are
// fractions of small numbers, and nine warps in ten have one next to a half: a slow path for all of those
// took 34 us for 4096 x 8192, comparing and selecting 26 us, rintf and a conversion for each element, on a
// half-rate pipe, 42 us.  This form takes 23.9 us (FP16 26.1; copying alone 16.3, the floor 15.6): the
// instructions bound it (issue slots 79 %, ALU pipe 49 %, FMA pipe 43 % busy).  CTAs walk over the groups with the next one's
// loads in flight.
constexpr int kPackBlocks = 5;  // CTAs on an SM (4: the same; 6, with fewer registers: 27.6 us)
template <typename T>
__global__ void __launch_bounds__(256, kPackBlocks) act8_pack_kernel(const T *x, int8_t *codes, float *scales, const PackArgs p) {
    const uint32_t l = threadIdx.x & 7u;
    const int64_t row = act8_row_bytes(p.k);
    int64_t unit = int64_t(blockIdx.x) * 32 + (threadIdx.x >> 3);  // (token, group)
    int64_t t = uint32_t(unit) / p.groups;  // (the first groups' index has 32 bits)
    uint32_t g = uint32_t(unit) % p.groups;
    Raw16<T> next;
    next.load(x + t * p.ldx + g * kActGroup + l * 16, unit < p.total ? int64_t(p.k) - int64_t(g * kActGroup + l * 16) : 0, p.aligned);
    while (__any_sync(0xffffffffu, unit < p.total)) {
        const Raw16<T> v = next;
        const int64_t u0 = unit, t0 = t;
        const uint32_t k0 = g * kActGroup + l * 16;
        const bool in = unit < p.total;
        unit += int64_t(gridDim.x) * 32;
        t += p.step_t;
        g += p.step_g;
        if (g >= p.groups) g -= p.groups, ++t;
        if (unit < p.total) next.load(x + t * p.ldx + g * kActGroup + l * 16, int64_t(p.k) - int64_t(g * kActGroup + l * 16), p.aligned);
        uint32_t top = in ? v.top() : 0u;
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        float a = __fdiv_rn(__uint_as_float(top), 127.0f);
        if (a == 0.0f) a = 1.0f;
        const bool bad = top >= 0x7f800000u;
        if (bad) a = __uint_as_float(0x7fffffffu);
        // B = 2^(30 - e) for a in [2^e, 2^(e + 1)): the difference of two multiples of a's last place (halved)
        // is 0 or at least 64 after it, so that the saturated product is 0 or 1
        const uint32_t ab = __float_as_uint(a);
        const float half = 0.5f * a, inv = __frcp_rn(a), unit_ = 12582912.0f;
        const float B = __uint_as_float((284u << 23) - (ab & 0x7f800000u)), halfB = half * B;
        const bool exact = bad || a < 0x1p-90f;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f = v.at(4 * i + e), r = __fmaf_rn(f, inv, unit_);
                const float rest = __fmaf_rn(unit_ - r, a, f);  // x - q a, exact
                // (an odd q gives way at half already: from half on, the sum is at least half a last place of halfB)
                const float limit = kHalves<T> ? __uint_as_float(__float_as_uint(-halfB) - (__float_as_uint(r) & 1u)) : -halfB;
                b[e] = __float_as_uint(r + fma_sat(rest, B, limit) - fma_sat(-rest, B, limit));
            }
            w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
        if (exact) {
            Slow16 slow;
#pragma unroll
            for (int i = 0; i < 16; ++i) slow.x[i] = v.at(i);
            act8_codes_slow(&slow, bad, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = slow.w[i];
        }
        if (in && k0 < row) *reinterpret_cast<uint4 *>(codes + t0 * row + k0) = make_uint4(w[0], w[1], w[2], w[3]);
        if (in && l == 0) scales[u0] = a;
    }
}

// place i of rows of `by`: its row and its place there (a 64-bit division only where i has more bits)
__device__ __forceinline__ int64_t row_of(int64_t i, uint32_t by, uint32_t &rest) {
    if (i >> 32) {
        rest = uint32_t(i % by);
        return i / by;
    }
    rest = uint32_t(i) % by;
    return uint32_t(i) / by;
}

// eight elements of a row, `valid` of them, rounded to T; `wide`: every row begins on 16 bytes
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8], uint32_t valid, bool wide) {
    if constexpr (sizeof(T) == 4) {
        if (wide && valid >= 8) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
            return;
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j < valid) p[j] = v[j];
    } else {
        uint16_t h[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) h[j] = Elem<T>::bits(v[j]);
        if (wide && valid >= 8) {
            const auto two = [&](int j) { return h[j] | (uint32_t(h[j + 1]) << 16); };
            *reinterpret_cast<uint4 *>(p) = make_uint4(two(0), two(2), two(4), two(6));
            return;
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (j < valid) reinterpret_cast<uint16_t *>(p)[j] = h[j];
    }
}

// x = RNE(a c) in the output's type.  A thread for eight features (8192 x 8192 to BF16: 51.5 us of a floor of 31;
// with a store for each element 150 us).  The conversions from integers bound it: the pipe that they run on is 71 %
// busy, the issue slots 51 %, DRAM 34 %.
template <typename T>
__global__ void __launch_bounds__(256) act8_unpack_kernel(const int8_t *codes, const float *scales, uint32_t k,
                                                          uint32_t groups, int64_t total, T *out, bool wide) {
    const uint32_t chunks = (k + 7) / 8;
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    uint32_t k0;
    const int64_t t = row_of(i, chunks, k0);
    k0 *= 8;
    const float a = __ldg(scales + t * groups + k0 / kActGroup);
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(codes + t * act8_row_bytes(k) + k0));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = a * float(int8_t((j < 4 ? w.x : w.y) >> (8 * (j & 3))));
    store8(out + t * int64_t(k) + k0, v, k - k0, wide);
}

// Weight: a lane per word of eight inputs, group / 8 neighbouring lanes per group.  Scale s = max / 7
// rounded to fp32 and then to S (1 where that is 0, NaN with codes 0 where the group has a NaN or an
// infinity); codes in -7 .. 7.  The exact quotients' instructions bound it (8192 x 8192 BF16, groups of 128:
// 105 us of a floor of 26; issue slots 86 % busy, ALU pipe 61 %, conversions' pipe 55 %, DRAM 17 %): a weight is
// quantized once.
template <typename T, typename S>
__global__ void __launch_bounds__(256) int4_quantize_kernel(const T *w, int64_t ldw, uint32_t k, uint32_t group,
                                                            uint32_t row_lanes, int64_t total, uint32_t *codes,
                                                            S *scales, bool aligned) {
    const int64_t id = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;  // row_lanes (a multiple of 16) per row
    const bool in = id < total;
    uint32_t j;
    const int64_t o = row_of(in ? id : 0, row_lanes, j);
    const uint32_t k0 = 8 * j;
    float v[8];
    load8<T>(w + o * ldw + k0, in ? int64_t(k) - k0 : 0, aligned, v);
    const uint32_t lanes = group / 8, top = group_top(v, int(lanes));
    const uint16_t sb = Elem<S>::bits(__fdiv_rn(__uint_as_float(top), 7.0f));
    float s = Elem<S>::f(sb);
    const bool bad = !(s < __uint_as_float(0x7f800000u));  // also a scale that overflows S
    if (s == 0.0f) s = 1.0f;
    if (bad) s = __uint_as_float(0x7fffffffu);
    const float unit = quotient_unit(s), su = s * unit, inv = __frcp_rn(su);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = bad ? 0 : quotient_code(v[i] * unit, su, inv, 7.0f);
        word |= uint32_t(c + 8) << (4 * (i / 2) + 16 * (i & 1));
    }
    const uint32_t words = uint32_t(int4_row_bytes(k) / 4), groups = (k + group - 1) / group;
    if (in && j < words) codes[o * words + j] = word;
    if (in && j % lanes == 0 && k0 < k)
        reinterpret_cast<uint16_t *>(scales)[o * groups + j / lanes] = bad ? uint16_t(0x7fffu) : Elem<S>::bits(s);
}

// W = RNE(s q): a thread for a word of eight inputs (8192 x 8192: 49.6 us of a floor of 26; with a store for each
// element 139 us).  Instructions bound it: issue slots 77 % busy, ALU pipe 61 %, conversions' pipe 54 %, DRAM 26 %.
template <typename S>
__global__ void __launch_bounds__(256) int4_dequantize_kernel(const uint32_t *codes, const S *scales, uint32_t k,
                                                              uint32_t group, int64_t total, S *out, bool wide) {
    const uint32_t used = (k + 7) / 8, words = uint32_t(int4_row_bytes(k) / 4), groups = (k + group - 1) / group;
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    uint32_t j;
    const int64_t o = row_of(i, used, j);
    const uint32_t w = __ldg(codes + o * words + j);
    const float s = Elem<S>::f(__ldg(reinterpret_cast<const uint16_t *>(scales) + o * groups + 8 * j / group));
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s * float(int((w >> (4 * (e / 2) + 16 * (e & 1))) & 15u) - 8);
    store8(out + o * int64_t(k) + 8 * j, v, k - 8 * j, wide);
}

bool is16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool blocks_of(int64_t threads, unsigned *grid) {
    const int64_t b = (threads + 255) / 256;
    *grid = unsigned(b);
    return b <= 0x7fffffff;
}
constexpr int64_t kMaxDim = int64_t(1) << 30;

}  // namespace
}  // namespace ep

extern "C" int ep_act8_pack(const void *d_x, int32_t dtype, int64_t m, int64_t k, int64_t ldx, void *d_codes,
                            float *d_scales, ep_stream_t stream) {
    using namespace ep;
    if (m < 0 || m > kMaxDim || k < 1 || k > kMaxDim || (m > 1 && ldx < k)) return EP_ERR_INVALID_ARG;
    if (dtype != EP_BF16 && dtype != EP_FP16 && dtype != EP_FP32) return EP_ERR_INVALID_ARG;
    if (m == 0) return EP_OK;
    const uint32_t elt = dtype == EP_FP32 ? 4 : 2;
    if (!d_x || !d_codes || !d_scales || (reinterpret_cast<uintptr_t>(d_x) & (elt - 1)) || !is16(d_codes) ||
        (reinterpret_cast<uintptr_t>(d_scales) & 3u))
        return EP_ERR_INVALID_ARG;
    const uint32_t groups = uint32_t((k + kActGroup - 1) / kActGroup);
    if (m > INT64_MAX / 64 / groups) return EP_ERR_UNSUPPORTED;
    PackArgs p{};
    p.ldx = ldx;
    p.total = m * groups;
    p.k = uint32_t(k);
    p.groups = groups;
    p.aligned = is16(d_x) && (m == 1 || ldx * elt % 16 == 0);
    const int sms = device_sms();
    if (sms < 1) return EP_ERR_CUDA;
    const unsigned grid = unsigned(std::min<int64_t>((p.total + 31) / 32, int64_t(sms) * kPackBlocks));
    p.step_t = int64_t(grid) * 32 / groups;
    p.step_g = uint32_t(int64_t(grid) * 32 % groups);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto *c = static_cast<int8_t *>(d_codes);
    if (dtype == EP_BF16)
        act8_pack_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(d_x), c, d_scales, p);
    else if (dtype == EP_FP16)
        act8_pack_kernel<<<grid, 256, 0, s>>>(static_cast<const __half *>(d_x), c, d_scales, p);
    else
        act8_pack_kernel<<<grid, 256, 0, s>>>(static_cast<const float *>(d_x), c, d_scales, p);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

extern "C" int ep_act8_unpack(const void *d_codes, const float *d_scales, int64_t m, int64_t k, void *d_out,
                              int32_t dtype, ep_stream_t stream) {
    using namespace ep;
    if (m < 0 || m > kMaxDim || k < 1 || k > kMaxDim) return EP_ERR_INVALID_ARG;
    if (dtype != EP_BF16 && dtype != EP_FP16 && dtype != EP_FP32) return EP_ERR_INVALID_ARG;
    if (m == 0) return EP_OK;
    const uint32_t elt = dtype == EP_FP32 ? 4 : 2;
    if (!d_out || !d_codes || !d_scales || (reinterpret_cast<uintptr_t>(d_out) & (elt - 1)) || !is16(d_codes) ||
        (reinterpret_cast<uintptr_t>(d_scales) & 3u))
        return EP_ERR_INVALID_ARG;
    const uint32_t groups = uint32_t((k + kActGroup - 1) / kActGroup), chunks = uint32_t((k + 7) / 8);
    if (m > INT64_MAX / 64 / chunks) return EP_ERR_UNSUPPORTED;
    const int64_t total = m * chunks;
    unsigned grid;
    if (!blocks_of(total, &grid)) return EP_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto *c = static_cast<const int8_t *>(d_codes);
    const bool wide = is16(d_out) && k * elt % 16 == 0;
    if (dtype == EP_BF16)
        act8_unpack_kernel<<<grid, 256, 0, s>>>(c, d_scales, uint32_t(k), groups, total, static_cast<__nv_bfloat16 *>(d_out), wide);
    else if (dtype == EP_FP16)
        act8_unpack_kernel<<<grid, 256, 0, s>>>(c, d_scales, uint32_t(k), groups, total, static_cast<__half *>(d_out), wide);
    else
        act8_unpack_kernel<<<grid, 256, 0, s>>>(c, d_scales, uint32_t(k), groups, total, static_cast<float *>(d_out), wide);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

namespace ep {
namespace {
template <typename T>
int quantize_from(const void *w, int64_t ldw, int64_t n, int64_t k, int32_t group, void *codes, void *scales,
                  int32_t scale_dtype, bool aligned, cudaStream_t s) {
    const uint32_t row_lanes = uint32_t((k + 127) / 128 * 16);
    if (n > INT64_MAX / 64 / row_lanes) return EP_ERR_UNSUPPORTED;
    const int64_t total = n * row_lanes;
    unsigned grid;
    if (!blocks_of(total, &grid)) return EP_ERR_UNSUPPORTED;
    auto *c = static_cast<uint32_t *>(codes);
    if (scale_dtype == EP_BF16)
        int4_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const T *>(w), ldw, uint32_t(k), uint32_t(group), row_lanes,
                                                  total, c, static_cast<__nv_bfloat16 *>(scales), aligned);
    else
        int4_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const T *>(w), ldw, uint32_t(k), uint32_t(group), row_lanes,
                                                  total, c, static_cast<__half *>(scales), aligned);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
}  // namespace
}  // namespace ep

extern "C" int ep_int4_quantize(const void *d_w, int32_t dtype, int64_t n, int64_t k, int64_t ldw, int32_t group,
                                void *d_codes, void *d_scales, int32_t scale_dtype, ep_stream_t stream) {
    using namespace ep;
    if (n < 1 || n > kMaxDim || k < 1 || k > kMaxDim || (n > 1 && ldw < k)) return EP_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return EP_ERR_INVALID_ARG;
    if (dtype != EP_BF16 && dtype != EP_FP16 && dtype != EP_FP32) return EP_ERR_INVALID_ARG;
    if (scale_dtype != EP_BF16 && scale_dtype != EP_FP16) return EP_ERR_INVALID_ARG;
    const uint32_t elt = dtype == EP_FP32 ? 4 : 2;
    if (!d_w || !d_codes || !d_scales || (reinterpret_cast<uintptr_t>(d_w) & (elt - 1)) || !is16(d_codes) ||
        (reinterpret_cast<uintptr_t>(d_scales) & 1u))
        return EP_ERR_INVALID_ARG;
    const bool aligned = is16(d_w) && (n == 1 || ldw * elt % 16 == 0);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == EP_BF16)
        return quantize_from<__nv_bfloat16>(d_w, ldw, n, k, group, d_codes, d_scales, scale_dtype, aligned, s);
    if (dtype == EP_FP16)
        return quantize_from<__half>(d_w, ldw, n, k, group, d_codes, d_scales, scale_dtype, aligned, s);
    return quantize_from<float>(d_w, ldw, n, k, group, d_codes, d_scales, scale_dtype, aligned, s);
}

extern "C" int ep_int4_dequantize(const void *d_codes, const void *d_scales, int32_t dtype, int64_t n, int64_t k,
                                  int32_t group, void *d_out, ep_stream_t stream) {
    using namespace ep;
    if (n < 1 || n > kMaxDim || k < 1 || k > kMaxDim) return EP_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return EP_ERR_INVALID_ARG;
    if (dtype != EP_BF16 && dtype != EP_FP16) return EP_ERR_INVALID_ARG;
    if (!d_codes || !d_scales || !d_out || !is16(d_codes) ||
        ((reinterpret_cast<uintptr_t>(d_scales) | reinterpret_cast<uintptr_t>(d_out)) & 1u))
        return EP_ERR_INVALID_ARG;
    const uint32_t used = uint32_t((k + 7) / 8);
    const int64_t total = n * used;
    unsigned grid;
    if (!blocks_of(total, &grid)) return EP_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto *c = static_cast<const uint32_t *>(d_codes);
    const bool wide = is16(d_out) && k % 8 == 0;
    if (dtype == EP_BF16)
        int4_dequantize_kernel<<<grid, 256, 0, s>>>(c, static_cast<const __nv_bfloat16 *>(d_scales), uint32_t(k),
                                                    uint32_t(group), total, static_cast<__nv_bfloat16 *>(d_out), wide);
    else
        int4_dequantize_kernel<<<grid, 256, 0, s>>>(c, static_cast<const __half *>(d_scales), uint32_t(k),
                                                    uint32_t(group), total, static_cast<__half *>(d_out), wide);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
