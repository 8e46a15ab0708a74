// Products with a 4-bit group-scaled weight: the linear layer's forward (ep_int4_linear), its input
// gradient (ep_int4_linear_dx) and the gradient of the group scales from an 8-bit activation
// checkpoint (ep_int4_scale_grad).
#include <algorithm>
#include <atomic>

#include "int4_gemm.cuh"

namespace ep {
namespace {

enum Product { kForward, kInputGrad, kScaleGrad };

template <typename T>
__device__ __forceinline__ float weight_code(const Int4Args &a, uint32_t o, uint32_t k) {
    const uint32_t w = __ldg(a.codes + int64_t(o) * a.words + k / 8), e = k & 7u;
    return float(int((w >> (4 * (e / 2) + 16 * (e & 1))) & 15u) - 8);
}
template <typename T>
__device__ __forceinline__ float weight_at(const Int4Args &a, uint32_t o, uint32_t k) {
    return weight_code<T>(a, o, k) * Elem<T>::f(__ldg(a.scales + int64_t(o) * a.groups + k / a.group));
}

// 64 x 128 tile of D[i, j] = sum_c A(i, c) B(c, j) in fp32, 32 deep steps through shared memory, 4 x 8
// per thread.  Forward: i token, j output feature, c input; input gradient: i token, j input, c output
// feature; scale gradient: i output feature, j input, c token (then the tile times the codes, summed
// over each group: 128 inputs hold whole groups).
template <typename T, int P>
__global__ void __launch_bounds__(256) int4_simple_kernel(const Int4Args a) {
    __shared__ float mem[64 * 129];  // the operands' steps, then (scale gradient) the tile
    auto sa = reinterpret_cast<float(*)[65]>(mem);
    auto sb = reinterpret_cast<float(*)[129]>(mem + 32 * 65);
    auto sd = reinterpret_cast<float(*)[129]>(mem);
    const int64_t I = P == kScaleGrad ? int64_t(a.n) : a.m, C = P == kForward ? a.k : P == kInputGrad ? int64_t(a.n) : a.m;
    const uint32_t J = P == kForward ? a.n : a.k;
    const int64_t i0 = int64_t(blockIdx.x) * 64;
    const uint32_t j0 = blockIdx.y * 128, ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float d[4][8] = {};
    for (int64_t c0 = 0; c0 < C; c0 += 32) {
        for (uint32_t e = threadIdx.x; e < 64 * 32; e += 256) {
            const uint32_t c = P == kScaleGrad ? e / 64 : e % 32, i = P == kScaleGrad ? e % 64 : e / 32;
            float v = 0.0f;
            if (i0 + i < I && c0 + c < C)
                v = Elem<T>::f(__ldg(P == kScaleGrad ? a.x + (c0 + c) * a.ldx + i0 + i : a.x + (i0 + i) * a.ldx + c0 + c));
            sa[c][i] = v;
        }
        for (uint32_t e = threadIdx.x; e < 128 * 32; e += 256) {
            const uint32_t c = P == kForward ? e % 32 : e / 128, j = P == kForward ? e / 32 : e % 128;
            float v = 0.0f;
            if (j0 + j < J && c0 + c < C) {
                if constexpr (P == kForward)
                    v = weight_at<T>(a, j0 + j, uint32_t(c0 + c));
                else if constexpr (P == kInputGrad)
                    v = weight_at<T>(a, uint32_t(c0 + c), j0 + j);
                else
                    v = float(a.act[(c0 + c) * act8_row_bytes(a.k) + j0 + j]) *
                        a.act_scales[(c0 + c) * a.act_groups + (j0 + j) / kActGroup];
            }
            sb[c][j] = v;
        }
        __syncthreads();
        for (uint32_t c = 0; c < 32; ++c)
            for (uint32_t y = 0; y < 4; ++y)
                for (uint32_t z = 0; z < 8; ++z) d[y][z] += sa[c][ti + 16 * y] * sb[c][tj + 16 * z];
        __syncthreads();
    }
    for (uint32_t y = 0; y < 4; ++y)
        for (uint32_t z = 0; z < 8; ++z) {
            const int64_t i = i0 + ti + 16 * y;
            const uint32_t j = j0 + tj + 16 * z;
            if constexpr (P == kScaleGrad) {
                sd[ti + 16 * y][tj + 16 * z] = i < I && j < J ? d[y][z] * weight_code<T>(a, uint32_t(i), j) : 0.0f;
            } else if (i < I && j < J) {
                const float b = P == kForward && a.bias ? Elem<T>::f(a.bias[j]) : 0.0f;
                a.out[i * J + j] = Elem<T>::bits(d[y][z] + b);
            }
        }
    if constexpr (P == kScaleGrad) {
        __syncthreads();
        const uint32_t per = 128 / a.group;
        for (uint32_t e = threadIdx.x; e < 64 * per; e += 256) {
            const uint32_t i = e / per, g = e % per;
            float s = 0.0f;
            for (uint32_t j = 0; j < a.group; ++j) s += sd[i][g * a.group + j];
            if (i0 + i < I && j0 / a.group + g < a.groups)
                a.out[(i0 + i) * a.groups + j0 / a.group + g] = Elem<T>::bits(s);
        }
    }
}

constexpr int64_t kMaxDim = int64_t(1) << 30;
bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool weight_ok(int64_t n, int64_t k, int32_t group, int32_t dtype) {
    return n >= 1 && n <= kMaxDim && k >= 1 && k <= kMaxDim && (group == 32 || group == 64 || group == 128) &&
           (dtype == EP_BF16 || dtype == EP_FP16);
}
Int4Args args_of(int64_t n, int64_t k, int32_t group, const void *codes, const void *scales) {
    Int4Args a{};
    a.codes = static_cast<const uint32_t *>(codes);
    a.scales = static_cast<const uint16_t *>(scales);
    a.n = uint32_t(n);
    a.k = uint32_t(k);
    a.group = uint32_t(group);
    a.groups = uint32_t((k + group - 1) / group);
    a.words = uint32_t(int4_row_bytes(k) / 4);
    a.act_groups = uint32_t((k + kActGroup - 1) / kActGroup);
    return a;
}
// the current device's SM count, looked up once per device
int device_sms() {
    static std::atomic<int> known[64];
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return 0;
    if ((sms = known[device].load()) == 0 &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess)
        known[device].store(sms);
    return sms;
}
template <int P>
int launch_simple(const Int4Args &a, int32_t dtype, cudaStream_t s) {
    const int64_t I = P == kScaleGrad ? int64_t(a.n) : a.m, J = P == kForward ? a.n : a.k;
    const dim3 grid(unsigned((I + 63) / 64), unsigned((J + 127) / 128));
    if ((I + 63) / 64 > 0x7fffffff || grid.y > 65535) return EP_ERR_UNSUPPORTED;
    if (dtype == EP_BF16)
        int4_simple_kernel<__nv_bfloat16, P><<<grid, 256, 0, s>>>(a);
    else
        int4_simple_kernel<__half, P><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

}  // namespace
}  // namespace ep

extern "C" int ep_int4_linear(const void *d_codes, const void *d_scales, int64_t n, int64_t k, int32_t group,
                              int32_t dtype, const void *d_x, int64_t m, int64_t ldx, const void *d_bias, void *d_y,
                              uint32_t *d_status, ep_stream_t stream) {
    using namespace ep;
    if (!weight_ok(n, k, group, dtype) || m < 0 || (m > 1 && ldx < k)) return EP_ERR_INVALID_ARG;
    if (m == 0) return EP_OK;
    if (!d_codes || !d_scales || !d_x || !d_y || misaligned(d_codes, 16) || misaligned(d_scales, 2) ||
        misaligned(d_x, 2) || misaligned(d_bias, 2) || misaligned(d_y, 2) || misaligned(d_status, 4))
        return EP_ERR_INVALID_ARG;
    Int4Args a = args_of(n, k, group, d_codes, d_scales);
    a.x = static_cast<const uint16_t *>(d_x);
    a.ldx = ldx;
    a.m = m;
    a.bias = static_cast<const uint16_t *>(d_bias);
    a.out = static_cast<uint16_t *>(d_y);
    a.status = d_status;
    const int sms = device_sms();
    if (sms < 1) return EP_ERR_CUDA;
    if (m <= kGemvTokens) return int4_gemv(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream));
    return launch_simple<kForward>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int ep_int4_linear_dx(const void *d_codes, const void *d_scales, int64_t n, int64_t k, int32_t group,
                                 int32_t dtype, const void *d_dy, int64_t m, int64_t lddy, void *d_dx,
                                 uint32_t *d_status, ep_stream_t stream) {
    using namespace ep;
    if (!weight_ok(n, k, group, dtype) || m < 0 || (m > 1 && lddy < n)) return EP_ERR_INVALID_ARG;
    if (m == 0) return EP_OK;
    if (!d_codes || !d_scales || !d_dy || !d_dx || misaligned(d_codes, 16) || misaligned(d_scales, 2) ||
        misaligned(d_dy, 2) || misaligned(d_dx, 2) || misaligned(d_status, 4))
        return EP_ERR_INVALID_ARG;
    Int4Args a = args_of(n, k, group, d_codes, d_scales);
    a.x = static_cast<const uint16_t *>(d_dy);
    a.ldx = lddy;
    a.m = m;
    a.out = static_cast<uint16_t *>(d_dx);
    return launch_simple<kInputGrad>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int ep_int4_scale_grad(const void *d_dy, int64_t lddy, const void *d_act, const float *d_act_scales,
                                  int64_t m, const void *d_codes, int64_t n, int64_t k, int32_t group, int32_t dtype,
                                  void *d_ds, uint32_t *d_status, ep_stream_t stream) {
    using namespace ep;
    if (!weight_ok(n, k, group, dtype) || m < 0 || (m > 1 && lddy < n)) return EP_ERR_INVALID_ARG;
    if (!d_codes || !d_ds || misaligned(d_codes, 16) || misaligned(d_ds, 2) || misaligned(d_status, 4))
        return EP_ERR_INVALID_ARG;
    if (m > 0 && (!d_dy || !d_act || !d_act_scales || misaligned(d_dy, 2) || misaligned(d_act, 16) ||
                  misaligned(d_act_scales, 4)))
        return EP_ERR_INVALID_ARG;
    Int4Args a = args_of(n, k, group, d_codes, nullptr);
    a.x = static_cast<const uint16_t *>(d_dy);
    a.ldx = lddy;
    a.m = m;
    a.act = static_cast<const int8_t *>(d_act);
    a.act_scales = d_act_scales;
    a.out = static_cast<uint16_t *>(d_ds);
    return launch_simple<kScaleGrad>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}
