// ep_int4_linear for few tokens (m <= kGemvTokens): every weight is read once from memory and multiplied
// for all tokens, so HBM bounds it (0.5 bytes and 2 m flops per weight).
#include <algorithm>

#include "int4_gemm.cuh"

namespace ep {
namespace {

// A warp takes 16 output features and a range of inputs in blocks of 128: lane (g = lane / 4, c = lane % 4)
// loads the 16 bytes of inputs 32 c .. 32 c + 31 of the block for features g and g + 8 (a quad reads 64
// contiguous bytes), turns pairs of codes into exact 16-bit integers (shift, mask-or with the bits of
// 128 or 1024, subtract) and feeds them to mma.m16n8k16 as A, with the tokens as B (8 per tile, absent
// ones 0).  The inputs that one mma contracts may be any 16 as long as A and B agree, so a lane's B
// fragments are contiguous inputs of its token, read as 16 bytes through L1.  Each group of inputs has
// its own accumulation, scaled in fp32 by s and added to the total: q and x are exact, only sums round.
// Groups of 64 (32) inputs: the quad first exchanges words so that each mma stays within a group
// (2 (4) shuffles per 16 bytes), after which lane c holds, of the block's group h, the inputs from
// lane_offset(h, c), 32 / (128 / group) of them.
// The tensor cores are the cheap way to the products (one instruction per 8 weights of a lane for up to
// 8 tokens); what bounds the kernel is the stream of weights.
template <uint32_t GPB>  // groups per block of 128 inputs
__device__ __forceinline__ uint32_t lane_offset(uint32_t h, uint32_t c) {
    if constexpr (GPB == 1) return 32 * c;
    if constexpr (GPB == 2) return 64 * h + 32 * (c & 1u) + 16 * (c >> 1);
    return 32 * h + 8 * c;
}

// the quad's words so that word GPB == 1: j, 2: 2 h + (0, 1), 4: h belongs to group h
template <uint32_t GPB>
__device__ __forceinline__ void exchange(uint32_t (&w)[4], uint32_t c) {
    if constexpr (GPB >= 2) {  // with the lane two away: it keeps the half of each chunk that c's bit 1 names
        const bool up = c & 2u;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[2], 2);
        const uint32_t b = __shfl_xor_sync(0xffffffffu, up ? w[1] : w[3], 2);
        w[0] = up ? a : w[0];
        w[1] = up ? b : w[1];
        w[2] = up ? w[2] : a;
        w[3] = up ? w[3] : b;
    }
    if constexpr (GPB == 4) {
        // now w[0], w[1]: words (2 b1, 2 b1 + 1) of chunk b0; w[2], w[3]: of chunk 2 + b0 (c = 2 b1 + b0)
        const bool up = c & 1u;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[1], 1);
        const uint32_t b = __shfl_xor_sync(0xffffffffu, up ? w[2] : w[3], 1);
        const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
        w[0] = up ? a : w0;  // chunk 0, word 2 b1 + b0 = c
        w[1] = up ? w1 : a;  // chunk 1
        w[2] = up ? b : w2;
        w[3] = up ? w3 : b;
    }
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (sizeof(typename Elem<T>::Pair) && Elem<T>::kMagic == 0x43004300u)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct GemvArgs {
    Int4Args a;
    uint32_t blocks;  // of 128 inputs
    uint32_t xvec;    // bytes that x may be read at once by: 16, 4 or 2
};

constexpr uint32_t kRowWarps = 4, kKWarps = 2;  // a CTA: 64 output features, its range of inputs in two halves

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <typename T, uint32_t GPB, uint32_t NT>
__global__ void __launch_bounds__(256, NT == 1 ? 3 : 2) int4_gemv_kernel(const __grid_constant__ GemvArgs p) {
    constexpr uint32_t kTok = 8 * NT, kPerGroup = 8 / GPB;  // mma steps per group
    __shared__ float part[kKWarps][64][kTok + 1];
    const Int4Args &a = p.a;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
    const uint32_t splits = gridDim.y, rank = blockIdx.y;  // a cluster: one CTA per split of the inputs
    const uint32_t row0 = blockIdx.x * 64 + (warp % kRowWarps) * 16, kw = warp / kRowWarps;
    const uint32_t slices = splits * kKWarps, slice = rank * kKWarps + kw;
    const uint32_t b0 = uint32_t(uint64_t(slice) * p.blocks / slices), b1 = uint32_t(uint64_t(slice + 1) * p.blocks / slices);
    // features beyond the last read the last one's codes; their sums are not written
    const uint32_t ra = min(row0 + g, a.n - 1), rb = min(row0 + g + 8, a.n - 1);
    const uint32_t *wa = a.codes + int64_t(ra) * a.words, *wb = a.codes + int64_t(rb) * a.words;
    const uint16_t *sa = a.scales + int64_t(ra) * a.groups, *sb = a.scales + int64_t(rb) * a.groups;
    const uint32_t m = uint32_t(a.m);

    float total[NT][4] = {};
    auto load = [&](uint32_t b, uint4 &u, uint4 &v, uint16_t (&s)[2 * GPB]) {
        const uint32_t w = 16 * b + 4 * c;
        u = v = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        if (w < a.words) {
            u = ldg_stream(wa + w);
            v = ldg_stream(wb + w);
        }
#pragma unroll
        for (uint32_t h = 0; h < GPB; ++h) {  // groups beyond the last: their codes are 0, any finite scale does
            const uint32_t gi = b * GPB + h;
            s[2 * h] = gi < a.groups ? __ldg(sa + gi) : uint16_t(0);
            s[2 * h + 1] = gi < a.groups ? __ldg(sb + gi) : uint16_t(0);
        }
    };
    auto compute = [&](uint32_t b, const uint4 &u, const uint4 &v, const uint16_t (&s)[2 * GPB]) {
        // this lane's B fragments: inputs lane_offset(h, c) .. of token g (and g + 8)
        uint32_t x[NT][16];
#pragma unroll
        for (uint32_t t = 0; t < NT; ++t) {
            const bool have = 8 * t + g < m;
            const uint16_t *row = a.x + int64_t(8 * t + g) * a.ldx;
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const uint32_t k = 128 * b + lane_offset<GPB>(q * GPB / 4, c) + 8 * (q % (4 / GPB));
                uint4 r = make_uint4(0u, 0u, 0u, 0u);
                if (have) {
                    if (p.xvec == 16) {
                        if (k < a.k) r = __ldg(reinterpret_cast<const uint4 *>(row + k));
                    } else if (p.xvec == 4 && k + 8 <= a.k) {
                        const uint32_t *r4 = reinterpret_cast<const uint32_t *>(row + k);
                        r = make_uint4(__ldg(r4), __ldg(r4 + 1), __ldg(r4 + 2), __ldg(r4 + 3));
                    } else if (k < a.k) {
                        uint32_t e[8];
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i) e[i] = k + i < a.k ? __ldg(row + k + i) : 0u;
                        r = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16));
                    }
                }
                x[t][4 * q] = r.x, x[t][4 * q + 1] = r.y, x[t][4 * q + 2] = r.z, x[t][4 * q + 3] = r.w;
            }
        }
        uint32_t wu[4] = {u.x, u.y, u.z, u.w}, wv[4] = {v.x, v.y, v.z, v.w};
        exchange<GPB>(wu, c);
        exchange<GPB>(wv, c);
#pragma unroll
        for (uint32_t h = 0; h < GPB; ++h) {
            float acc[NT][4] = {};
#pragma unroll
            for (uint32_t j = 0; j < kPerGroup; ++j) {
                const uint32_t step = h * kPerGroup + j, word = step / 2, i = 2 * (step & 1u);
                // pairs 2 i, 2 i + 1 of a word: A's k 2 c, 2 c + 1 and 2 c + 8, 2 c + 9
                const uint32_t f[4] = {code_pair<T>(wu[word], i), code_pair<T>(wv[word], i), code_pair<T>(wu[word], i + 1),
                                       code_pair<T>(wv[word], i + 1)};
#pragma unroll
                for (uint32_t t = 0; t < NT; ++t) mma16816<T>(acc[t], f, x[t][2 * step], x[t][2 * step + 1]);
            }
            const float fa = Elem<T>::f(s[2 * h]), fb = Elem<T>::f(s[2 * h + 1]);
#pragma unroll
            for (uint32_t t = 0; t < NT; ++t) {
                total[t][0] = fmaf(fa, acc[t][0], total[t][0]);
                total[t][1] = fmaf(fa, acc[t][1], total[t][1]);
                total[t][2] = fmaf(fb, acc[t][2], total[t][2]);
                total[t][3] = fmaf(fb, acc[t][3], total[t][3]);
            }
        }
    };

    // two blocks a turn, the next turn's loads in flight while this one is multiplied
    uint4 u[2], v[2];
    uint16_t s[2][2 * GPB];
    for (uint32_t i = 0; i < 2; ++i)
        if (b0 + i < b1) load(b0 + i, u[i], v[i], s[i]);
    for (uint32_t b = b0; b < b1; b += 2) {
        uint4 un[2], vn[2];
        uint16_t sn[2][2 * GPB];
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i)
            if (b + 2 + i < b1) load(b + 2 + i, un[i], vn[i], sn[i]);
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i)
            if (b + i < b1) compute(b + i, u[i], v[i], s[i]);
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            u[i] = un[i], v[i] = vn[i];
#pragma unroll
            for (uint32_t h = 0; h < 2 * GPB; ++h) s[i][h] = sn[i][h];
        }
    }

    // the CTA's sums: feature rows, tokens 2 c, 2 c + 1 (+ 8 t)
    const uint32_t r = (warp % kRowWarps) * 16 + g;
#pragma unroll
    for (uint32_t t = 0; t < NT; ++t) {
        part[kw][r][8 * t + 2 * c] = total[t][0];
        part[kw][r][8 * t + 2 * c + 1] = total[t][1];
        part[kw][r + 8][8 * t + 2 * c] = total[t][2];
        part[kw][r + 8][8 * t + 2 * c + 1] = total[t][3];
    }
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    // this CTA's share of the 64 features: the splits' sums in order, the bias, one rounding
    const uint32_t lo = rank * 64 / splits, hi = (rank + 1) * 64 / splits, rows = hi - lo;
    for (uint32_t e = threadIdx.x; e < rows * m; e += 256) {
        const uint32_t t = e / rows, f = lo + e % rows, o = blockIdx.x * 64 + f;
        if (o >= a.n) continue;
        float y = 0.0f;
        if (splits > 1) {
            for (uint32_t q = 0; q < splits; ++q)
#pragma unroll
                for (uint32_t w = 0; w < kKWarps; ++w) y += ld_cluster(&part[w][f][t], q);
        } else {
#pragma unroll
            for (uint32_t w = 0; w < kKWarps; ++w) y += part[w][f][t];
        }
        if (a.bias) y += Elem<T>::f(__ldg(a.bias + o));
        a.out[int64_t(t) * a.n + o] = Elem<T>::bits(y);
    }
    if (splits > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

template <typename T, uint32_t NT>
int launch_gemv(const GemvArgs &p, dim3 grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = grid.y;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const auto kern = p.a.group == 128 ? int4_gemv_kernel<T, 1, NT>
                      : p.a.group == 64 ? int4_gemv_kernel<T, 2, NT>
                                        : int4_gemv_kernel<T, 4, NT>;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

}  // namespace

int int4_gemv(const Int4Args &a, int32_t dtype, int sms, cudaStream_t s) {
    GemvArgs p;
    p.a = a;
    p.blocks = (a.k + 127) / 128;
    const bool one = a.m == 1;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x);
    p.xvec = at % 16 == 0 && (one || a.ldx % 8 == 0) && a.k % 8 == 0 ? 16 : at % 4 == 0 && (one || a.ldx % 2 == 0) ? 4 : 2;
    // splits of the inputs over a cluster: as many as keep every CTA resident at once (one wave), each
    // warp with at least one block
    const uint32_t nt = a.m <= 8 ? 1 : 2, tiles = (a.n + 63) / 64, slots = uint32_t(sms) * (nt == 1 ? 3 : 2);
    uint32_t splits = std::min(8u, std::max(1u, slots / tiles));
    splits = std::max(1u, std::min(splits, p.blocks / kKWarps));
    const dim3 grid(tiles, splits);
    if (dtype == EP_BF16)
        return nt == 1 ? launch_gemv<__nv_bfloat16, 1>(p, grid, s) : launch_gemv<__nv_bfloat16, 2>(p, grid, s);
    return nt == 1 ? launch_gemv<__half, 1>(p, grid, s) : launch_gemv<__half, 2>(p, grid, s);
}

}  // namespace ep
