// ep_int4_linear for few tokens (m <= kGemvTokens): every weight is read once from memory and multiplied
// for all tokens (0.5 bytes and 2 m flops per weight: HBM's time is the floor).
// Measured on a B200: 8192 x 28672, groups of 128, one token 29.8 us, 8 tokens 33.8, 16 tokens 47.8; groups
// of 64 and 32, one token 36.2 and 42.2.  The stream alone takes 18.5 us at the copy rate and 20.8 us by these
// loads, 25.9 without x's.  No unit is busy enough to bound it (one token: L1 65 %, issue slots 54 %, ALU pipe 53 %, DRAM
// 45 %): 16 warps on an SM at 122 registers leave it waiting for loads (3.1 cycles an instruction), among which the
// codes' expansion (9 instructions for 8 weights) and x's reads through L1 come one after the other.  1024 x 1024:
// 2.4 us, a launch.
#include <algorithm>

#include "int4_gemm.cuh"

namespace ep {
namespace {

// A warp takes RG tiles of 16 output features and a range of inputs in blocks of 128: lane (g = lane / 4,
// c = lane % 4) loads the 16 bytes of inputs 32 c .. 32 c + 31 of the block for features g and g + 8 of a
// tile (a quad reads 64 contiguous bytes), turns pairs of codes into exact 16-bit numbers (code_pairs) and
// feeds them to mma.m16n8k16 as A, with the tokens as B (8 per tile, absent ones the last one's).  The inputs
// that one mma contracts may be any 16 as long as A and B agree, so a lane's B fragments are contiguous inputs
// of its token, read as 16 bytes through L1.  Each group of inputs has its own accumulation, scaled in fp32 by s
// and added to the total: q and x are exact, only sums round.
// Groups of 64 (32) inputs: the quad first exchanges words so that each mma stays within a group
// (2 (4) shuffles per 16 bytes), after which lane c holds, of the block's half (quarter) h, the inputs from
// lane_offset(h, c), 16 (8) of them.
// The tensor cores are the cheap way to the products: one instruction per 8 weights of a lane for up to 8 tokens.
template <uint32_t X>  // parts of the block of 128 inputs
__device__ __forceinline__ uint32_t lane_offset(uint32_t h, uint32_t c) {
    if constexpr (X == 1) return 32 * c;
    if constexpr (X == 2) return 64 * h + 32 * (c & 1u) + 16 * (c >> 1);
    return 32 * h + 8 * c;
}

// the quad's words so that word 2 h, 2 h + 1 (X == 2) or h (X == 4) belongs to part h
template <uint32_t X>
__device__ __forceinline__ void exchange(uint32_t (&w)[4], uint32_t c) {
    if constexpr (X >= 2) {  // with the lane two away: it keeps the half of each chunk that c's bit 1 names
        const bool up = c & 2u;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[2], 2);
        const uint32_t b = __shfl_xor_sync(0xffffffffu, up ? w[1] : w[3], 2);
        w[0] = up ? a : w[0];
        w[1] = up ? b : w[1];
        w[2] = up ? w[2] : a;
        w[3] = up ? w[3] : b;
    }
    if constexpr (X == 4) {
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

// d = a b (+ d unless `first`)
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
    const float c0 = first ? 0.0f : d[0], c1 = first ? 0.0f : d[1], c2 = first ? 0.0f : d[2], c3 = first ? 0.0f : d[3];
    if constexpr (Elem<T>::kMagic == 0x43004300u)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
            "%12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
            "%12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// A sum `y` that came out infinite or NaN, by a warp.  It stands unless a scale of its feature is infinite (times a
// group's sum, it hides an input whose product is NaN, or is of the other sign) or its token has finite activations
// from 2^117 on (BF16: sums of x q may pass fp32's range where the scale brings them back).  Then it is taken again
// input by input as the formula has it, x[t, k] (s[o, k / group] q[o, k]), each lane every 32nd input, added in a fixed
// order: x as 2^-64 x and q as q / 16, so that nothing passes fp32's range whose result does not (activations below 2^-62
// are lost beside those).  `last` and `huge`, kept by the caller: the token looked at last, and what was found.
// 8192 x 28672, an infinity or NaN as the last input of each token: 25 us more for one, 0.34 ms for 16.
template <typename T>
__device__ float formula_sum(const Int4Args &a, uint32_t o, uint32_t t, float y, uint32_t &last, bool &huge) {
    constexpr uint32_t kAhead = 8;  // loads in flight
    const uint32_t lane = threadIdx.x & 31u, group_bits = 31 - __clz(a.group);
    const uint32_t *codes = a.codes + int64_t(o) * a.words;
    const uint16_t *scales = a.scales + int64_t(o) * a.groups, *x = a.x + int64_t(t) * a.ldx;
    if (Elem<T>::kInf == 0x7f80u && t != last) {
        bool nan = false;  // (then y stands)
        last = t;
        huge = false;
        for (uint32_t k0 = 0; k0 < a.k && !nan; k0 += 32 * kAhead) {
            bool mine = false;
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                const uint32_t k = k0 + 32 * i + lane, u = k < a.k ? __ldg(x + k) & 0x7fffu : 0u;
                mine |= u >= 0x7a00u && u < 0x7f80u;
                nan |= u > 0x7f80u;
            }
            nan = __any_sync(0xffffffffu, nan);
            huge |= __any_sync(0xffffffffu, mine);
        }
        if (nan) huge = false;
    }
    bool infinite = false;
    for (uint32_t g = lane; g < a.groups; g += 32) infinite |= (__ldg(scales + g) & 0x7fffu) == Elem<T>::kInf;
    if (!__any_sync(0xffffffffu, infinite) && !huge) return y;
    float sum = 0.0f;
    for (uint32_t k0 = 0; k0 < a.k; k0 += 32 * kAhead) {
        uint32_t word[kAhead];
        uint16_t xs[kAhead], ss[kAhead];
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) {
            const uint32_t k = min(k0 + 32 * i + lane, a.k - 1);
            word[i] = __ldg(codes + k / 8), xs[i] = __ldg(x + k), ss[i] = __ldg(scales + (k >> group_bits));
        }
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) {
            const uint32_t k = k0 + 32 * i + lane, e = k & 7u, code = (word[i] >> (4 * (e / 2) + 16 * (e & 1u))) & 15u;
            const float q = (__uint_as_float(0x4b000000u | code) - 8388616.0f) * 0.0625f;  // (2^23 + code) - (2^23 + 8)
            const float w = Elem<T>::f(ss[i]) * q, v = Elem<T>::f(xs[i]);
            // (a small v times an infinite w is infinite)
            if (k < a.k) sum = fmaf(fabsf(w) == __uint_as_float(0x7f800000u) ? v : v * 0x1p-64f, w, sum);
        }
        if (__any_sync(0xffffffffu, sum != sum)) return __uint_as_float(0x7fffffffu);  // NaN stays
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum * 0x1p68f;
}

struct GemvArgs {
    Int4Args a;
    uint32_t blocks;     // of 128 inputs
    uint32_t xvec;       // bytes that x may be read at once by: 16, 4 or 2
    uint32_t row_warps;  // 1, 2, 4 or 8 warps take different features, the 8 / row_warps of a feature a range of inputs each
    uint32_t rows;       // features of a warp, at most 16 RG
};

constexpr uint32_t kWarps = 8;
constexpr uint32_t ctas_on_sm(uint32_t rg) { return rg == 4 ? 1 : 2; }

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A block's scales of one feature: as one load where rows of scales allow it (SVEC), one for each otherwise
template <uint32_t GPB, bool SVEC>
struct Scales {
    uint16_t s[GPB];
    __device__ __forceinline__ void load(const uint16_t *p) {
#pragma unroll
        for (uint32_t h = 0; h < GPB; ++h) s[h] = __ldg(p + h);
    }
    __device__ __forceinline__ uint16_t get(uint32_t h) const { return s[h]; }
    __device__ __forceinline__ void set(uint32_t h, uint16_t v) { s[h] = v; }
};
template <uint32_t GPB>
struct Scales<GPB, true> {
    uint32_t s[GPB / 2];
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (GPB == 2) {
            s[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
            s[0] = v.x, s[1] = v.y;
        }
    }
    __device__ __forceinline__ uint16_t get(uint32_t h) const { return uint16_t(s[h / 2] >> (16 * (h & 1u))); }
    __device__ __forceinline__ void set(uint32_t h, uint16_t v) {
        s[h / 2] = h & 1u ? (s[h / 2] & 0xffffu) | uint32_t(v) << 16 : (s[h / 2] & 0xffff0000u) | v;
    }
};

// the words and scales of one block of 128 inputs for a lane's 2 RG features
template <uint32_t GPB, uint32_t RG, bool SVEC>
struct Block {
    uint4 w[2 * RG];
    Scales<GPB, SVEC> s[2 * RG];
};

// RG: 16-feature tiles of a warp; NT: 8-token tiles; VEC: x is read 16 bytes at a time; SVEC: Scales
template <typename T, uint32_t GPB, uint32_t NT, uint32_t RG, bool VEC, bool SVEC>
__global__ void __launch_bounds__(32 * kWarps, ctas_on_sm(RG)) int4_gemv_kernel(const __grid_constant__ GemvArgs p) {
    constexpr uint32_t kTok = 8 * NT, kPerGroup = 8 / GPB, kDeep = RG == 1 && NT == 1 ? 4 : 2;  // mma steps per group, blocks in flight
    // how far the quad's words are exchanged: for the groups, and for groups of 128 where it pays that the quad's
    // reads of x then lie in one line of 128 bytes (16 tokens: 4096 x 11008 13.6 us against 17.4, but 8192 x 28672,
    // with 64 features a warp, 51.4 against 48.8; 1 and 8 tokens there: 35.5 and 36.2 against 29.7 and 33.7)
    constexpr uint32_t X = GPB == 1 && NT == 2 && RG == 1 ? 2 : GPB;
    __shared__ float part[kWarps][16 * RG][kTok + 1];
    const Int4Args &a = p.a;
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
    const uint32_t slices = kWarps / p.row_warps, rw = warp / slices, slice = warp % slices;
    const uint32_t row0 = (blockIdx.x * p.row_warps + rw) * p.rows;
    const uint32_t b0 = slice * p.blocks / slices, b1 = (slice + 1) * p.blocks / slices;
    const uint32_t m = uint32_t(a.m), whole = VEC ? min(b1, a.k / 128) : b0;  // blocks b0 .. whole - 1 lie within k
    // a lane without a feature loads nothing and multiplies zeros; tokens beyond the last read the last
    // one's x: sums that are not written
    const uint32_t *wp[2 * RG];
    const uint16_t *sp[2 * RG], *xp[NT];
    bool have[2 * RG];
#pragma unroll
    for (uint32_t i = 0; i < 2 * RG; ++i) {
        const uint32_t r = row0 + 8 * i + g;
        have[i] = 8 * i + g < p.rows && r < a.n;
        wp[i] = a.codes + int64_t(have[i] ? r : 0) * a.words + 16 * b0 + 4 * c;
        sp[i] = a.scales + int64_t(have[i] ? r : 0) * a.groups + b0 * GPB;
    }
#pragma unroll
    for (uint32_t t = 0; t < NT; ++t) xp[t] = a.x + int64_t(min(8 * t + g, m - 1)) * a.ldx + 128 * b0;

    float total[RG][NT][4] = {};
    auto load = [&](uint32_t ahead, Block<GPB, RG, SVEC> &k) {  // a whole block, `ahead` of the current one
#pragma unroll
        for (uint32_t i = 0; i < 2 * RG; ++i) {
            if (have[i]) {
                k.w[i] = ldg_stream(wp[i] + 16 * ahead);
                k.s[i].load(sp[i] + ahead * GPB);
            }
        }
    };
    auto multiply = [&](Block<GPB, RG, SVEC> &k, const uint32_t (&x)[NT][16]) {
        uint32_t w[2 * RG][4];
#pragma unroll
        for (uint32_t i = 0; i < 2 * RG; ++i) {
            w[i][0] = k.w[i].x, w[i][1] = k.w[i].y, w[i][2] = k.w[i].z, w[i][3] = k.w[i].w;
            exchange<X>(w[i], c);
        }
#pragma unroll
        for (uint32_t h = 0; h < GPB; ++h) {
            float acc[RG][NT][4];
#pragma unroll
            for (uint32_t j = 0; j < kPerGroup; j += 2) {
                const uint32_t step = h * kPerGroup + j, word = step / 2;
#pragma unroll
                for (uint32_t r = 0; r < RG; ++r) {
                    // pairs 2 i, 2 i + 1 of a word: A's k 2 c, 2 c + 1 and 2 c + 8, 2 c + 9
                    uint32_t u[4], v[4];
                    code_pairs<T>(w[2 * r][word], u);
                    code_pairs<T>(w[2 * r + 1][word], v);
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        const uint32_t f[4] = {u[2 * i], v[2 * i], u[2 * i + 1], v[2 * i + 1]};
#pragma unroll
                        for (uint32_t t = 0; t < NT; ++t)
                            mma16816<T>(acc[r][t], f, x[t][2 * (step + i)], x[t][2 * (step + i) + 1], j + i == 0);
                    }
                }
            }
#pragma unroll
            for (uint32_t r = 0; r < RG; ++r) {
                const float fa = Elem<T>::f(k.s[2 * r].get(h)), fb = Elem<T>::f(k.s[2 * r + 1].get(h));
#pragma unroll
                for (uint32_t t = 0; t < NT; ++t) {
                    total[r][t][0] = fmaf(fa, acc[r][t][0], total[r][t][0]);
                    total[r][t][1] = fmaf(fa, acc[r][t][1], total[r][t][1]);
                    total[r][t][2] = fmaf(fb, acc[r][t][2], total[r][t][2]);
                    total[r][t][3] = fmaf(fb, acc[r][t][3], total[r][t][3]);
                }
            }
        }
    };
    // this lane's B fragments of a block: inputs lane_offset(h, c) .. of token g (and g + 8)
    auto compute = [&](uint32_t ahead, Block<GPB, RG, SVEC> &k) {
        uint32_t x[NT][16];
#pragma unroll
        for (uint32_t t = 0; t < NT; ++t)
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const uint4 r = __ldg(reinterpret_cast<const uint4 *>(xp[t] + lane_offset<X>(0, c) + 128 * ahead +
                                                                      lane_offset<X>(q * X / 4, 0) + 8 * (q % (4 / X))));
                x[t][4 * q] = r.x, x[t][4 * q + 1] = r.y, x[t][4 * q + 2] = r.z, x[t][4 * q + 3] = r.w;
            }
        multiply(k, x);
    };
    const Block<GPB, RG, SVEC> zero = [] {
        Block<GPB, RG, SVEC> z;
        for (uint32_t i = 0; i < 2 * RG; ++i) {
            z.w[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
            for (uint32_t h = 0; h < GPB; ++h) z.s[i].set(h, 0);
        }
        return z;
    }();
    // kDeep blocks' loads in flight, each turn multiplies the oldest and loads the next
    if (b0 < whole) {
        Block<GPB, RG, SVEC> k[kDeep];
#pragma unroll
        for (uint32_t i = 0; i < kDeep; ++i) {
            k[i] = zero;
            if (b0 + i < whole) load(i, k[i]);
        }
        for (uint32_t b = b0; b < whole; b += kDeep) {
#pragma unroll
            for (uint32_t i = 0; i < kDeep; ++i) {
                if (b + i >= whole) break;
                compute(i, k[i]);
                if (b + i + kDeep < whole) load(i + kDeep, k[i]);
            }
#pragma unroll
            for (uint32_t i = 0; i < 2 * RG; ++i) wp[i] += 16 * kDeep, sp[i] += GPB * kDeep;
#pragma unroll
            for (uint32_t t = 0; t < NT; ++t) xp[t] += 128 * kDeep;
        }
    }
    // the block that k ends in, and every block of an x that is not 16-byte aligned: each word, group and
    // input checked (beyond k: q = 0, x = 0)
    for (uint32_t b = max(b0, whole); b < b1; ++b) {
        Block<GPB, RG, SVEC> k = zero;
#pragma unroll
        for (uint32_t i = 0; i < 2 * RG; ++i) {
            const int64_t r = row0 + 8 * i + g;
            if (have[i] && 16 * b + 4 * c < a.words) k.w[i] = ldg_stream(a.codes + r * a.words + 16 * b + 4 * c);
#pragma unroll
            for (uint32_t h = 0; h < GPB; ++h)
                if (have[i] && b * GPB + h < a.groups) k.s[i].set(h, __ldg(a.scales + r * a.groups + b * GPB + h));
        }
        uint32_t x[NT][16];
#pragma unroll
        for (uint32_t t = 0; t < NT; ++t) {
            const uint16_t *row = a.x + int64_t(min(8 * t + g, m - 1)) * a.ldx;
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const uint32_t at = 128 * b + lane_offset<X>(q * X / 4, c) + 8 * (q % (4 / X));
                const uint16_t *src = row + at;
                uint32_t *dst = &x[t][4 * q];
                if (p.xvec >= 4 && at + 8 <= a.k) {
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) dst[i] = __ldg(reinterpret_cast<const uint32_t *>(src) + i);
                } else {
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        dst[i] = (at + 2 * i < a.k ? __ldg(src + 2 * i) : 0u) |
                                 (at + 2 * i + 1 < a.k ? uint32_t(__ldg(src + 2 * i + 1)) << 16 : 0u);
                }
            }
        }
        multiply(k, x);
    }

    // the warps' sums: features, tokens 2 c, 2 c + 1 (+ 8 t)
#pragma unroll
    for (uint32_t i = 0; i < RG; ++i)
#pragma unroll
        for (uint32_t t = 0; t < NT; ++t) {
            part[warp][16 * i + g][8 * t + 2 * c] = total[i][t][0];
            part[warp][16 * i + g][8 * t + 2 * c + 1] = total[i][t][1];
            part[warp][16 * i + g + 8][8 * t + 2 * c] = total[i][t][2];
            part[warp][16 * i + g + 8][8 * t + 2 * c + 1] = total[i][t][3];
        }
    __syncthreads();
    // each feature's slices in order, the bias, one rounding
    const uint32_t rows = p.row_warps * p.rows;
    const auto joined = [&](uint32_t t, uint32_t f) {
        float y = 0.0f;
        for (uint32_t q = 0; q < slices; ++q) y += part[f / p.rows * slices + q][f % p.rows][t];
        return y * Codes<T>::kUnit;
    };
    const auto finite = [](float y) { return fabsf(y) < __uint_as_float(0x7f800000u); };
    const auto write = [&](uint32_t t, uint32_t o, float y) {
        if (a.bias) y += Elem<T>::f(__ldg(a.bias + o));
        a.out[int64_t(t) * a.n + o] = Elem<T>::bits(y);
    };
    bool bad = false;
    for (uint32_t e = threadIdx.x; e < rows * m; e += 32 * kWarps) {
        const uint32_t t = e / rows, f = e % rows, o = blockIdx.x * rows + f;
        if (o >= a.n) continue;
        const float y = joined(t, f);
        if (finite(y)) write(t, o, y);
        else bad = true;
    }
    // the warp's others, one after the other
    if (!__any_sync(0xffffffffu, bad)) return;
    uint32_t last = ~0u;
    bool huge = false;
#pragma unroll 1
    for (uint32_t e0 = 32 * warp; e0 < rows * m; e0 += 32 * kWarps)
#pragma unroll 1
        for (uint32_t e = e0; e < min(e0 + 32, rows * m); ++e) {
            const uint32_t t = e / rows, f = e % rows, o = blockIdx.x * rows + f;
            float y = joined(t, f);
            if (o >= a.n || finite(y)) continue;
            y = formula_sum<T>(a, o, t, y, last, huge);
            if (lane == 0) write(t, o, y);
        }
}

template <typename T, uint32_t GPB, uint32_t NT, uint32_t RG>
int launch_gemv(const GemvArgs &p, unsigned grid, cudaStream_t s) {
    // (one scale a block is one load either way; without whole blocks none is made)
    const bool svec = GPB > 1 && p.a.groups % GPB == 0 && (reinterpret_cast<uintptr_t>(p.a.scales) & (2 * GPB - 1)) == 0;
    const auto kern = p.xvec != 16 ? int4_gemv_kernel<T, GPB, NT, RG, false, false>
                      : svec       ? int4_gemv_kernel<T, GPB, NT, RG, true, (GPB > 1)>
                                   : int4_gemv_kernel<T, GPB, NT, RG, true, false>;
    kern<<<grid, 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
template <typename T, uint32_t NT, uint32_t RG>
int launch_gemv_group(const GemvArgs &p, unsigned grid, cudaStream_t s) {
    return p.a.group == 128  ? launch_gemv<T, 1, NT, RG>(p, grid, s)
           : p.a.group == 64 ? launch_gemv<T, 2, NT, RG>(p, grid, s)
                             : launch_gemv<T, 4, NT, RG>(p, grid, s);
}
template <typename T>
int launch_gemv_for(const GemvArgs &p, uint32_t nt, uint32_t rg, unsigned grid, cudaStream_t s) {
    if (nt == 1) return rg == 1 ? launch_gemv_group<T, 1, 1>(p, grid, s) : launch_gemv_group<T, 1, 2>(p, grid, s);
    return rg == 1 ? launch_gemv_group<T, 2, 1>(p, grid, s) : launch_gemv_group<T, 2, 4>(p, grid, s);
}

}  // namespace

int int4_gemv(const Int4Args &a, int32_t dtype, int sms, cudaStream_t s) {
    GemvArgs p;
    p.a = a;
    p.blocks = (a.k + 127) / 128;
    const bool one = a.m == 1;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x);
    p.xvec = at % 16 == 0 && (one || a.ldx % 8 == 0) ? 16 : at % 4 == 0 && (one || a.ldx % 2 == 0) ? 4 : 2;
    // Every CTA resident at once with an equal share of the features, in equal waves where a share would be
    // more than the CTA's warps hold; few features leave more warps to share the inputs.  A warp with more
    // features reads x less often: 16 where a share holds no more, otherwise 32 (8192 x 28672, one token: 29.7 us;
    // 16: 33.9; 64: 39.9), or 64 and one CTA on an SM for two token tiles, where x would fill the L1's bandwidth
    // (16 tokens: 48.6 us; 32: 58.5)
    const uint32_t nt = a.m <= 8 ? 1 : 2;
    uint32_t rg = 1, share;
    for (;;) {
        const uint32_t slots = uint32_t(sms) * ctas_on_sm(rg), most = 16 * rg * kWarps;
        const uint32_t waves = (a.n + slots * most - 1) / (slots * most);
        share = std::max((a.n + slots * waves - 1) / (slots * waves), 16u);
        if (rg > 1 || share == 16) break;
        rg = nt == 1 ? 2 : 4;
    }
    p.row_warps = 1;
    while (p.row_warps * 16 * rg < share) p.row_warps *= 2;
    p.rows = (share + p.row_warps - 1) / p.row_warps;
    const unsigned grid = (a.n + p.row_warps * p.rows - 1) / (p.row_warps * p.rows);
    return dtype == EP_BF16 ? launch_gemv_for<__nv_bfloat16>(p, nt, rg, grid, s) : launch_gemv_for<__half>(p, nt, rg, grid, s);
}

}  // namespace ep
