// Products with a 4-bit group-scaled weight: the linear layer's forward (ep_int4_linear), its input
// gradient (ep_int4_linear_dx) and the gradient of the group scales from an 8-bit activation
// checkpoint (ep_int4_scale_grad), as tcgen05 GEMMs whose quantized operand is expanded on the way
// from memory to the tensor cores.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "int4_gemm.cuh"

namespace ep {
namespace {

enum Product { kForward, kInputGrad, kScaleGrad };

// Tiles of D = a sum over a contraction in steps of 64 (or 128, see the launch):
//   forward         D[o, t]: 128 output features x bn tokens, contraction over the inputs k
//   input gradient  D[k, t]: 128 inputs x bn tokens, contraction over the output features o
//   scale gradient  D[o, k]: 128 output features x 128 inputs, contraction over the tokens t
// One CTA per SM walks over tiles.  In the PAIR form two CTAs of a cluster share a tile twice as wide
// (cta_group::2): each expands 128 rows of the quantized operand and copies half of the dense one (forward and
// input gradient: its 128 features against all bn tokens; scale gradient: its 128 output features
// against all 256 inputs), so that an SM's shared memory carries 32 KB a step instead of 48: its
// bandwidth, taken by the copies in, the expanded stores and the matrix unit's reads, is what bounds the
// single form (2048 x 8192 x 8192 BF16, forward, input gradient and scale gradient: single 211, 232 and 339 us,
// paired 184, 189 and 204 us, 1494 to 1351 TFLOP/s of a floor of 169 us; the tensor pipe is then 90 % (scale
// gradient 75 %) busy, the issue slots 50 to 63 % with the expansion, and the card near its power limit).
// 17 to 64 tokens: 8192 x 28672 takes 57 to 65 us where the codes' stream takes 18.5: the expansion's and
// its handshakes' instructions (in steps of 64, 320 on each scheduler) fill 73 % of the issue slots of the
// SMs in use; six groups of expansion warps instead of four, more stages and more raw slots changed nothing.
// Roles: warps 0..15 expand the quantized operand (weight codes, or checkpoint codes in the scale gradient),
// warps 16..19 turn finished accumulators into output, warp 20 issues the matrix instructions (PAIR: the
// first CTA's, for both), warp 21 copies the quantized operand's bytes, warp 22 the dense operand (x or
// dy) by TMA, or warps 22..25 through registers where it is not 16-byte aligned.
// Rings in shared memory, running on over the tiles:
//   raw    the quantized operand's bytes, by TMA, slots of four 64s: steps of as many groups of four expansion
//          warps, or of half as many (W = 2; passing a slot costs a group 400 cycles, a seventh of its work on a step)
//   stage  one step's operands (W 64s of the contraction): 16 KB expanded (16-bit), and the dense tile (up to 256 or, scale gradient,
//          twice 64 rows of 128 bytes), both rows of 64 elements with the 128-byte swizzle
// The expanded operand's rows follow the stored codes (64 consecutive inputs of one output feature or
// token), so the forward's W is K-major (rows o, 64 k), and the input gradient's W^T and the scale
// gradient's x are MN-major (rows o or t, twice 64 k); dy is MN-major in the scale gradient (rows t, twice
// 64 o).  Two accumulators in tensor memory: one tile's is read out while the next one's is built.
// Few tiles: the contraction is split over a cluster's CTAs, whose accumulators (scale gradient: group
// sums) are joined through distributed shared memory, in rank order; over no more CTAs than leave room for all
// clusters at once (32 tokens, 2048 x 8192, 16 tiles: split over 6 13.0 us, over 8, in two waves, 21.5).
constexpr uint32_t kGroups = 4, kExpandWarps = 4 * kGroups, kOutWarp0 = kExpandWarps, kOutWarps = 4;
constexpr uint32_t kMmaWarp = kOutWarp0 + kOutWarps, kRawWarp = kMmaWarp + 1, kDenseWarp0 = kRawWarp + 1, kLoadWarps = 4;
constexpr uint32_t kQuantBytes = 16384, kBarBytes = 512, kMaxStages = 8, kMaxRaws = 8;
constexpr uint32_t kPairMask = 3;  // both CTAs of a pair

struct MmaArgs {
    CUtensorMap dense, raw;
    Int4Args a;
    uint32_t bn;        // columns of an accumulator: tokens, or inputs (scale gradient)
    uint32_t tiles, tiles_b;  // of D, and of its second index
    uint32_t steps;     // of 64 W along the contraction
    uint32_t slots;     // raw slots along the contraction, of 64 kSlotSteps
    uint32_t stages, raws, dense_bytes;
    uint32_t idesc, tmem_cols;  // tensor memory: two accumulators
    uint32_t dense_align;  // 4 or 2 bytes, where the dense operand is not copied by TMA
};

constexpr uint32_t kSlotSteps = 4;  // 64s of the contraction in a raw slot: 4 / W steps, each of another group of expansion warps
template <int P>
struct Shape {
    static constexpr uint32_t kRawBytes = P == kScaleGrad ? 32768 : 16384;
};

// shared-memory matrix descriptor, 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 bytes apart.
// K-major: `lead` is not used.  MN-major: each row holds 64 consecutive M (N) of one k, and `lead` is the
// distance to the next 64.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lead) {
    return uint64_t((addr >> 4) & 0x3fffu) | (uint64_t((lead >> 4) & 0x3fffu) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}
// an arrival when the matrix instructions before it are done, on the barrier of this CTA, or of both
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(uint16_t(kPairMask))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}
// the address of a place of this CTA's shared memory in the pair's first CTA
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(addr));
    return there;
}
// an arrival on the barrier of the CTA whose warp 20 issues the matrix instructions
template <bool PAIR>
__device__ __forceinline__ void arrive_issuer(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_first(bar)) : "memory");
    else
        mbar_arrive(bar);
}
// loads that stay where they are written (the compiler moves others down to their use, a whole step later)
__device__ __forceinline__ uint32_t ldg_now32(const void *p) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ldg_now16(const void *p) {
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// columns `from` (not a multiple of 32) to the next multiple of 32 of 128 swizzled rows of 64 elements, by a warp
__device__ __forceinline__ void zero_behind(uint32_t tile, uint32_t from, uint32_t lane) {
    const uint32_t none[4] = {};
#pragma unroll 1
    for (uint32_t r = lane; r < 128; r += 32)
#pragma unroll 1
        for (uint32_t i = from; i & 31u;) {
            const uint32_t at = tile + 128 * r + 16 * ((i >> 3) ^ (r & 7u)) + 2 * (i & 7u);
            if (i & 7u) {
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(uint16_t(0)) : "memory");
                ++i;
            } else {
                sts128(at, none);
                i += 8;
            }
        }
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 16-bit pairs times a scale, each product rounded once: the matrix unit's operands have 16 bits, and a scale that
// changes along the contraction (over its groups, or over every o of the input gradient) cannot wait for the
// accumulator.  Against 64 bits the forward's and the input gradient's relative error is 0.0021 in BF16 and 0.00028 in
// FP16, of which rounding the result alone makes 0.0017 and 0.00021; a second operand for the rounding's remainder would
// double the matrix instructions, which bound the large products.
template <typename T>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    using Pair = typename Elem<T>::Pair;
    const Pair d = __hmul2(*reinterpret_cast<const Pair *>(&a), *reinterpret_cast<const Pair *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// Checkpoint codes: bytes 2 i, 2 i + 1 of a word as exact pairs.  BF16: the low seven bits under the
// exponent of 128, minus 128 or (bit 7 is the exponent's last place) 256: c.  FP16: c + 128 under 1024,
// times 1/64 minus 18: c / 64.
// The scale comes as two 16-bit parts of a (FP16: of 64 a, so that small scales keep their digits), hi + lo;
// c hi + (c lo) by one fused multiply-add rounds a c once but for 2^-9 (2^-12) of c lo.
template <typename T>
struct Act;
template <>
struct Act<__nv_bfloat16> {
    static constexpr float kScale = 1.0f;
    __device__ static uint32_t pair(uint32_t w, uint32_t i) {
        const uint32_t p = __byte_perm(w, 0x43434343u, i ? 0x4342u : 0x4140u), mag = p & 0xff7fff7fu, off = p & 0xff80ff80u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&mag), *reinterpret_cast<const __nv_bfloat162 *>(&off));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
};
template <>
struct Act<__half> {
    static constexpr float kScale = 64.0f;
    __device__ static uint32_t pair(uint32_t w, uint32_t i) {
        const uint32_t p = __byte_perm(w, 0x64646464u, i ? 0x4342u : 0x4140u) ^ 0x00800080u;
        return Codes<__half>::fma2(p, 0x24002400u, 0xcc80cc80u);  // (1024 + 128 + c) / 64 - 18
    }
};

// A walk over the steps of a CTA's tiles, `n` steps a tile: tile `tile`, its step `i`
struct Walk {
    uint32_t tile, i;
    __device__ __forceinline__ void advance(uint32_t by, uint32_t n, uint32_t walkers) {
        for (i += by; i >= n; i -= n) tile += walkers;
    }
};
// A place in a ring of `size` buffers and the parity of its turn
struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void advance(uint32_t by, uint32_t size) {
        for (at += by; at >= size; at -= size) phase ^= 1u;
    }
};

// W: 64s of the contraction in a step
template <typename T, int P, bool TMA, bool PAIR, uint32_t W>
__global__ void __launch_bounds__((kDenseWarp0 + (TMA ? 1 : kLoadWarps)) * 32, 1)
    int4_mma_kernel(const __grid_constant__ MmaArgs p) {
    static_assert(TMA || !PAIR, "a pair copies its dense operand by TMA");
    static_assert(W == 1 || (W == 2 && TMA && !PAIR && P == kForward), "wide steps");
    constexpr uint32_t kSpan = 64 * W, kSteps = kSlotSteps / W;  // a step's contraction, steps of a raw slot
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t kRawBytes = Shape<P>::kRawBytes, kWide = PAIR ? 256 : 128;
    const Int4Args &a = p.a;
    // (the shuffle tells the compiler that the role is the warp's: its loops' values then stay in uniform
    // registers, which the matrix instructions take their operands from)
    const uint32_t lane = threadIdx.x & 31u, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const uint32_t stage_bytes = W * (kQuantBytes + p.dense_bytes);
    const uint32_t raw0 = base + p.stages * stage_bytes, bars = raw0 + p.raws * kRawBytes;
    auto full = [&](uint32_t i) { return bars + 8 * i; };  // both operands of a stage
    auto stage_free = [&](uint32_t i) { return bars + 64 + 8 * i; };
    auto raw_full = [&](uint32_t i) { return bars + 128 + 8 * i; };
    auto raw_free = [&](uint32_t i) { return bars + 192 + 8 * i; };
    auto acc_full = [&](uint32_t i) { return bars + 256 + 8 * i; };
    auto acc_free = [&](uint32_t i) { return bars + 272 + 8 * i; };
    const uint32_t tmem_slot = bars + 288;
    // the walkers over tiles are CTAs or pairs; `half` is this CTA's place in its pair
    const uint32_t half = PAIR ? blockIdx.x & 1u : 0u, walker = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const uint32_t walkers = PAIR ? gridDim.x / 2 : gridDim.x;
    // this CTA's share of the contraction (whole raw slots)
    const uint32_t splits = PAIR ? 1 : gridDim.y, rank = PAIR ? 0 : blockIdx.y;
    const uint32_t slot_lo = uint32_t(uint64_t(rank) * p.slots / splits), slot_hi = uint32_t(uint64_t(rank + 1) * p.slots / splits);
    const uint32_t step_lo = slot_lo * kSteps, steps = min(slot_hi * kSteps, p.steps) - step_lo;
    // a tile's first index of D's rows (this CTA's 128 of them) and of its columns
    auto row0 = [&](uint32_t tile) { return kWide * (tile / p.tiles_b) + 128 * half; };
    auto col0 = [&](uint32_t tile) { return int64_t(tile % p.tiles_b) * p.bn; };
    // the first of the CTA's 128 features of the quantized operand: o (forward) or k
    auto quant0 = [&](uint32_t tile) { return P == kScaleGrad ? uint32_t(col0(tile)) + 128 * half : row0(tile); };

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < p.stages; ++i) {
            // four expansion warps, the dense operand's copy (or its warps), the other CTA's stage
            mbar_init(full(i), 4 + (TMA ? 1 : kLoadWarps) + (PAIR && half == 0 ? 1 : 0));
            mbar_init(stage_free(i), 1);
        }
        for (uint32_t i = 0; i < p.raws; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_free(i), kExpandWarps);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_free(i), PAIR ? 2 * kOutWarps : kOutWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // the other CTA's barriers are ready
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = __shfl_sync(0xffffffffu, lds32(tmem_slot), 0);
    uint32_t err = 0;
    // sums for the cluster lie where the stages were (one tile a CTA then)
    float *joint = reinterpret_cast<float *>(smem);

    if (warp < kExpandWarps) {
        // ---- expand the quantized operand: group warp / 4 takes every kGroups-th step, a row of 64 elements
        // (128 bytes) a thread: row r of the 128, that is (forward) output feature r, or (input gradient, scale
        // gradient) output feature or token r % 64, inputs 64 (r / 64) .. of the tile's 128
        const uint32_t group = warp >> 2, r = 32 * (warp & 3u) + lane, cc = r >> 6;
        const uint32_t group_bits = 31 - __clz(a.group);
        uint32_t scale[W][2];
        // the thread's scales in a step (0 where there is none), read one step ahead.  What only a new tile
        // changes is kept: recomputed each step, its division and products cost as much as the expansion
        const uint16_t *scale_row = nullptr;  // of the tile: row r's (forward), or its first row's, at its first k
        const float *act_row = nullptr;
        uint32_t scale_k = 0;                 // first k of the thread's 64 (input gradient)
        bool scale_in = false;
        auto enter_tile = [&](uint32_t tile) {
            if (tile >= p.tiles) return;
            const uint32_t a0 = quant0(tile);
            if constexpr (P == kScaleGrad) {
                act_row = a.act_scales + int64_t(kSpan * step_lo + (r & 63u)) * a.act_groups + a0 / 128;
                scale_in = a0 < a.k;
            } else if constexpr (P == kForward) {
                scale_in = a0 + r < a.n;
                scale_row = a.scales + int64_t(a0 + r) * a.groups;
            } else {
                scale_k = a0 + 64 * cc;
                scale_in = scale_k < a.k;
                scale_row = a.scales + int64_t(kSpan * step_lo + (r & 63u)) * a.groups + (scale_k >> group_bits);
            }
        };
        auto load_scales = [&](uint32_t i) {  // step i of the tile entered last
#pragma unroll
            for (uint32_t w = 0; w < W; ++w) {
                const uint32_t from = kSpan * i + 64 * w, at_k = kSpan * step_lo + from;  // along the contraction
                scale[w][0] = scale[w][1] = 0u;
                if constexpr (P == kScaleGrad) {
                    if (scale_in && at_k + (r & 63u) < a.m) scale[w][0] = ldg_now32(act_row + int64_t(from) * a.act_groups);
                } else {
                    const uint32_t k = P == kForward ? at_k : scale_k;
                    const uint16_t *at = P == kForward ? scale_row + (k >> group_bits) : scale_row + int64_t(from) * a.groups;
                    if (scale_in && (P == kForward ? W == 1 || k < a.k : at_k + (r & 63u) < a.n)) {
                        scale[w][0] = ldg_now16(at);
                        // one load for groups of 64 and more: every lane's is a line of its own.  Inputs beyond the
                        // last have codes of 0, which stand for -8: they get the scale 0, which no scale's range can
                        // spoil
                        if (k + 32 < a.k) scale[w][1] = a.group == 32 ? ldg_now16(at + 1) : scale[w][0];
                    }
                }
            }
        };
        Walk mine{walker, 0};  // this group's next step
        mine.advance(group, steps, walkers);
        Ring stage, raw;
        stage.advance(group, p.stages);
        enter_tile(mine.tile);
        if (mine.tile < p.tiles) load_scales(mine.i);
        // every group passes every slot, in order, and frees it, whether it has a step there or not: none is
        // ever further ahead of another than the ring is long, so no turn is taken for another
        for (Walk at{walker, 0}; at.tile < p.tiles; raw.advance(1, p.raws)) {
            if (!mbar_wait(raw_full(raw.at), raw.phase)) {
                err = EP_DEC_TIMEOUT;
                break;
            }
            const uint32_t left = min(kSteps, steps - at.i), js = mine.i - at.i;
            const bool has = mine.tile == at.tile && js < left;
            at.i += left;
            if (at.i == steps) at.i = 0, at.tile += walkers;
            if (!has) {
                __syncwarp();
                if (lane == 0) mbar_arrive(raw_free(raw.at));
                continue;
            }
            uint32_t now[W][2];
#pragma unroll
            for (uint32_t w = 0; w < W; ++w) now[w][0] = scale[w][0], now[w][1] = scale[w][1];
            const uint32_t tile = mine.tile;
            mine.advance(kGroups, steps, walkers);
            if (mine.tile != tile) enter_tile(mine.tile);
            if (mine.tile < p.tiles) load_scales(mine.i);
            const uint32_t src = raw0 + raw.at * kRawBytes;
#pragma unroll
            for (uint32_t w = 0; w < W; ++w) {
                const uint32_t sub = js * W + w;  // which 64 of the slot's
                uint32_t out[8][4];
                if constexpr (P == kScaleGrad) {
                    const float s = __uint_as_float(now[w][0]) * Act<T>::kScale;
                    uint32_t hi = Elem<T>::bits(s), lo = Elem<T>::bits(s - Elem<T>::f(uint16_t(hi)));
                    hi |= hi << 16;
                    lo |= lo << 16;
                    const uint32_t row = 64 * sub + (r & 63u);
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        uint32_t q[4];
                        lds128(q, src + 128 * row + 16 * ((4 * cc + i) ^ (row & 7u)));
#pragma unroll
                        for (uint32_t e = 0; e < 8; ++e) {
                            const uint32_t v = Act<T>::pair(q[e / 2], e & 1u);
                            out[2 * i + e / 4][e & 3u] = Codes<T>::fma2(v, hi, mul2<T>(v, lo));
                        }
                    }
                } else {
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        uint32_t q[4];
                        if constexpr (P == kForward) {
                            lds128(q, src + 128 * r + 16 * ((2 * sub + i) ^ (r & 7u)));
                        } else {
                            const uint32_t row = 64 * sub + (r & 63u);
                            lds128(q, src + 64 * row + 16 * ((2 * cc + i) ^ ((row >> 1) & 3u)));
                        }
                        const uint32_t s2 = now[w][i] | (now[w][i] << 16);
#pragma unroll
                        for (uint32_t e = 0; e < 4; ++e) {
                            code_pairs<T>(q[e], out[4 * i + e]);
#pragma unroll
                            for (uint32_t h = 0; h < 4; ++h) out[4 * i + e][h] = mul2<T>(out[4 * i + e][h], s2);
                        }
                    }
                }
                if (w == 0 && !mbar_wait(stage_free(stage.at), stage.phase ^ 1u)) {
                    err = EP_DEC_TIMEOUT;
                    break;
                }
                const uint32_t dst = base + stage.at * stage_bytes + w * kQuantBytes + 128 * r;
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) sts128(dst + 16 * (i ^ (r & 7u)), out[i]);
            }
            if (err) break;
            // the stores are visible to the matrix unit, and the loads that fed them are done, so that the slot can
            // be written again (freed before the stores, loads still under way returned the next slot's bytes)
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full(stage.at));
                mbar_arrive(raw_free(raw.at));
            }
            stage.advance(kGroups, p.stages);
        }
    } else if (warp < kMmaWarp) {
        // ---- the output: warp q of the four reads lanes 32 q .. of the accumulator
        const uint32_t q = warp - kOutWarp0;
        Ring acc;
        for (uint32_t tile = walker; tile < p.tiles; tile += walkers, acc.advance(1, 2)) {
            const uint32_t a0 = row0(tile);
            const int64_t b0 = col0(tile);
            // scale gradient: the lane's output feature o, and its codes of the tile (their loads under way while
            // the tile's sums are; loaded as they are used they made a tile's output 4 us)
            const uint32_t o = a0 + 32 * q + lane;
            uint4 codes[P == kScaleGrad ? kWide / 32 : 1];
            if constexpr (P == kScaleGrad) {
                const uint4 *at = reinterpret_cast<const uint4 *>(a.codes + int64_t(min(o, a.n - 1)) * a.words + b0 / 8);
#pragma unroll
                for (uint32_t c = 0; c < kWide / 32; ++c)  // 32 inputs: 16 bytes
                    codes[c] = uint32_t(b0) + 32 * c < 8 * a.words
                                   ? __ldg(at + c)
                                   : make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
            }
            // a whole tile's wait: its limit grows with the contraction
            bool ready = false;
            for (uint32_t i = 0; i <= steps / 1024 && !ready; ++i) ready = mbar_wait(acc_full(acc.at), acc.phase);
            if (!ready) {
                err = EP_DEC_TIMEOUT;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t from = tmem + ((32u * q) << 16) + acc.at * p.bn;
            if constexpr (P == kScaleGrad) {
                // its row of D times its codes, summed over 32 inputs, then over a group
                uint16_t *out = a.out + int64_t(o) * a.groups + b0 / a.group;
                float sum = 0.0f, all = 0.0f;
#pragma unroll
                for (uint32_t c = 0; c < kWide / 32; ++c) {
                    const uint32_t w[4] = {codes[c].x, codes[c].y, codes[c].z, codes[c].w};
                    float s = 0.0f;
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        uint32_t d[16];
                        tmem_load16(d, from + 32 * c + 16 * h);
#pragma unroll
                        for (uint32_t e = 0; e < 16; ++e) {
                            // (2^23 + the code, less 2^23 + 8: a conversion runs at an eighth of the rate)
                            const uint32_t in = e & 7u, code = (w[2 * h + e / 8] >> (4 * (in / 2) + 16 * (in & 1u))) & 15u;
                            s = fmaf(__uint_as_float(d[e]), __uint_as_float(0x4b000000u | code) - 8388616.0f, s);
                        }
                    }
                    all += s;
                    if (splits > 1) {
                        joint[4 * (32 * q + lane) + c] = s;
                        continue;
                    }
                    sum += s;
                    if ((32 * (c + 1)) % a.group == 0) {  // a group's end (groups do not cross tiles)
                        if (o < a.n && b0 / a.group + c * 32 / a.group < a.groups) out[c * 32 / a.group] = Elem<T>::bits(sum);
                        sum = 0.0f;
                    }
                }
                // Where a sum is NaN, the group that k ends in again, without the columns behind the last input: an
                // infinite dy times their zeros is NaN and no part of the formula.  (Left out in the loop above, with
                // an index compared for every column or every 16, they made 1024 x 4096 x 4096 35.3 us instead of 33.4.)
                const uint32_t inputs = a.k - uint32_t(b0);
                if (inputs < kWide && inputs % a.group != 0 && __any_sync(0xffffffffu, all != all)) {
                    const uint32_t g = inputs / a.group;
                    sum = 0.0f;
                    for (uint32_t c = g * a.group / 32; c < (g + 1) * a.group / 32; ++c) {
                        const uint32_t *w = a.codes + int64_t(min(o, a.n - 1)) * a.words + b0 / 8 + 4 * c;
                        float s = 0.0f;
#pragma unroll 1
                        for (uint32_t h = 0; h < 2; ++h) {
                            uint32_t d[16];
                            tmem_load16(d, from + 32 * c + 16 * h);
#pragma unroll
                            for (uint32_t e = 0; e < 16; ++e) {
                                const uint32_t in = e & 7u, at = 32 * c + 16 * h + e;
                                const uint32_t code = at < inputs ? (__ldg(w + 2 * h + e / 8) >> (4 * (in / 2) + 16 * (in & 1u))) & 15u : 8u;
                                s = fmaf(at < inputs ? __uint_as_float(d[e]) : 0.0f, float(int(code) - 8), s);
                            }
                        }
                        if (splits > 1) joint[4 * (32 * q + lane) + c] = s;
                        sum += s;
                    }
                    if (splits == 1 && o < a.n) out[g] = Elem<T>::bits(sum);
                }
            } else {
                const uint32_t J = P == kForward ? a.n : a.k, f = 32 * q + lane, j = a0 + f;
                const float b = P == kForward && a.bias && j < J ? Elem<T>::f(__ldg(a.bias + j)) : 0.0f;
                for (uint32_t c = 0; c < p.bn; c += 16) {
                    uint32_t d[16];
                    tmem_load16(d, from + c);
                    if (splits > 1) {
#pragma unroll
                        for (uint32_t i = 0; i < 16; ++i) joint[128 * (c + i) + f] = __uint_as_float(d[i]);
                    } else if (j < J) {
#pragma unroll
                        for (uint32_t i = 0; i < 16; ++i)
                            if (b0 + c + i < a.m)
                                a.out[(b0 + c + i) * J + j] = Elem<T>::bits(__uint_as_float(d[i]) * Codes<T>::kUnit + b);
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_issuer<PAIR>(acc_free(acc.at));
        }
    } else if (warp == kMmaWarp) {
        // ---- the matrix instructions, 16 of the contraction each, issued by one elected lane of a converged
        // warp: little may lie between two steps' instructions, which take 512 cycles a step back to back (of
        // 256 columns).  A pair's second CTA passes on to the first that its stages are full
        const bool elected = elect_one();
        // forward: the step with inputs behind the last that share its 32's scale, whose infinity times their code 0
        // is NaN and no part of the formula.  They are zeroed here, where there is time: looked for by the warps
        // that expand, 17 tokens of 8192 x 28672 took 64.5 us instead of 60.2, 2048 of 8192 x 8192 194 instead of 181
        const uint32_t end_step = a.k % 32 != 0 ? a.k / kSpan - step_lo : ~0u;
        Ring stage, acc;
        for (uint32_t tile = walker; tile < p.tiles && !err; tile += walkers, acc.advance(1, 2)) {
            if (half == 0 && !mbar_wait(acc_free(acc.at), acc.phase ^ 1u)) {
                err = EP_DEC_TIMEOUT;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + acc.at * p.bn;
            for (uint32_t i = 0; i < steps; ++i) {
                const uint32_t quant = base + stage.at * stage_bytes, dense = quant + W * kQuantBytes;
                // a step of 16: 32 bytes along K-major rows, 16 rows of 128 bytes of the others
                constexpr uint64_t kQ = P == kForward ? 2 : 128, kD = P == kScaleGrad ? 128 : 2;
                if (!mbar_wait(full(stage.at), stage.phase)) {
                    err = EP_DEC_TIMEOUT;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (P == kForward && i == end_step) {
                    zero_behind(quant + (W == 2 ? (a.k >> 6) & 1u : 0u) * kQuantBytes, a.k & 63u, lane);
                    fence_proxy_async();
                    __syncwarp();
                }
                if (half == 0) {
                    if (elected) {
#pragma unroll
                        for (uint32_t w = 0; w < W; ++w) {
                            const uint64_t dq = desc128(quant + w * kQuantBytes, P == kForward ? 0 : 8192);
                            const uint64_t dd = desc128(dense + w * p.dense_bytes, P == kScaleGrad ? 8192 : 0);
#pragma unroll
                            for (uint32_t h = 0; h < 4; ++h)
                                mma_f16<PAIR>(d, P == kScaleGrad ? dd + h * kD : dq + h * kQ,
                                              P == kScaleGrad ? dq + h * kQ : dd + h * kD, p.idesc, i > 0 || w > 0 || h > 0);
                        }
                        mma_commit<PAIR>(stage_free(stage.at));
                    }
                } else if (elected) {
                    arrive_issuer<PAIR>(full(stage.at));
                }
                __syncwarp();
                stage.advance(1, p.stages);
            }
            if (half == 0 && elected) mma_commit<PAIR>(acc_full(acc.at));
            __syncwarp();
        }
    } else if (warp == kRawWarp) {
        // ---- the quantized operand's bytes, as buffers come free
        if (lane == 0) {
            Ring raw;
            uint32_t copies = 0;
            for (uint32_t tile = walker; tile < p.tiles && !err; tile += walkers) {
                const uint32_t a0 = quant0(tile);
                for (uint32_t slot = slot_lo; slot < slot_hi; ++slot, ++copies, raw.advance(1, p.raws)) {
                    if (!mbar_wait(raw_free(raw.at), raw.phase ^ 1u)) {
                        err = EP_DEC_TIMEOUT;
                        break;
                    }
                    const uint32_t dst = raw0 + raw.at * kRawBytes, bar = raw_full(raw.at);
                    mbar_expect(bar, kRawBytes);
                    if constexpr (P == kForward)
                        tma_load(dst, &p.raw, 128 * slot, a0, bar);
                    else if constexpr (P == kInputGrad)
                        tma_load(dst, &p.raw, a0 / 2, 256 * slot, bar);
                    else
                        tma_load(dst, &p.raw, a0, 256 * slot, bar);
                }
            }
            // no copy is in flight when the CTA ends: the last use of each buffer
            for (uint32_t i = copies > p.raws ? copies - p.raws : 0; i < copies; ++i)
                if (!mbar_wait(raw_full(i % p.raws), (i / p.raws) & 1u)) err = EP_DEC_TIMEOUT;
        }
        __syncwarp();
    } else if (TMA) {
        // ---- the dense operand by TMA
        if (lane == 0) {
            Ring stage;
            uint32_t copies = 0;
            for (uint32_t tile = walker; tile < p.tiles && !err; tile += walkers) {
                const uint32_t b0 = P == kScaleGrad ? row0(tile) : uint32_t(col0(tile)) + (PAIR ? p.bn / 2 : 0u) * half;
                for (uint32_t i = 0; i < steps; ++i, ++copies, stage.advance(1, p.stages)) {
                    if (!mbar_wait(stage_free(stage.at), stage.phase ^ 1u)) {
                        err = EP_DEC_TIMEOUT;
                        break;
                    }
                    const uint32_t bar = full(stage.at);
                    mbar_expect(bar, W * p.dense_bytes);
#pragma unroll
                    for (uint32_t w = 0; w < W; ++w) {
                        const uint32_t dst = base + stage.at * stage_bytes + W * kQuantBytes + w * p.dense_bytes;
                        const uint32_t c = kSpan * (step_lo + i) + 64 * w;  // (beyond the contraction: zeros)
                        if constexpr (P == kScaleGrad) {
                            tma_load(dst, &p.dense, b0, c, bar);
                            tma_load(dst + 8192, &p.dense, b0 + 64, c, bar);
                        } else {
                            tma_load(dst, &p.dense, c, b0, bar);
                        }
                    }
                }
            }
            for (uint32_t i = copies > p.stages ? copies - p.stages : 0; i < copies; ++i)
                if (!mbar_wait(full(i % p.stages), (i / p.stages) & 1u)) err = EP_DEC_TIMEOUT;
        }
        __syncwarp();
    } else {
        // ---- the dense operand through registers: 16-byte chunks of 8 elements, each checked
        const uint32_t cols_all = P == kForward ? a.k : a.n;
        Ring stage;
        for (uint32_t tile = walker; tile < p.tiles && !err; tile += walkers) {
            const int64_t b0 = P == kScaleGrad ? int64_t(row0(tile)) : col0(tile);
            for (uint32_t i = 0; i < steps; ++i, stage.advance(1, p.stages)) {
                const uint32_t step = step_lo + i;
                if (!mbar_wait(stage_free(stage.at), stage.phase ^ 1u)) {
                    err = EP_DEC_TIMEOUT;
                    break;
                }
                const uint32_t dst = base + stage.at * stage_bytes + kQuantBytes;
                // four chunks of a thread at a time, their loads in flight together
                const uint32_t chunks = p.dense_bytes / 16, first = threadIdx.x - 32 * kDenseWarp0;
                for (uint32_t e0 = first; e0 < chunks; e0 += 4 * 32 * kLoadWarps) {
                    uint32_t v[4][4];
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {
                        const uint32_t e = e0 + u * 32 * kLoadWarps, c = e & 7u;
                        const uint32_t r = P == kScaleGrad ? (e >> 3) & 63u : e >> 3, box = P == kScaleGrad ? e >> 9 : 0u;
                        const int64_t t = (P == kScaleGrad ? 64 * int64_t(step) : b0) + r;
                        const uint32_t col = (P == kScaleGrad ? uint32_t(b0) + 64 * box : 64 * step) + 8 * c;
                        const uint16_t *src = a.x + t * a.ldx + col;
                        v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0u;
                        if (e >= chunks || t >= a.m || col >= cols_all) continue;
                        if (p.dense_align >= 4 && col + 8 <= cols_all) {
#pragma unroll
                            for (uint32_t h = 0; h < 4; ++h) v[u][h] = __ldg(reinterpret_cast<const uint32_t *>(src) + h);
                        } else {
#pragma unroll
                            for (uint32_t h = 0; h < 4; ++h) {
                                const uint32_t lo = col + 2 * h < cols_all ? __ldg(src + 2 * h) : 0u;
                                const uint32_t hi = col + 2 * h + 1 < cols_all ? __ldg(src + 2 * h + 1) : 0u;
                                v[u][h] = lo | (hi << 16);
                            }
                        }
                    }
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {
                        const uint32_t e = e0 + u * 32 * kLoadWarps, row = e >> 3;  // 128-byte rows, boxes of 64
                        if (e < chunks) sts128(dst + 128 * row + 16 * ((e & 7u) ^ (row & 7u)), v[u]);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(full(stage.at));
            }
        }
    }

    // ---- a split contraction: each CTA adds its share of the tile over the cluster
    if (splits > 1) {
        const uint32_t a0 = row0(walker);
        const int64_t b0 = col0(walker);
        cluster_sync();
        if constexpr (P == kScaleGrad) {
            const uint32_t per = 128 / a.group, span = 4 / per;
            for (uint32_t e = rank * blockDim.x + threadIdx.x; e < 128 * per; e += splits * blockDim.x) {
                const uint32_t o = a0 + e / per, i = e % per, g = uint32_t(b0) / a.group + i;
                float s = 0.0f;
                for (uint32_t c = 0; c < splits; ++c)
                    for (uint32_t h = i * span; h < (i + 1) * span; ++h) s += ld_cluster(&joint[4 * (e / per) + h], c);
                if (o < a.n && g < a.groups) a.out[int64_t(o) * a.groups + g] = Elem<T>::bits(s);
            }
        } else {
            const uint32_t J = P == kForward ? a.n : a.k, f = threadIdx.x & 127u, j = a0 + f, rows = blockDim.x / 128;
            if (threadIdx.x / 128 < rows && j < J) {
                const float b = P == kForward && a.bias ? Elem<T>::f(__ldg(a.bias + j)) : 0.0f;
                for (uint32_t c = rank * rows + threadIdx.x / 128; c < p.bn && b0 + c < a.m; c += splits * rows) {
                    float s = 0.0f;
                    for (uint32_t h = 0; h < splits; ++h) s += ld_cluster(&joint[128 * c + f], h);
                    a.out[(b0 + c) * J + j] = Elem<T>::bits(s * Codes<T>::kUnit + b);
                }
            }
        }
        cluster_sync();
    }
    if (err && a.status && lane == 0) atomicOr(a.status, err);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other still reads or signals it
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
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
constexpr size_t kSmemMost = 232448;

// How many clusters of `size` CTAs, one on each SM, run at once on the current device: a cluster lies within one
// GPC, whose SMs it may not use up (looked up once per device and size)
uint32_t clusters_at_once(int device, uint32_t size) {
    static std::atomic<int> known[64][9];
    int n = known[device][size].load();
    if (n) return uint32_t(n);
    const auto kern = int4_mma_kernel<__nv_bfloat16, kForward, true, false, 1>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, size);
    cfg.blockDim = dim3((kDenseWarp0 + 1) * 32);
    cfg.dynamicSmemBytes = kSmemMost;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = size;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMost)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();  // (a query's error is not the launch's)
        return 0;
    }
    known[device][size].store(n);
    return uint32_t(n);
}

// the launch: single or paired CTAs, tiles, the contraction's split, rings as deep as fit
template <typename T, int P>
int launch_mma(const Int4Args &a, int sms, cudaStream_t s) {
    MmaArgs p{};
    p.a = a;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return EP_ERR_CUDA;
    const int64_t contraction = P == kForward ? a.k : P == kInputGrad ? int64_t(a.n) : a.m;
    const uint32_t sixty_fours = uint32_t((contraction + 63) / 64);
    p.slots = (sixty_fours + kSlotSteps - 1) / kSlotSteps;
    const uint64_t dense_cols = P == kForward ? a.k : a.n;
    const int64_t ld = a.m > 1 ? a.ldx : int64_t((dense_cols + 7) / 8 * 8);
    const bool tma = !misaligned(a.x, 16) && ld % 8 == 0 && ld < (int64_t(1) << 38) && a.m <= 0x7fffffff;
    p.dense_align = !misaligned(a.x, 4) && ld % 2 == 0 ? 4 : 2;
    const uint64_t rows = P == kInputGrad ? a.k : a.n, cols = P == kScaleGrad ? a.k : uint64_t(a.m);
    // pairs where their tiles (256 x 256) keep most SMs busy: from 3/8 of a tile per SM, a quarter in the
    // scale gradient, whose single tiles are half as wide.  Measured, pairs against single CTAs with the
    // contraction split: forward 512 x 4096 x 4096 (32 tiles) 31 us against 25, 1024 x 4096 x 4096 (64) 32
    // against 33; scale gradient 2048 x 1024 x 1536 (24) 18.6 against 17.0, 2048 x 1536 x 2048 (48) 20 against 29
    const uint64_t pair_tiles = ((rows + 255) / 256) * ((cols + 255) / 256);
    const bool pair = tma && cols > 128 && pair_tiles * 8 >= uint64_t(sms) * (P == kScaleGrad ? 2 : 3);
    const uint64_t tiles_a = pair ? (rows + 255) / 256 : (rows + 127) / 128;
    uint64_t tiles_b;
    if (P == kScaleGrad) {
        p.bn = pair ? 256 : 128;
        tiles_b = (cols + p.bn - 1) / p.bn;
        p.dense_bytes = 16384;
    } else {
        const uint32_t unit = pair ? 32 : 16;
        tiles_b = (cols + 255) / 256;
        p.bn = uint32_t(((cols + tiles_b - 1) / tiles_b + unit - 1) / unit * unit);
        p.dense_bytes = (pair ? p.bn / 2 : p.bn) * 128;
    }
    if (tiles_a * tiles_b > 0x3fffffff) return EP_ERR_UNSUPPORTED;
    p.tiles = uint32_t(tiles_a * tiles_b);
    p.tiles_b = uint32_t(tiles_b);
    uint32_t splits = 1;
    if (!pair && p.tiles < uint32_t(sms)) {
        splits = std::max(1u, std::min({8u, sms / p.tiles, p.slots}));
        while (splits > 1 && p.tiles > clusters_at_once(device, splits)) --splits;
    }
    // Steps of 128 spend fewer instructions on their barriers, where they leave three raw slots: forward, 17
    // tokens, 8192 x 28672 56.7 us against 63.1, 48 tokens 60.5 against 64.2, 4096 x 4096 11.5 against 12.2; with 64
    // tokens, and two slots, 83.7 against 64.6; the input gradient, one token, 8192 x 8192 29.9 against 24.7
    constexpr uint32_t kWide = P == kForward ? 2 : 1;
    const bool wide = kWide == 2 && tma && !pair && p.bn <= 48 && sixty_fours >= 8 * splits;
    const uint32_t w = wide ? kWide : 1;
    p.steps = (sixty_fours + w - 1) / w;
    const uint32_t stage = w * (kQuantBytes + p.dense_bytes), raw = Shape<P>::kRawBytes;
    // 64 KB of raw slots where that leaves five stages, otherwise two slots and as many stages as fit
    // (2048 x 8192 x 8192 forward, paired: 4 slots and 5 stages 187 us, 2 and 6 195 us)
    const uint32_t room = uint32_t(kSmemMost - kBarBytes);
    p.raws = 65536 / raw;
    if (room < p.raws * raw + 5 * stage) p.raws = 2;
    p.stages = std::min<uint32_t>(kMaxStages, (room - p.raws * raw) / stage);
    p.raws = std::min<uint32_t>(kMaxRaws, (room - p.stages * stage) / raw);
    // a group waits for the matrix instructions that read its stage last; it has seen those of the turn
    // before done only if the ring holds a step of every group
    if (p.stages < kGroups) return EP_ERR_UNSUPPORTED;
    const size_t bytes = size_t(p.stages) * stage + size_t(p.raws) * raw + kBarBytes;
    // accumulator fp32, A and B of T; the scale gradient's operands and the input gradient's weight MN-major
    const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    p.idesc = (1u << 4) | (type << 7) | (type << 10) | (P != kForward ? 1u << 15 : 0u) | (P == kScaleGrad ? 1u << 16 : 0u) |
              ((p.bn >> 3) << 17) | (((pair ? 256u : 128u) >> 4) << 24);
    p.tmem_cols = 32;
    while (p.tmem_cols < 2 * p.bn) p.tmem_cols *= 2;
    const CUtensorMapDataType dt = type ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t pitch = P == kScaleGrad ? uint64_t(act8_row_bytes(a.k)) : uint64_t(a.words) * 4;
    const void *quant = P == kScaleGrad ? static_cast<const void *>(a.act) : static_cast<const void *>(a.codes);
    if (!tensor_map(&p.raw, quant, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, pitch, P == kScaleGrad ? uint64_t(a.m) : a.n, pitch,
                    P == kInputGrad ? 64 : 128, P == kForward ? 128 : 256))
        return EP_ERR_CUDA;
    if (tma && !tensor_map(&p.dense, a.x, dt, 2, dense_cols, uint64_t(a.m), uint64_t(ld) * 2, 64,
                           P == kScaleGrad ? 64 : p.dense_bytes / 128))
        return EP_ERR_CUDA;
    const uint32_t form = pair ? 2 : wide ? 3 : tma ? 1 : 0;
    const auto kern = pair   ? int4_mma_kernel<T, P, true, true, 1>
                      : wide ? int4_mma_kernel<T, P, true, false, kWide>
                      : tma  ? int4_mma_kernel<T, P, true, false, 1>
                             : int4_mma_kernel<T, P, false, false, 1>;
    static std::atomic<uint64_t> allowed[4];  // devices on which the kernel may use kSmemMost
    if (!(allowed[form].load() >> device & 1u)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMost)) != cudaSuccess)
            return EP_ERR_CUDA;
        allowed[form].fetch_or(uint64_t(1) << device);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = pair ? dim3(2 * std::min(p.tiles, uint32_t(sms) / 2))
                       : dim3(splits > 1 ? p.tiles : std::min(p.tiles, uint32_t(sms)), splits);
    cfg.blockDim = dim3((kDenseWarp0 + (tma ? 1 : kLoadWarps)) * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = pair ? 2 : 1;
    attr[0].val.clusterDim.y = splits;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pair || splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
template <int P>
int launch(const Int4Args &a, int32_t dtype, int sms, cudaStream_t s) {
    return dtype == EP_BF16 ? launch_mma<__nv_bfloat16, P>(a, sms, s) : launch_mma<__half, P>(a, sms, s);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

}  // namespace

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

bool tensor_map(CUtensorMap *map, const void *base, CUtensorMapDataType type, uint32_t elt, uint64_t cols, uint64_t rows,
                uint64_t pitch, uint32_t box_cols, uint32_t box_rows) {
    static std::atomic<void *> known{nullptr};
    void *fn = known.load();
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !fn)
            return false;
        known.store(fn);
    }
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
    const uint32_t row = box_cols * elt;
    const CUtensorMapSwizzle swizzle = row == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_32B;
    const auto encode = [&] {
        return reinterpret_cast<EncodeTiled>(fn)(map, type, 2, const_cast<void *>(base), dims, strides, box, one,
                                                 CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult rc = encode();
    if (rc == CUDA_ERROR_INVALID_CONTEXT || rc == CUDA_ERROR_NOT_INITIALIZED) {
        // a thread that has made no runtime call that binds the device's context (autograd's, say)
        int device;
        if (cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess) rc = encode();
    }
    return rc == CUDA_SUCCESS;
}

}  // namespace ep

extern "C" int ep_int4_linear(const void *d_codes, const void *d_scales, int64_t n, int64_t k, int32_t group,
                              int32_t dtype, const void *d_x, int64_t m, int64_t ldx, const void *d_bias, void *d_y,
                              uint32_t *d_status, ep_stream_t stream) {
    using namespace ep;
    if (!weight_ok(n, k, group, dtype) || m < 0 || m > kMaxDim || (m > 1 && ldx < k)) return EP_ERR_INVALID_ARG;
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
    return launch<kForward>(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int ep_int4_linear_dx(const void *d_codes, const void *d_scales, int64_t n, int64_t k, int32_t group,
                                 int32_t dtype, const void *d_dy, int64_t m, int64_t lddy, void *d_dx,
                                 uint32_t *d_status, ep_stream_t stream) {
    using namespace ep;
    if (!weight_ok(n, k, group, dtype) || m < 0 || m > kMaxDim || (m > 1 && lddy < n)) return EP_ERR_INVALID_ARG;
    if (m == 0) return EP_OK;
    if (!d_codes || !d_scales || !d_dy || !d_dx || misaligned(d_codes, 16) || misaligned(d_scales, 2) ||
        misaligned(d_dy, 2) || misaligned(d_dx, 2) || misaligned(d_status, 4))
        return EP_ERR_INVALID_ARG;
    Int4Args a = args_of(n, k, group, d_codes, d_scales);
    a.x = static_cast<const uint16_t *>(d_dy);
    a.ldx = lddy;
    a.m = m;
    a.out = static_cast<uint16_t *>(d_dx);
    a.status = d_status;
    const int sms = device_sms();
    if (sms < 1) return EP_ERR_CUDA;
    return launch<kInputGrad>(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int ep_int4_scale_grad(const void *d_dy, int64_t lddy, const void *d_act, const float *d_act_scales,
                                  int64_t m, const void *d_codes, int64_t n, int64_t k, int32_t group, int32_t dtype,
                                  void *d_ds, uint32_t *d_status, ep_stream_t stream) {
    using namespace ep;
    if (!weight_ok(n, k, group, dtype) || m < 0 || m > kMaxDim || (m > 1 && lddy < n)) return EP_ERR_INVALID_ARG;
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
    a.status = d_status;
    if (m == 0)  // an empty sum
        return cudaMemsetAsync(d_ds, 0, size_t(n) * a.groups * 2, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? EP_OK
                   : EP_ERR_CUDA;
    const int sms = device_sms();
    if (sms < 1) return EP_ERR_CUDA;
    return launch<kScaleGrad>(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream));
}
