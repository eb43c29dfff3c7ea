// matmul.cu -- block-scaled products y = a w^T in BF16 on the 5th-generation
// tensor cores: MXFP8 x MXFP8 (1x32 UE8M0 scales) and NVFP4 x NVFP4 (1x16
// E4M3 scales and an FP32 global scale per batch index), for the quantised
// weights and activations of the rollout ("Low Precision RL", "Modes" 3 and
// 4; verl NVFP4 QAT article 2.5).
//
//   y[b][m][n] = bf16(ga_b gw_b sum_k dec(a[b][m][k]) sa[b][m][k / V]
//                                    dec(w[b][n][k]) sw[b][n][k / V])
//
// with V = 32, ga = gw = 1 for MXFP8 and V = 16 for NVFP4.  The tensor core
// multiplies codes and scales exactly and accumulates in FP32; the global
// scales multiply the finished FP32 sum, and the one rounding to BF16 is the
// output's.
//
// Scales arrive in the tile layout of pwq_internal.h (mma_scale_offset): a
// 512-byte tile is one tcgen05.cp (32 lines of 16 bytes) into four TMEM
// columns.
#include <algorithm>
#include <cuda.h>

#include "pwq_early.cuh"
#include "pwq_internal.h"
#include "pwq_tcgen05.cuh"

namespace pwq {
namespace {

__device__ uint32_t g_matmul_error = 0u;

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// A wait that gives up records it; the caller then leaves its loop and runs
// to the end of the kernel, so that TMEM is freed and every barrier is met.
__device__ __forceinline__ bool wait_or_record(uint32_t bar, uint32_t parity) {
    if (mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
    atomicOr(&g_matmul_error, kErrMatmulTimeout);
    return false;
}

// The same for a converged warp: every lane waits, and all get one answer.
// (One lane that polls for the warp takes 200 clocks longer to get through.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_record(bar, parity));
}

// True in every thread of the epilogue's 128 when `ok` is true in all of them.
__device__ __forceinline__ bool vote_all(bool ok) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)ok) : "memory");
    return r != 0u;
}

// ga * gw as a product of two FP32 factors, so that neither the scale nor a
// partial product leaves the FP32 range when the result does not: one factor
// is 1 unless the product of the scales is outside [2^-100, 2^100].
__device__ __forceinline__ float2 output_scale(const float* ga, const float* gw, int b) {
    if (!ga) return make_float2(1.0f, 1.0f);
    const double p = (double)ld_f32(ga + b) * (double)ld_f32(gw + b);
    if (p < 0x1p-100 && p > 0.0) return make_float2(0x1p-100f, (float)(p * 0x1p100));
    if (p > 0x1p100 && p < 0x1p1000) return make_float2(0x1p100f, (float)(p * 0x1p-100));
    return make_float2((float)p, 1.0f);
}

// An accumulator times the output scale (none for MXFP8).
template <ProductFormat kF>
__device__ __forceinline__ float scaled(uint32_t acc, float2 sc) {
    const float v = __uint_as_float(acc);
    return kF == ProductFormat::kNvfp4 ? v * sc.x * sc.y : v;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
}

// ---------------------------------------------------------------- few tokens: weights on the 128 lanes
//
// One CTA (one CTA per K range of a cluster) takes 128 weight rows as the
// MMA's M side and kTok tokens as its N side, so that one token costs an
// N = 16 MMA, not an M = 128 one, and y[t][n] leaves TMEM with consecutive
// lanes on consecutive n.  Weights stream once through a ring of 128-byte
// steps; few weight rows are split along K over the CTAs of a cluster, whose
// FP32 partials meet in distributed shared memory and are added in rank
// order (the result does not depend on timing).
//
// Bound by the weight's bytes and, for small weights, by the launch and the
// first loads' latency: 19456 x 2560 at one token takes 7.0 us in NVFP4
// (28 MB, 4.0 TB/s), 2560 x 9728 at eight in MXFP8 7.2 to 7.9 us on several
// GPUs (26 MB, 3.3 to 3.6 TB/s).
//
// Warps 0..3 epilogue, 4 and 6 TMA producers (codes, scales), 5 MMA issuer and TMEM owner.

constexpr int kTokThreads = 224, kMaxSplit = 8;

struct TokArgs {
    CUtensorMap w, ws, t, ts;    // weight codes / scales, token codes / scales
    const float* gt;             // NVFP4 global scales, null for MXFP8
    const float* gw;
    uint16_t* y;
    int64_t y_bs, y_rs;          // elements
    int n, m;                    // weight rows, tokens
    int w_bands, t_bands;        // 128-row scale bands per batch slab
    int steps, last_mmas;        // 128-byte steps of K, MMAs of the last one
    int split;                   // CTAs per cluster along K
    int y8;                      // y rows are 8-byte aligned
    FastDiv w_tiles, t_tiles;
};

template <ProductFormat kF, int kTok>
struct TokCfg {
    using T = ProductTraits<kF>;
    static constexpr uint32_t kW = 128u * kStepBytes, kT = (uint32_t)kTok * kStepBytes;
    static constexpr uint32_t kStage = kW + kT + 2u * T::kScaleBytes;
    // two CTAs per SM: a tile more than there are SMs must not cost a second wave
    // (NVFP4, 64 tokens, 152 tiles: 16.7 us with four stages and one CTA per SM, 11.4 us with three and two)
    static constexpr int kStages = kTok <= 16 || (kTok == 32 && !T::kFp4)  ? 5
                                   : kTok == 32 || (kTok == 64 && !T::kFp4) ? 4
                                                                           : 3;
    static constexpr uint32_t kSmem = kStages * kStage + 1024u;   // + alignment of the ring to 1024 bytes
    // TMEM: kTok accumulator columns, then a buffer of weight and token scale columns for each stage
    static constexpr uint32_t kScaleCols = 4u * T::kScaleTiles;
    static constexpr uint32_t kCols = 256u;   // two CTAs per SM fill it
    static_assert(kTok + 2u * kStages * kScaleCols <= kCols, "TMEM");
    static_assert(128u * kTok * 4u <= kStages * kStage, "the FP32 partial reuses the ring");
};

template <ProductFormat kF, int kTok>
__global__ void __launch_bounds__(kTokThreads, 2) tokens_kernel(const __grid_constant__ TokArgs a) {
    using T = ProductTraits<kF>;
    using C = TokCfg<kF, kTok>;
    constexpr int kS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kS + 1];
    __shared__ uint32_t tmem_word;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8u * kS, done = full + 16u * kS;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    const uint32_t rank = blockIdx.x % (uint32_t)a.split;
    uint32_t tile = blockIdx.x / (uint32_t)a.split;
    const uint32_t tq = fdiv(tile, a.w_tiles);
    const int wt = (int)(tile - tq * a.w_tiles.d);
    const int b = (int)fdiv(tq, a.t_tiles);
    const int tt = (int)(tq - (uint32_t)b * a.t_tiles.d);
    const int n0 = wt * 128, t0 = tt * kTok;
    // this CTA's steps of K
    const int s0 = (int)((int64_t)a.steps * rank / a.split), s1 = (int)((int64_t)a.steps * (rank + 1) / a.split);
    const int steps = s1 - s0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(full + 8u * i, 1);
            mbar_init(empty + 8u * i, 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 4 && elect_one()) {
        prefetch_tensor_map(&a.w);
        prefetch_tensor_map(&a.t);
        prefetch_tensor_map(&a.ws);
        prefetch_tensor_map(&a.ts);
    }
    if (warp == 5) tmem_alloc<1>(smem_addr(&tmem_word), C::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    let_later_kernels_start();
    wait_for_earlier_kernels();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_word, 0);

    if (warp == 4 || warp == 6) {
        const bool codes = warp == 4;   // the other one loads the scales
        const int w_band = b * a.w_bands + wt, t_band = b * a.t_bands + t0 / 128;
        int i = 0;
        for (; i < steps; ++i) {
            const int st = i % kS;
            if (i >= kS && !warp_wait(empty + 8u * st, ((i / kS) - 1) & 1)) break;
            const uint32_t at = ring + (uint32_t)st * C::kStage, bar = full + 8u * st;
            const int s = s0 + i;
            if (elect_one()) {
                if (codes) {
                    mbar_arrive_expect_tx(bar, C::kStage);
                    tma_load_3d(at, &a.w, bar, s * (int)kStepBytes, n0, b);
                    tma_load_3d(at + C::kW, &a.t, bar, s * (int)kStepBytes, t0, b);
                } else {
                    tma_load_3d(at + C::kW + C::kT, &a.ws, bar, 0, s * T::kScaleTiles, w_band);
                    tma_load_3d(at + C::kW + C::kT + T::kScaleBytes, &a.ts, bar, 0, s * T::kScaleTiles, t_band);
                }
            }
            __syncwarp();
        }
        // no copy is in flight when the CTA ends
        if (codes)
            for (int j = max(0, i - kS); j < i; ++j)
                if (!warp_wait(full + 8u * (j % kS), (j / kS) & 1)) break;
    } else if (warp == 5) {
        constexpr uint32_t idesc = mma_idesc<kF>(128, kTok);
        const uint32_t tok_col = (uint32_t)(t0 % 128) / 32u;   // 64-token tiles: the band's upper half
        const bool leader = elect_one();
        bool ready = false;   // the next operands' barrier, tested while a step is issued
        for (int i = 0; i < steps; ++i) {
            const int st = i % kS, nx = (i + 1) % kS;
            if (!__all_sync(0xffffffffu, ready) && !warp_wait(full + 8u * st, (i / kS) & 1)) break;
            tc_fence_after();
            const uint32_t at = ring + (uint32_t)st * C::kStage;
            const uint32_t sw = tmem + kTok + (uint32_t)st * 2u * C::kScaleCols, sx = sw + C::kScaleCols;
            const uint64_t dw = desc_swizzle128(at), dx = desc_swizzle128(at + C::kW);
            const int mmas = s0 + i == a.steps - 1 ? a.last_mmas : kMmasPerStep;
            if (leader) {
#pragma unroll
                for (int j = 0; j < T::kScaleTiles; ++j) {
                    copy_scales<1>(sw + 4u * j, desc_scales(at + C::kW + C::kT + 512u * j));
                    copy_scales<1>(sx + 4u * j, desc_scales(at + C::kW + C::kT + T::kScaleBytes + 512u * j));
                }
#pragma unroll
                for (int j = 0; j < kMmasPerStep; ++j) {
                    if (j >= mmas) break;
                    const uint32_t id = T::kFp4 ? idesc : idesc | (uint32_t)j << 4 | (uint32_t)j << 29;
                    const uint32_t so = T::kFp4 ? 4u * j : 0u;
                    mma_block_scaled<kF, 1>(tmem, dw + 2u * j, dx + 2u * j, id, sw + so, sx + so + tok_col,
                                            (i | j) != 0);
                }
            }
            ready = mbar_test(full + 8u * nx, ((i + 1) / kS) & 1);
            if (leader) mma_commit(empty + 8u * st);
        }
        __syncwarp();
        if (elect_one()) mma_commit(done);
        __syncwarp();
    } else {
        const bool ok = vote_all(warp != 0 || warp_wait(done, 0));   // the first warp polls for the four
        tc_fence_after();
        const float2 sc = output_scale(a.gt, a.gw, b);
        const int n = n0 + warp * 32 + lane;
        uint16_t* y = a.y + (int64_t)b * a.y_bs + n;
        const uint32_t row = tmem + ((uint32_t)warp << 21);   // lane 32 * warp in bits 16..
        constexpr int kChunk = kTok < 32 ? 16 : 32;
        for (int c0 = 0; c0 < kTok; c0 += kChunk) {
            uint32_t v[kChunk];
            if constexpr (kChunk == 16) tmem_ld16(row + c0, v);
            else tmem_ld32(row + c0, v);
            tmem_ld_wait();
            if (!ok) {
#pragma unroll
                for (int c = 0; c < kChunk; ++c) v[c] = 0u;
            }
            if (a.split == 1) {
#pragma unroll
                for (int c = 0; c < kChunk; ++c) {
                    const int t = t0 + c0 + c;
                    if (t < a.m && n < a.n)
                        y[(int64_t)t * a.y_rs] = bf16_bits(scaled<kF>(v[c], sc));
                }
            } else {
                // the loads have landed and the MMAs read the ring no more
#pragma unroll
                for (int c = 0; c < kChunk; ++c)
                    asm volatile("st.shared.b32 [%0], %1;" :: "r"(ring + ((uint32_t)(c0 + c) * 128u + threadIdx.x) * 4u),
                                 "r"(v[c]) : "memory");
            }
        }
    }
    if (a.split > 1) {
        __syncwarp();
        cluster_sync();
        if (warp < 4) {
            // this CTA finishes tokens rank, rank + split, ...; a warp takes one at a time, a lane four weight
            // rows, and the partials of all CTAs are loaded before the first addition (a load from a
            // neighbour takes several hundred clocks)
            const float2 sc = output_scale(a.gt, a.gw, b);
            const int n = n0 + lane * 4;
            for (int c = (int)rank + warp * a.split; c < kTok && t0 + c < a.m; c += 4 * a.split) {
                const uint32_t at = ring + (uint32_t)c * 512u + (uint32_t)lane * 16u;
                float4 v[kMaxSplit];
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q)
                    if (q < a.split) v[q] = ld_cluster_v4(cluster_addr(at, (uint32_t)q));
                float4 s = v[0];
#pragma unroll
                for (int q = 1; q < kMaxSplit; ++q)
                    if (q < a.split) {
                        s.x += v[q].x;
                        s.y += v[q].y;
                        s.z += v[q].z;
                        s.w += v[q].w;
                    }
                const uint2 o = make_uint2(pack_bf16x2(s.x * sc.x * sc.y, s.y * sc.x * sc.y),
                                           pack_bf16x2(s.z * sc.x * sc.y, s.w * sc.x * sc.y));
                uint16_t* y = a.y + (int64_t)b * a.y_bs + (int64_t)(t0 + c) * a.y_rs + n;
                if (a.y8 && n + 4 <= a.n) {
                    st_v2(y, o);
                } else {
                    if (n < a.n) y[0] = (uint16_t)o.x;
                    if (n + 1 < a.n) y[1] = (uint16_t)(o.x >> 16);
                    if (n + 2 < a.n) y[2] = (uint16_t)o.y;
                    if (n + 3 < a.n) y[3] = (uint16_t)(o.y >> 16);
                }
            }
        }
        __syncwarp();
        cluster_sync();   // no CTA leaves while its partial is being read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) tmem_free<1>(tmem, C::kCols);
}

// ---------------------------------------------------------------- many tokens: CTA pairs
//
// A pair of CTAs (two SMs, cta_group::2) takes 256 weight rows, 128 per CTA,
// times up to 256 tokens, half of whose codes each CTA loads: per 128-byte
// step of K an SM brings in 32 KB of codes for 512 tensor-core clocks, half
// of what one CTA alone would need for a 128 x 256 tile.  The kernel is
// persistent, one pair per two SMs, tiles in groups of kGroup token tiles so
// that the pairs at work share operands in L2.
//
// What bounds it.  In steady use, power: every sample under these products
// shows the 1000 W cap, with the SMs at 1.2 to 1.43 GHz (MXFP8 8192^3 1.21 GHz,
// NVFP4 4096 x 19456 x 2560 1.43), and what saves clocks without saving energy
// saves no time there.  8192^3 runs at 2.6 PFLOP/s sustained and 3.07 in six
// launches after a pause (MXFP8), 4.9 and 5.8 (NVFP4).  In clocks: a step of
// MXFP8 takes 512, its MMAs; one of NVFP4 takes 643 at 256 tokens, what issuing
// twelve scale copies beside four MMAs takes, and about 800 while the epilogue
// warp of the same scheduler is at work; a tile's start costs 660 and 1040 (its
// accumulator shares columns with the one before).  Issuing the copies from a
// warp of their own brought the NVFP4 step to 490 to 610 clocks: one launch
// alone 85 -> 76 us, eight in a row 84.3 -> 81.9, forty in a row 89.0 -> 92.6.
// The loads bound nothing: without them a step takes the same.
//
// Issue: the issuer tests the next step's barriers while it issues a step and
// waits only when the test failed (two waits at the start of each step made
// every step take 0.31 us even at 32 tokens, where it takes 0.07 us now).
//
// Tensor memory: 512 columns hold scale buffers of a step each (MXFP8 one per
// stage of the ring; NVFP4, 48 columns each, three, filled again once the
// step that read them has been seen to end: with two that wait cost 10 to 13 %
// of the step) and two accumulators, which overlap where two of 256 columns
// do not fit: the epilogue takes the shared columns into registers first and
// then lets the next tile begin.
//
// Output: 32 tokens at a time, TMEM fragments are transposed by stmatrix into
// [token][64 weight rows] boxes (128-byte swizzle, no bank conflicts) and
// stored by TMA, one warp pair per box.  Rows of y that are not 16-byte
// aligned, or whose length is no multiple of 8 (TMA would write the whole last
// 16 bytes), are stored from the boxes by the two warps, a word per lane:
// NVFP4 4096 x 19455 x 2560 took 144 us with an element per lane straight
// from TMEM, 126 now, and 81 without the stores (unaligned rows make two
// requests to L2 of each 128 bytes).
//
// The token tile is a multiple of 64 columns up to 256, or of 32 when one
// tile holds every token: the MMA takes scale columns two by two, so a tile
// starts at a multiple of 64 rows of a 128-row band (and its scales span at
// most two bands).  The host picks the one with the least work in the last wave.
//
// Warps 0..3 epilogue, 4 and 6 TMA producers (codes, scales), 5 MMA issuer
// (first CTA) and TMEM owner.  Launched in clusters of two.

constexpr int kPairThreads = 224;
constexpr uint32_t kGroup = 8;
constexpr int kOutTokens = 32;                                    // tokens per output store
constexpr uint32_t kOutBytes = 64u * kOutTokens * 2u;             // 64 weight rows x 32 tokens, BF16

struct PairArgs {
    CUtensorMap w, ws, t, ts, y;
    const float* gt;
    const float* gw;
    uint16_t* yp;                // y_tma == 0: rows that TMA does not take
    int64_t y_bs, y_rs;          // elements
    int y_tma;
    int n, m;
    int w_bands, t_bands;
    int steps, last_mmas;
    int tile_t, t_band_box;      // tokens per tile, scale bands per tile
    uint32_t stages, stage, scale_stage, out_at, scales_at;   // ring: stages, bytes of codes and of scales per stage
    uint32_t scale_bufs;         // scale buffers in TMEM
    uint32_t t_tiles, tiles;
    FastDiv per_batch, per_group;   // w_tiles * t_tiles, w_tiles * kGroup
};

constexpr int kMaxStages = 10;                                     // as many as ever fit (MXFP8, tiles of 32 tokens)
constexpr uint32_t kPairSmem = 232448u - 512u;   // dynamic shared memory of a CTA (the rest is static)

template <ProductFormat kF>
struct PairCfg {
    using T = ProductTraits<kF>;
    static constexpr uint32_t kW = 128u * kStepBytes;
    static constexpr uint32_t kOutBufs = T::kFp4 ? 4u : 3u;                   // output staging buffers per warp pair
    static constexpr uint32_t kScaleCols = 12u * T::kScaleTiles;              // per buffer: 4 weights + 8 tokens per tile
    // 32-column chunks that two accumulators of 256 columns share: with three buffers of 48 / six of 12
    static constexpr int kMaxShared = T::kFp4 ? 5 : 3;
};

struct PairTile {
    int wt, tt, b;
};
__device__ __forceinline__ PairTile pair_tile(const PairArgs& a, uint32_t i) {
    PairTile r;
    const uint32_t b = fdiv(i, a.per_batch);
    i -= b * a.per_batch.d;
    const uint32_t g = fdiv(i, a.per_group);
    i -= g * a.per_group.d;
    const uint32_t in_group = min(kGroup, a.t_tiles - g * kGroup);
    r.wt = (int)(i / in_group);
    r.tt = (int)(g * kGroup + i - (uint32_t)r.wt * in_group);
    r.b = (int)b;
    return r;
}

// Stores `rows` (up to 16) token rows of a box, from token 0 or 16 on, as rows
// of y that TMA does not take: 64 weight rows, `valid` of which exist.  A row
// is one 128-byte run: a lane stores the aligned word of two elements, and
// where the row starts in the middle of a word the first lane stores both ends.
__device__ __forceinline__ void store_rows(uint32_t box, int c, int rows, uint16_t* y, int64_t y_rs, int valid,
                                           int lane) {
    box += (uint32_t)c * 128u;
    auto word = [&](int r) {   // elements 2 lane and 2 lane + 1 of row r
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];"
                     : "=r"(v)
                     : "r"(box + r * 128u + ((((uint32_t)lane >> 2) ^ (r & 7u)) * 16u + ((uint32_t)lane & 3u) * 4u)));
        return v;
    };
    if (valid < 64 || rows < 16) {
        for (int r = 0; r < rows; ++r) {
            const uint32_t v = word(r);
            uint16_t* row = y + r * y_rs + 2 * lane;
            if (2 * lane < valid) row[0] = (uint16_t)v;
            if (2 * lane + 1 < valid) row[1] = (uint16_t)(v >> 16);
        }
        return;
    }
    char* at = reinterpret_cast<char*>(y) + 4 * lane;
    const int64_t pitch = 2 * y_rs;
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += 8) {
        uint32_t v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = word(r0 + r);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            // a row in the middle of a word: elements 2 lane - 1 and 2 lane; the first lane: 63 and 0
            char* row = at + (r0 + r) * pitch;
            const uint32_t odd = (uint32_t)(uintptr_t)row & 2u;
            const uint32_t w = __byte_perm(__shfl_sync(0xffffffffu, v[r], lane + 31), v[r], odd ? 0x5432 : 0x7654);
            asm volatile(
                "{\n\t.reg .pred ends;\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tsetp.ne.u32 ends, %2, 0;\n\t"
                "@!ends st.global.b32 [%0], %1;\n\t@ends st.global.b16 [%0 + 2], hi;\n\t"
                "@ends st.global.b16 [%0 + 128], lo;\n\t}"
                :: "l"(row - odd), "r"(w), "r"(lane == 0 ? odd : 0u) : "memory");
        }
    }
}

template <ProductFormat kF>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ PairArgs a) {
    using T = ProductTraits<kF>;
    using C = PairCfg<kF>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 4];
    __shared__ uint32_t tmem_word;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u, scales = ring + a.scales_at;
    const uint32_t full = smem_addr(bars), empty = full + 8u * kMaxStages;
    const uint32_t acc_full = empty + 8u * kMaxStages, acc_free = acc_full + 16u;   // [2] each
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;
    // the second accumulator's column, and the 32-column chunks that the two share
    const uint32_t scale_at = 512u - a.scale_bufs * C::kScaleCols;
    const uint32_t acc1 = min((uint32_t)a.tile_t, (scale_at - (uint32_t)a.tile_t) / 32u * 32u);
    const int shared = (a.tile_t - (int)acc1) / 32;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < a.stages; ++i) {
            mbar_init(full + 8u * i, 1);
            mbar_init(empty + 8u * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8u * i, 1);
            mbar_init(acc_free + 8u * i, 8);   // four epilogue warps of either CTA
        }
        fence_mbar_init();
    }
    if (warp == 4 && elect_one()) {
        prefetch_tensor_map(&a.w);
        prefetch_tensor_map(&a.t);
        prefetch_tensor_map(&a.ws);
        prefetch_tensor_map(&a.ts);
    }
    if (warp == 5) tmem_alloc<2>(smem_addr(&tmem_word), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    let_later_kernels_start();
    wait_for_earlier_kernels();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_word, 0);

    if (warp == 4 || warp == 6) {
        const bool codes = warp == 4;   // the other one loads the scales
        const uint32_t tok_bytes = (uint32_t)a.tile_t / 2u * kStepBytes;
        const uint32_t bytes = C::kW + tok_bytes + (1u + (uint32_t)a.t_band_box) * T::kScaleBytes;
        RingPos pos;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t i = first; ok && i < a.tiles; i += stride) {
            const PairTile p = pair_tile(a, i);
            const int wt = p.wt * 2 + (int)rank, t0 = p.tt * a.tile_t;
            const int w_band = p.b * a.w_bands + wt, t_band = p.b * a.t_bands + t0 / 128;
            const int w_row = wt * 128, t_row = t0 + (int)rank * (a.tile_t / 2);
            for (int s = 0; s < a.steps; ++s) {
                const uint32_t st = pos.at, bar = cluster_addr(full + 8u * st, 0);
                if (!warp_wait(empty + 8u * st, pos.phase ^ 1u)) {   // passes at once on the first lap
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (codes) {
                        const uint32_t at = ring + st * a.stage;
                        if (rank == 0) mbar_arrive_expect_tx(full + 8u * st, 2u * bytes);
                        tma_load_3d_pair(at, &a.w, bar, s * (int)kStepBytes, w_row, p.b);
                        tma_load_3d_pair(at + C::kW, &a.t, bar, s * (int)kStepBytes, t_row, p.b);
                    } else {
                        const uint32_t sc = scales + st * a.scale_stage;
                        tma_load_3d_pair(sc, &a.ws, bar, 0, s * T::kScaleTiles, w_band);
                        tma_load_3d_pair(sc + T::kScaleBytes, &a.ts, bar, 0, s * T::kScaleTiles, t_band);
                    }
                }
                __syncwarp();
                pos.next(a.stages);
                ++issued;
            }
        }
        // no copy of either CTA is in flight when the pair ends: the stages' last uses, oldest first
        if (rank == 0 && codes) {
            const uint32_t end = pos.at;
            for (uint32_t j = 0; j < a.stages; ++j) {
                const bool last_lap = j < a.stages - end;   // used on the lap before, if there was one
                if ((!last_lap || issued >= a.stages) && !warp_wait(full + 8u * pos.at, pos.phase ^ 1u)) break;
                pos.next(a.stages);
            }
        }
    } else if (warp == 5) {
        if (rank == 0) {
            const uint32_t idesc = mma_idesc<kF>(256, a.tile_t);
            // NVFP4: three scale buffers, each free again when the step three before has ended (`old`).  MXFP8: a
            // buffer for each stage, free with it.
            RingPos pos, old;
            uint32_t it = 0, n = 0, sbuf = 0;
            bool ok = true, ready = false;
            const bool leader = elect_one();
            for (uint32_t i = first; ok && i < a.tiles; i += stride, ++n) {
                const PairTile p = pair_tile(a, i);
                const uint32_t buf = n & 1u, acc = tmem + buf * acc1;
                const uint32_t tok_col = (uint32_t)(p.tt * a.tile_t % 128) / 32u;
                // the accumulator is free: with shared columns, once the previous tile's have been read;
                // without, once the tile before that has been read
                if (shared > 0 && n >= 1) ok = warp_wait(acc_free + 8u * (buf ^ 1u), ((n - 1u) / 2u) & 1u);
                if (shared == 0 && n >= 2) ok = warp_wait(acc_free + 8u * buf, (n / 2u - 1u) & 1u);
                if (!ok) break;
                for (int s = 0; s < a.steps; ++s) {
                    const uint32_t st = pos.at;
                    // `ready`: the barriers were tested while the last step was issued
                    if (!__all_sync(0xffffffffu, ready)) {
                        ok = warp_wait(full + 8u * st, pos.phase);
                        if (T::kFp4 && ok && it >= 3u) ok = warp_wait(empty + 8u * old.at, old.phase);
                        if (!ok) break;
                    }
                    if (T::kFp4 && it >= 3u) old.next(a.stages);
                    tc_fence_after();
                    const uint32_t at = ring + st * a.stage, sc = scales + st * a.scale_stage;
                    const uint32_t sw = tmem + scale_at + (T::kFp4 ? sbuf : st) * C::kScaleCols;
                    const uint64_t dw = desc_swizzle128(at), dx = desc_swizzle128(at + C::kW);
                    const int mmas = s == a.steps - 1 ? a.last_mmas : kMmasPerStep;
                    if (leader) {
#pragma unroll
                        for (int j = 0; j < kMmasPerStep; ++j) {
                            if (j >= mmas) break;
                            const int tile = T::kFp4 ? j : 0;   // scale tile of the step: 4 + 8 columns
                            const uint32_t cw = sw + 12u * tile, cx = cw + 4u;
                            if (T::kFp4 || j == 0) {
                                copy_scales<2>(cw, desc_scales(sc + 512u * tile));
                                copy_scales<2>(cx, desc_scales(sc + T::kScaleBytes + 512u * tile));
                                if (a.t_band_box == 2)
                                    copy_scales<2>(cx + 4u, desc_scales(sc + 2u * T::kScaleBytes + 512u * tile));
                            }
                            const uint32_t id = T::kFp4 ? idesc : idesc | (uint32_t)j << 4 | (uint32_t)j << 29;
                            mma_block_scaled<kF, 2>(acc, dw + 2u * j, dx + 2u * j, id, cw, cx + tok_col, (s | j) != 0);
                        }
                    }
                    ++it;
                    if (++sbuf == 3u) sbuf = 0u;
                    pos.next(a.stages);
                    const bool operands = mbar_test(full + 8u * pos.at, pos.phase);
                    const bool buffer = !T::kFp4 || it < 3u || mbar_test(empty + 8u * old.at, old.phase);
                    if (leader) mma_commit_pair(empty + 8u * st);
                    ready = operands && buffer;
                }
                if (elect_one()) mma_commit_pair(acc_full + 8u * buf);
                __syncwarp();
            }
        }
    } else {
        uint32_t n = 0, stores = 0;
        const uint32_t row = tmem + ((uint32_t)warp << 21);
        const uint32_t out = ring + a.out_at + (uint32_t)(warp >> 1) * C::kOutBufs * kOutBytes;
        // this lane's stmatrix row: token lane % 8 of eight, weight rows 8 (lane / 8) .. + 7 of the warp's 32
        const uint32_t c8 = (uint32_t)lane & 7u;
        const uint32_t frag = c8 * 128u + (((uint32_t)(warp & 1) * 4u + ((uint32_t)lane >> 3)) ^ c8) * 16u;
        for (uint32_t i = first; i < a.tiles; i += stride, ++n) {
            const PairTile p = pair_tile(a, i);
            const uint32_t buf = n & 1u, acc = row + buf * acc1, free_bar = cluster_addr(acc_free + 8u * buf, 0);
            const int n0 = (p.wt * 2 + (int)rank) * 128, t0 = p.tt * a.tile_t, chunks = a.tile_t / 32;
            const float2 sc = output_scale(a.gt, a.gw, p.b);
            const int x = n0 + (warp >> 1) * 64;   // the warp pair's 64 weight rows
            // shared columns first: the first buffer's last ones, the second buffer's first ones
            auto column = [&](int k) { return 32 * (buf == 0 ? chunks - 1 - k : k); };
            auto load = [&](int k, uint32_t (&v)[32]) {
                tmem_ld_frag32(acc + column(k), v);
                tmem_ld_frag32(acc + (16u << 16) + column(k), v + 16);
            };
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(free_bar);
            };
            auto store = [&](int k, const uint32_t (&v)[32]) {
                const int t = t0 + column(k);
                if (t >= a.m || n0 >= a.n) return;   // the same for the CTA
                // the buffer was seen free before the previous store's barrier (or is new)
                const uint32_t box = out + stores % C::kOutBufs * kOutBytes, dst = box + frag;
                ++stores;
#pragma unroll
                for (int r = 0; r < 4; ++r) {   // eight tokens
                    uint32_t h[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int e = 16 * (g >> 1) + 4 * r + 2 * (g & 1);
                        h[g] = pack_bf16x2(scaled<kF>(v[e], sc), scaled<kF>(v[e + 1], sc));
                    }
                    stmatrix_trans(dst + r * 1024u, h[0], h[1], h[2], h[3]);
                }
                const bool first_warp = (warp & 1) == 0;   // of the pair: its elected lane issues
                if (a.y_tma) {
                    fence_async_shared();
                    if (first_warp && elect_one()) bulk_wait_read<C::kOutBufs - 2>();   // the next buffer has been read
                }
                __syncwarp();
                asm volatile("bar.sync %0, 64;" :: "r"(2 + (warp >> 1)) : "memory");
                if (a.y_tma) {
                    if (first_warp && x < a.n && elect_one()) {
                        tma_store_3d(&a.y, box, x, t, p.b);
                        bulk_commit();
                    }
                } else {
                    const int c0 = (warp & 1) * 16, valid = min(64, a.n - x), rows = min(16, a.m - t - c0);
                    uint16_t* yp = a.yp + (int64_t)p.b * a.y_bs + x + (int64_t)(t + c0) * a.y_rs;
                    store_rows(box, c0, rows, yp, a.y_rs, valid, lane);
                }
                __syncwarp();
            };
            // the first warp polls for the four, which go on or leave together
            if (!vote_all(warp != 0 || warp_wait(acc_full + 8u * buf, (n / 2u) & 1u))) break;
            tc_fence_after();
            if (shared > 0) {
                uint32_t held[C::kMaxShared][32];
#pragma unroll
                for (int k = 0; k < C::kMaxShared; ++k)
                    if (k < shared) load(k, held[k]);
                tmem_ld_wait();
                release();
#pragma unroll
                for (int k = 0; k < C::kMaxShared; ++k)
                    if (k < shared) store(k, held[k]);
            }
            for (int k = shared; k < chunks; ++k) {
                uint32_t v[32];
                load(k, v);
                tmem_ld_wait();
                if (shared == 0 && k == chunks - 1) release();
                store(k, v);
            }
        }
        if ((warp & 1) == 0 && elect_one()) bulk_wait<0>();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs are done with TMEM, barriers and operands
    if (warp == 5) tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------- host side

// Code rows [batch][rows][bytes] as a 3-D map of 128-byte wide boxes, 128-byte swizzle.
bool code_map(EncodeTiledFn encode, CUtensorMap* map, const View& v, int64_t row_bytes, uint32_t box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)row_bytes, (cuuint64_t)v.rows, (cuuint64_t)v.batch};
    const cuuint64_t strides[2] = {(cuuint64_t)v.rstride,
                                   (cuuint64_t)(v.batch > 1 ? v.bstride : v.rows * v.rstride)};
    const cuuint32_t box[3] = {kStepBytes, box_rows, 1}, es[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, v.ptr, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile-layout scales as [band][column tile][128 words]: a box is `tiles`
// consecutive 512-byte tiles of `bands` bands; tiles past the last column read as zero.
bool scale_map(EncodeTiledFn encode, CUtensorMap* map, const uint8_t* scales, int64_t bands, int64_t col_tiles,
               uint32_t tiles, uint32_t box_bands) {
    const cuuint64_t dims[3] = {128, (cuuint64_t)col_tiles, (cuuint64_t)bands};
    const cuuint64_t strides[2] = {512, (cuuint64_t)(col_tiles * 512)};
    const cuuint32_t box[3] = {128, tiles, box_bands}, es[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <ProductFormat kF, int kTok>
cudaError_t launch_tokens(const Product& p, EncodeTiledFn encode, cudaStream_t s) {
    using T = ProductTraits<kF>;
    using C = TokCfg<kF, kTok>;
    static int configured[kMaxDevices] = {0};
    const void* fn = (const void*)tokens_kernel<kF, kTok>;
    cudaError_t e = set_smem_limit_once(configured, &fn, 1, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t row_bytes = T::kFp4 ? p.k / 2 : p.k;
    const int64_t col_tiles = mma_scale_col_tiles(p.k / (T::kFp4 ? 16 : 32));
    const int64_t w_tiles = (p.w.rows + 127) / 128, t_tiles = (p.a.rows + kTok - 1) / kTok;
    const int64_t tiles = p.a.batch * w_tiles * t_tiles;
    TokArgs a;
    a.w_bands = (int)w_tiles;
    a.t_bands = (int)((p.a.rows + 127) / 128);
    if (!code_map(encode, &a.w, p.w, row_bytes, 128) || !code_map(encode, &a.t, p.a, row_bytes, kTok) ||
        !scale_map(encode, &a.ws, p.w_scale, p.a.batch * a.w_bands, col_tiles, T::kScaleTiles, 1) ||
        !scale_map(encode, &a.ts, p.a_scale, p.a.batch * a.t_bands, col_tiles, T::kScaleTiles, 1))
        return cudaErrorInvalidValue;
    a.gt = p.a_gs;
    a.gw = p.w_gs;
    a.y = reinterpret_cast<uint16_t*>(p.y.ptr);
    a.y_bs = p.y.bstride / 2;
    a.y_rs = p.y.rstride / 2;
    a.y8 = (uintptr_t)p.y.ptr % 8 == 0 && p.y.rstride % 8 == 0 && (p.y.batch == 1 || p.y.bstride % 8 == 0);
    a.n = (int)p.w.rows;
    a.m = (int)p.a.rows;
    a.steps = (int)((row_bytes + kStepBytes - 1) / kStepBytes);
    a.last_mmas = (int)((row_bytes - (int64_t)(a.steps - 1) * kStepBytes + 31) / 32);
    a.w_tiles = make_fastdiv((uint32_t)w_tiles);
    a.t_tiles = make_fastdiv((uint32_t)t_tiles);
    // Split K while the CTAs stay within 4/3 of the SMs and keep 2.5 steps each: at 4096 x 2560 and one token,
    // 32 tiles in 128 CTAs take 4.9 us (MXFP8), in 256 CTAs 6.2 us; NVFP4 2560 x 4096 in 4 parts of 4 steps
    // 5.1 us, in 8 of 2 steps 5.9 us.
    const int64_t sms = sm_count(current_device()), limit = sms + sms / 3;
    a.split = 1;
    while (a.split < kMaxSplit && tiles * a.split * 2 <= limit && a.split * 2 * 5 <= a.steps * 2) a.split *= 2;
    if (tiles * a.split > (int64_t)0x7fffffff) return cudaErrorInvalidValue;
    return launch_early(tokens_kernel<kF, kTok>, (unsigned)(tiles * a.split), kTokThreads, C::kSmem, s,
                        (unsigned)a.split, a);
}

// Tokens per tile of the pair kernel: the fewest (waves of tiles) x (time of
// a tile).  A step takes about as long as the bytes that it brings in (256
// weight rows, the tile's tokens, scales worth 24 rows): measured, for 256 /
// 192 / 128 / 64 tokens, 0.44 / 0.34 / 0.29 / 0.26 us in NVFP4 and 0.51 / 0.31 /
// 0.27 / 0.24 in MXFP8 (9472 tokens, 4096 weight rows; at 256 the power cap
// slows MXFP8).  A tile's start and the part of its epilogue that nothing hides
// take 1.1 us in NVFP4, 0.3 to 0.8 in MXFP8: about two steps.
int pair_tile_tokens(int64_t m, int64_t w_tiles, int64_t batch, int64_t pairs, int64_t steps) {
    int best = 256;
    int64_t best_cost = -1;
    for (int t = 256; t >= 32; t -= 32) {
        if (t % 64 != 0 && m > t) continue;
        const int64_t tiles = batch * w_tiles * ((m + t - 1) / t);
        const int64_t cost = (tiles + pairs - 1) / pairs * (steps * (256 + t + 24) + 1000);
        if (best_cost < 0 || cost < best_cost) {
            best = t;
            best_cost = cost;
        }
    }
    return best;
}

template <ProductFormat kF>
cudaError_t launch_pairs(const Product& p, EncodeTiledFn encode, cudaStream_t s) {
    using T = ProductTraits<kF>;
    using C = PairCfg<kF>;
    static int configured[kMaxDevices] = {0};
    const void* fn = (const void*)pair_kernel<kF>;
    cudaError_t e = set_smem_limit_once(configured, &fn, 1, (int)kPairSmem);
    if (e != cudaSuccess) return e;
    const int64_t row_bytes = T::kFp4 ? p.k / 2 : p.k;
    const int64_t col_tiles = mma_scale_col_tiles(p.k / (T::kFp4 ? 16 : 32));
    const int64_t pairs = sm_count(current_device()) / 2, w_tiles = (p.w.rows + 255) / 256;
    PairArgs a;
    a.steps = (int)((row_bytes + kStepBytes - 1) / kStepBytes);
    a.tile_t = pair_tile_tokens(p.a.rows, w_tiles, p.a.batch, pairs, a.steps);
    a.t_band_box = 128 % a.tile_t == 0 ? 1 : 2;
    const int64_t t_tiles = (p.a.rows + a.tile_t - 1) / a.tile_t;
    a.w_bands = (int)((p.w.rows + 127) / 128);
    a.t_bands = (int)((p.a.rows + 127) / 128);
    if (!code_map(encode, &a.w, p.w, row_bytes, 128) ||
        !code_map(encode, &a.t, p.a, row_bytes, (uint32_t)a.tile_t / 2) ||
        !scale_map(encode, &a.ws, p.w_scale, p.a.batch * a.w_bands, col_tiles, T::kScaleTiles, 1) ||
        !scale_map(encode, &a.ts, p.a_scale, p.a.batch * a.t_bands, col_tiles, T::kScaleTiles,
                   (uint32_t)a.t_band_box))
        return cudaErrorInvalidValue;
    // output by TMA where its rows are whole 16-byte units at 16-byte addresses (a store that ends inside a
    // unit overwrites the rest of it), else by the epilogue's warps
    a.y_tma = p.y.cols % 8 == 0 && (uintptr_t)p.y.ptr % 16 == 0 && p.y.rstride % 16 == 0 &&
              (p.y.batch == 1 || p.y.bstride % 16 == 0);
    if (a.y_tma) {
        const cuuint64_t dims[3] = {(cuuint64_t)p.y.cols, (cuuint64_t)p.y.rows, (cuuint64_t)p.y.batch};
        const cuuint64_t strides[2] = {(cuuint64_t)p.y.rstride,
                                       (cuuint64_t)(p.y.batch > 1 ? p.y.bstride : p.y.rows * p.y.rstride)};
        const cuuint32_t box[3] = {64, kOutTokens, 1}, es[3] = {1, 1, 1};
        if (encode(&a.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.y.ptr, dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    a.gt = p.a_gs;
    a.gw = p.w_gs;
    a.yp = reinterpret_cast<uint16_t*>(p.y.ptr);
    a.y_bs = p.y.bstride / 2;
    a.y_rs = p.y.rstride / 2;
    a.n = (int)p.w.rows;
    a.m = (int)p.a.rows;
    a.last_mmas = (int)((row_bytes - (int64_t)(a.steps - 1) * kStepBytes + 31) / 32);
    a.t_tiles = (uint32_t)t_tiles;
    a.tiles = (uint32_t)(p.a.batch * w_tiles * t_tiles);
    a.per_batch = make_fastdiv((uint32_t)(w_tiles * t_tiles));
    a.per_group = make_fastdiv((uint32_t)w_tiles * kGroup);
    // as many stages as fit: few tokens leave room for more weight rows in flight
    a.stage = (C::kW + (uint32_t)a.tile_t / 2u * kStepBytes + 1023u) / 1024u * 1024u;
    a.scale_stage = (1u + (uint32_t)a.t_band_box) * T::kScaleBytes;
    const uint32_t out = 2u * C::kOutBufs * kOutBytes;
    a.stages = std::min<uint32_t>(kMaxStages, (kPairSmem - 1024u - out) / (a.stage + a.scale_stage));
    a.scale_bufs = T::kFp4 ? 3u : a.stages;
    a.out_at = a.stages * a.stage;
    a.scales_at = a.out_at + out;
    const unsigned grid = 2u * (unsigned)std::min<int64_t>(a.tiles, pairs);
    return launch_early(pair_kernel<kF>, grid, kPairThreads, 1024u + a.scales_at + a.stages * a.scale_stage, s, 2u, a);
}

template <ProductFormat kF>
cudaError_t launch_product(const Product& p, cudaStream_t s) {
    EncodeTiledFn encode = encode_tiled_fn();
    if (!encode) return cudaErrorNotSupported;
    const int64_t m = p.a.rows, w_tiles = (p.w.rows + 255) / 256, pairs = sm_count(current_device()) / 2;
    const int64_t steps = ((kF == ProductFormat::kNvfp4 ? p.k / 2 : p.k) + kStepBytes - 1) / kStepBytes;
    if (m <= 64) {
        // One token tile.  The pairs win where they are at least 60 % busy (128 x 1536 x 2048 at 64 tokens:
        // NVFP4 47 against 62 us, MXFP8 78 against 81), else the finer tiles and the split K of the token
        // kernel do (19456 x 2560, 76 tiles on 74 pairs: NVFP4 8.5 against 11.2 us at one token).
        const int64_t tiles = p.a.batch * w_tiles, waves = (tiles + pairs - 1) / pairs;
        if (5 * tiles >= 3 * waves * pairs) return launch_pairs<kF>(p, encode, s);
        // tokens per tile: the smallest MMA width that holds them all
        if (m <= 16) return launch_tokens<kF, 16>(p, encode, s);
        if (m <= 32) return launch_tokens<kF, 32>(p, encode, s);
        return launch_tokens<kF, 64>(p, encode, s);
    }
    // A few more tokens against few weight rows and a long K: at most 20 pairs would work (2560 x 9728,
    // MXFP8: 128 tokens 12.7 against 22.6 us, 256 tokens 16.3 against 22.8; 2560 x 4096, NVFP4, 256 tokens the
    // pairs win, 8.8 against 10.4).
    if (p.a.batch * w_tiles <= 20) {
        if (m <= 128 && steps >= 16) return launch_tokens<kF, 64>(p, encode, s);
        if (m <= 256 && steps >= 32) return launch_tokens<kF, 128>(p, encode, s);
    }
    return launch_pairs<kF>(p, encode, s);
}

}  // namespace

cudaError_t launch_mxfp8_matmul(const Product& p, cudaStream_t s) {
    return launch_product<ProductFormat::kMxfp8>(p, s);
}
cudaError_t launch_nvfp4_matmul(const Product& p, cudaStream_t s) {
    return launch_product<ProductFormat::kNvfp4>(p, s);
}

cudaError_t read_and_clear_matmul_error(uint32_t* code) {
    uint32_t zero = 0u;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_matmul_error, sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_matmul_error, &zero, sizeof(uint32_t));
}

}  // namespace pwq
