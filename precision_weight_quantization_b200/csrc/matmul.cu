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

// ga * gw as a product of two FP32 factors, so that neither the scale nor a
// partial product leaves the FP32 range when the result does not: one factor
// is 1 unless the product of the scales is outside [2^-100, 2^100].
__device__ __forceinline__ float2 output_scale(const float* ga, const float* gw, int b) {
    if (!ga) return make_float2(1.0f, 1.0f);
    const double p = (double)ga[b] * (double)gw[b];
    if (p < 0x1p-100 && p > 0.0) return make_float2(0x1p-100f, (float)(p * 0x1p100));
    if (p > 0x1p100 && p < 0x1p1000) return make_float2(0x1p100f, (float)(p * 0x1p-100));
    return make_float2((float)p, 1.0f);
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
// Warps 0..3 epilogue, 4 TMA producer, 5 MMA issuer and TMEM owner.

constexpr int kTokThreads = 192;

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
    FastDiv w_tiles, t_tiles;
};

template <ProductFormat kF, int kTok>
struct TokCfg {
    using T = ProductTraits<kF>;
    static constexpr uint32_t kW = 128u * kStepBytes, kT = (uint32_t)kTok * kStepBytes;
    static constexpr uint32_t kStage = kW + kT + 2u * T::kScaleBytes;
    static constexpr int kStages = kTok <= 64 ? 4 : 3;
    static constexpr uint32_t kSmem = kStages * kStage + 1024u;   // + alignment of the ring to 1024 bytes
    // TMEM: kTok accumulator columns, then two buffers of weight and token scale columns
    static constexpr uint32_t kScaleCols = 4u * T::kScaleTiles;
    static constexpr uint32_t kCols = kTok + 4u * kScaleCols <= 128u ? 128u : 256u;
    static_assert(kTok + 4u * kScaleCols <= kCols, "TMEM");
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    if (warp == 5) tmem_alloc<1>(smem_addr(&tmem_word), C::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_word;

    if (warp == 4) {
        if (lane == 0) {
            int i = 0;
            for (; i < steps; ++i) {
                const int st = i % kS;
                if (i >= kS && !wait_or_record(empty + 8u * st, ((i / kS) - 1) & 1)) break;
                const uint32_t at = ring + (uint32_t)st * C::kStage, bar = full + 8u * st;
                mbar_arrive_expect_tx(bar, C::kStage);
                const int s = s0 + i;
                tma_load_3d(at, &a.w, bar, s * (int)kStepBytes, n0, b);
                tma_load_3d(at + C::kW, &a.t, bar, s * (int)kStepBytes, t0, b);
                tma_load_3d(at + C::kW + C::kT, &a.ws, bar, 0, s * T::kScaleTiles, b * a.w_bands + wt);
                tma_load_3d(at + C::kW + C::kT + T::kScaleBytes, &a.ts, bar, 0, s * T::kScaleTiles,
                            b * a.t_bands + t0 / 128);
            }
            // no copy is in flight when the CTA ends
            for (int j = max(0, i - kS); j < i; ++j) wait_or_record(full + 8u * (j % kS), (j / kS) & 1);
        }
    } else if (warp == 5) {
        if (lane == 0) {
            constexpr uint32_t idesc = mma_idesc<kF>(128, kTok);
            for (int i = 0; i < steps; ++i) {
                const int st = i % kS;
                if (!wait_or_record(full + 8u * st, (i / kS) & 1)) break;
                // the scale columns of step i - 2 are read no more
                if (i >= 2 && !wait_or_record(empty + 8u * ((i - 2) % kS), ((i - 2) / kS) & 1)) break;
                tc_fence_after();
                const uint32_t at = ring + (uint32_t)st * C::kStage;
                const uint32_t sw = tmem + kTok + (uint32_t)(i & 1) * 2u * C::kScaleCols, sx = sw + C::kScaleCols;
#pragma unroll
                for (int j = 0; j < T::kScaleTiles; ++j) {
                    copy_scales<1>(sw + 4u * j, desc_scales(at + C::kW + C::kT + 512u * j));
                    copy_scales<1>(sx + 4u * j, desc_scales(at + C::kW + C::kT + T::kScaleBytes + 512u * j));
                }
                const uint64_t dw = desc_swizzle128(at), dx = desc_swizzle128(at + C::kW);
                const int mmas = s0 + i == a.steps - 1 ? a.last_mmas : kMmasPerStep;
                for (int j = 0; j < mmas; ++j) {
                    const uint32_t id = T::kFp4 ? idesc : idesc | (uint32_t)j << 4 | (uint32_t)j << 29;
                    const uint32_t so = T::kFp4 ? 4u * j : 0u;
                    mma_block_scaled<kF, 1>(tmem, dw + 2u * j, dx + 2u * j, id, sw + so, sx + so, (i | j) != 0);
                }
                mma_commit(empty + 8u * st);
            }
            mma_commit(done);
        }
    } else {
        const bool ok = wait_or_record(done, 0);
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
            if (steps == 0 || !ok) {
#pragma unroll
                for (int c = 0; c < kChunk; ++c) v[c] = 0u;
            }
            if (a.split == 1) {
#pragma unroll
                for (int c = 0; c < kChunk; ++c) {
                    const int t = t0 + c0 + c;
                    if (t < a.m && n < a.n)
                        y[(int64_t)t * a.y_rs] = bf16_bits(__uint_as_float(v[c]) * sc.x * sc.y);
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
            const float2 sc = output_scale(a.gt, a.gw, b);
            const int n = n0 + (int)threadIdx.x;
            uint16_t* y = a.y + (int64_t)b * a.y_bs + n;
            for (int c = (int)rank; c < kTok && t0 + c < a.m; c += a.split) {
                float sum = 0.0f;
                for (int q = 0; q < a.split; ++q)
                    sum += ld_cluster_f32(cluster_addr(ring + ((uint32_t)c * 128u + threadIdx.x) * 4u, (uint32_t)q));
                if (n < a.n) y[(int64_t)(t0 + c) * a.y_rs] = bf16_bits(sum * sc.x * sc.y);
            }
        }
        __syncwarp();
        cluster_sync();   // no CTA leaves while its partial is being read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) tmem_free<1>(tmem, C::kCols);
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
    a.n = (int)p.w.rows;
    a.m = (int)p.a.rows;
    a.steps = (int)((row_bytes + kStepBytes - 1) / kStepBytes);
    a.last_mmas = (int)((row_bytes - (int64_t)(a.steps - 1) * kStepBytes + 31) / 32);
    a.w_tiles = make_fastdiv((uint32_t)w_tiles);
    a.t_tiles = make_fastdiv((uint32_t)t_tiles);
    // split K while the tiles leave half of the resident CTA slots (two per SM) empty
    const int64_t slots = 2 * (int64_t)sm_count(current_device());
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= slots && a.split * 2 <= a.steps) a.split *= 2;
    if (tiles * a.split > (int64_t)0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.split));
    cfg.blockDim = dim3(kTokThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tokens_kernel<kF, kTok>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <ProductFormat kF>
cudaError_t launch_product(const Product& p, cudaStream_t s) {
    EncodeTiledFn encode = encode_tiled_fn();
    if (!encode) return cudaErrorNotSupported;
    // tokens per tile: the smallest MMA width that holds them all, at most 128
    if (p.a.rows <= 16) return launch_tokens<kF, 16>(p, encode, s);
    if (p.a.rows <= 32) return launch_tokens<kF, 32>(p, encode, s);
    if (p.a.rows <= 64) return launch_tokens<kF, 64>(p, encode, s);
    return launch_tokens<kF, 128>(p, encode, s);
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
