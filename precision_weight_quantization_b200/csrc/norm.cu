// norm.cu -- root-mean-square norm with the residual's addition and a
// block-scaled output, forward and backward: the step in front of every
// quantised linear layer of the rollout and of quantisation-aware training
// ("Low Precision RL", "Modes" 3 and 4; verl NVFP4 QAT article 2.2, 2.3).
//
//   h = bf16(fl(x + residual))                     (h = x without a residual)
//   rstd = (sum_d h_d^2 / D + eps)^(-1/2)
//   y = bf16(h rstd weight)                        (one rounding)
//
// and the output is MXFP8 or NVFP4 (amax given) of y, bit for bit what
// mxfp8_quant / nvfp4_quant write for that y, or its dequantised BF16 value.
// One launch reads x and the residual once and writes h and the codes once;
// y never reaches memory.
//
// y is the BF16 nearest to the exact product, so that codes do not depend on
// the order of a sum.  The squares are summed in 64 bits.  With rstd = m 2^E,
// h 2^E is exact, (h 2^E) weight is exact (8 + 8 significant bits), and the
// one FP32 rounding of its product with m is off by less than two units; so
// only a product within two units of a BF16 tie (5 in 65536) is formed again
// in 64 bits.  The kernel is bound by HBM when it issues fewer than about 20
// instructions per element: hence the packed additions and products, and the
// tie test on eight low halves at once.
#include <algorithm>

#include "pwq_early.cuh"
#include "pwq_internal.h"

namespace pwq {
namespace {

enum class NormOut { kMxfp8, kNvfp4, kMxfp8Fake, kNvfp4Fake };

struct NormArgs {
    View x, res, h, out;         // res.ptr / h.ptr null without a residual
    const uint4* weight;
    double eps, d, inv_d;        // D and its reciprocal
    const float* amax;           // NVFP4: [batch]
    float* gs;                   // NVFP4 codes: [batch]
    uint8_t* scale;              // codes: block scales
    float* rstd;                 // [batch * rows] or null
    FastDiv rows;                // rows per batch slab
    uint32_t total_rows;
    int vecs;                    // D / 8
    int s_cols;                  // scale columns per row
    int sf_mma;                  // tile layout
    uint32_t sf_ct;
    int64_t sf_slab;
    uint32_t row_ctas, pad_rows; // CTAs that own rows; padding rows of the tile layout per slab
    uint64_t pad_words;          // 4-byte words of those rows over all slabs
};

// bf16(x + residual) of BF16 pairs in one rounding.  (The same value as the
// FP32 sum rounded to BF16: an FP32 sum of two BF16 is exact, or its smaller
// term is too small to reach a tie.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint4 add_bf16(uint4 a, uint4 b) {
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

// The sum of the squares of 8 elements, as two chains (a chain of 64-bit
// additions over a thread's 32 elements would take longer than its loads).
__device__ __forceinline__ double squares(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double lo = 0.0, hi = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = (double)bf16_lo(w[i]), b = (double)bf16_hi(w[i]);
        lo = __fma_rn(a, a, lo);
        hi = __fma_rn(b, b, hi);
    }
    return lo + hi;
}

// A 64-bit value as FP32 that rounds to the same BF16: the nearest FP32,
// moved off a BF16 tie towards the value where it is not the value itself.
__device__ __forceinline__ float narrow_for_bf16(float h, float w, double rstd) {
    const double t = __dmul_rn((double)h * (double)w, rstd);
    const float f = __double2float_rn(t);
    const double back = (double)f;
    if ((__float_as_uint(f) & 0xffffu) != 0x8000u || back == t) return f;
    return __uint_as_float(__float_as_uint(f) + (fabs(t) > fabs(back) ? 1u : 0xffffffffu));
}

// s / D from the correctly rounded reciprocal rd of D: a product and one
// residual correction (Markstein, as div_fast), exact when the quotient is.
__device__ __forceinline__ double mean_of(double s, double d, double rd) {
    const double q = __dmul_rn(s, rd);
    return __fma_rn(__fma_rn(-q, d, s), rd, q);
}

// v^(-1/2) to 64-bit accuracy for v in [1e-16, 1e80]: v = m 4^k with m in
// [1, 4), the FP32 rsqrtf of m (error e0 below 2^-20), and one step of
// Householder's third-order iteration for x^(-1/2), y (1 + e / 2 + 3 e^2 / 8)
// with e = 1 - m y^2, whose error is of the order e0^3.  A power of four
// gives its root exactly.  (IEEE square root and division take about 200
// instructions in every thread, a third of the kernel's.)
__device__ __forceinline__ double inverse_sqrt(double v) {
    const int hi = __double2hiint(v), k2 = ((hi >> 20) - 1023) & ~1;
    const double m = __hiloint2double(hi - (k2 << 20), __double2loint(v));
    const double y = (double)rsqrtf((float)m);
    const double e = __fma_rn(-__dmul_rn(m, y), y, 1.0);
    const double r = __fma_rn(__dmul_rn(y, e), __fma_rn(e, 0.375, 0.5), y);
    return __hiloint2double(__double2hiint(r) - ((k2 / 2) << 20), __double2loint(r));
}

// The row's rstd from its sum of squares.  inverse_sqrt works on exponent bits,
// so a sum that is not finite is answered here: infinite (h holds an infinity,
// perhaps of a sum x + residual that overflowed) gives 0, NaN gives NaN.  Two
// selects beside the chain, no branch: one row of 2560 takes 2.0 us, 2.3 with one.
__device__ __forceinline__ double rstd_of(double sum, double d, double inv_d, double eps) {
    const double r = inverse_sqrt(mean_of(sum, d, inv_d) + eps);
    const uint32_t hi = (uint32_t)__double2hiint(sum);
    const bool finite = hi < 0x7ff00000u, inf = hi == 0x7ff00000u && __double2loint(sum) == 0;
    return __hiloint2double(finite ? __double2hiint(r) : inf ? 0 : 0x7ff80000, finite ? __double2loint(r) : 0);
}

// The row's rstd for normalise(): hs = 2^E with E = max(exponent of rstd,
// -16) (h 2^E is then a multiple of 2^-149, exact), m = fl(rstd 2^-E).
// Rows whose rstd is below 2^-60, zero or NaN form every product in 64 bits.
struct RowScale {
    double rstd;
    uint64_t hs2, m2;   // {hs, hs}, {m, m}
    bool wide;
};
__device__ __forceinline__ RowScale row_scale(double rstd) {
    RowScale r;
    r.rstd = rstd;
    const int E = max((__double2hiint(rstd) >> 20) - 1023, -16);
    const float hs = __uint_as_float((uint32_t)(E + 127) << 23);
    const float m = (float)(rstd * __hiloint2double((1023 - E) << 20, 0));
    r.hs2 = f32x2(hs, hs);
    r.m2 = f32x2(m, m);
    // not in [2^-60, infinity): rstd is zero or positive, so its upper word orders it
    r.wide = (uint32_t)__double2hiint(rstd) - (963u << 20) >= (2047u - 963u) << 20;
    return r;
}

__device__ __noinline__ uint4 normalise_wide(uint4 hv, uint4 wv, double rstd) {
    const uint32_t h[4] = {hv.x, hv.y, hv.z, hv.w}, w[4] = {wv.x, wv.y, wv.z, wv.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = pack_bf16x2(narrow_for_bf16(bf16_lo(h[i]), bf16_lo(w[i]), rstd),
                           narrow_for_bf16(bf16_hi(h[i]), bf16_hi(w[i]), rstd));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// y = bf16(h rstd weight) of 8 elements, and in `mag` per half the largest magnitude of y (amax_word8).
__device__ __forceinline__ uint4 normalise(uint4 hv, uint4 wv, const RowScale& rs, uint32_t& mag) {
    const uint32_t h[4] = {hv.x, hv.y, hv.z, hv.w}, w[4] = {wv.x, wv.y, wv.z, wv.w};
    uint32_t o[4], low[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t hf = f32x2_bits(h[i] << 16, h[i] & 0xffff0000u), wf = f32x2_bits(w[i] << 16, w[i] & 0xffff0000u);
        const float2 q = f32x2_split(mul_f32x2(mul_f32x2(mul_f32x2(hf, rs.hs2), wf), rs.m2));
        o[i] = pack_bf16x2(q.x, q.y);
        // low halves + 0x8002: 0 .. 4 within two units of a tie; the carry from the lower into the upper
        // half adds at most 1, so up to 5 counts
        low[i] = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x5410) + 0x80028002u;
    }
    uint32_t lo = __vminu2(__vminu2(low[0], low[1]), __vminu2(low[2], low[3]));
    lo = min(lo & 0xffffu, lo >> 16);
    // an infinite y: the product may have left FP32 although the value did not
    mag = hmax_abs(hmax_abs(o[0], o[1]), hmax_abs(o[2], o[3]));
    const uint32_t hi = mag & 0x7fff7fffu;
    const bool inf = (hi & 0xffffu) >= 0x7f80u || hi >= 0x7f800000u;
    if (lo <= 5u || inf || rs.wide) {
        const uint4 y = normalise_wide(hv, wv, rs.rstd);
        mag = amax_word8(y);
        return y;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A block's scale byte, written by one of its lanes: `at` is the row's first
// byte in the tile layout or the dense one.  The row's last block also writes
// the zeros that pad its columns to a multiple of four in the tile layout.
__device__ __forceinline__ void store_scale(const NormArgs& a, uint8_t* at, int col, uint32_t byte) {
    if (!a.sf_mma) {
        at[col] = (uint8_t)byte;
        return;
    }
    uint8_t* p = at + (uint32_t)(col >> 2) * 512u;
    p[col & 3] = (uint8_t)byte;
    if (col == a.s_cols - 1)
        for (int c = (col & 3) + 1; c < 4; ++c) p[c] = 0u;
}

// One row per CTA, kVec 8-element vectors per thread, all loaded before any
// is used: many rows take four (fewer warps per row, more rows in flight),
// few rows one (the row's latency counts).  Four (MXFP8) or two (NVFP4)
// neighbouring lanes hold a block: 16-byte loads stay coalesced and the block
// maximum takes one or two shuffles.
template <NormOut kOut, int kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, (kVec == 5 ? 768 : 1024) / kMaxThreads) norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr bool kMx = kOut == NormOut::kMxfp8 || kOut == NormOut::kMxfp8Fake;
    constexpr bool kFake = kOut == NormOut::kMxfp8Fake || kOut == NormOut::kNvfp4Fake;
    const int threads = (int)blockDim.x;
    let_later_kernels_start();
    wait_for_earlier_kernels();
    if (!kFake && blockIdx.x >= a.row_ctas) {   // zero scales of the rows that pad the last band
        for (uint64_t i = (uint64_t)(blockIdx.x - a.row_ctas) * threads + threadIdx.x; i < a.pad_words;
             i += (uint64_t)(gridDim.x - a.row_ctas) * threads) {
            const uint64_t row = i / a.sf_ct;
            const uint32_t ct = (uint32_t)(i - row * a.sf_ct);
            const uint32_t b = (uint32_t)(row / a.pad_rows), m = a.rows.d + (uint32_t)(row - (uint64_t)b * a.pad_rows);
            st_u32(a.scale + (int64_t)b * a.sf_slab + mma_scale_offset(m, 4u * ct, a.sf_ct), 0u);
        }
        return;
    }
    __shared__ double part[kMaxThreads / 32];
    const uint32_t r = blockIdx.x;
    const uint32_t b = fdiv(r, a.rows), m = r - b * a.rows.d;
    const int lane = threadIdx.x & 31;
    const char* x = a.x.ptr + (int64_t)b * a.x.bstride + (int64_t)m * a.x.rstride + 16 * threadIdx.x;
    const int step = 16 * threads;   // bytes between a thread's vectors
    uint4 v[kVec], wv[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        v[i] = i * threads + (int)threadIdx.x < a.vecs ? ld_once_v4(x + i * step) : make_uint4(0u, 0u, 0u, 0u);
    const float amax_in = kMx ? 0.0f : ld_f32(a.amax + b);
    if (a.res.ptr) {
        const char* res = a.res.ptr + (int64_t)b * a.res.bstride + (int64_t)m * a.res.rstride + 16 * threadIdx.x;
        char* h = a.h.ptr + (int64_t)b * a.h.bstride + (int64_t)m * a.h.rstride + 16 * threadIdx.x;
        uint4 u[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            u[i] = i * threads + (int)threadIdx.x < a.vecs ? ld_once_v4(res + i * step) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            v[i] = add_bf16(v[i], u[i]);
            if (i * threads + (int)threadIdx.x < a.vecs) st_v4(h + i * step, v[i]);
        }
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int k = i * threads + (int)threadIdx.x;
        wv[i] = k < a.vecs ? ld_v4(a.weight + k) : make_uint4(0u, 0u, 0u, 0u);
        s += squares(v[i]);
    }
    s = warp_sum(s);
    if (threads > 32) {
        if (lane == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        // the same order in every thread; few rows: the latency counts (one row of 7168 2.7 us, 3.0 with the loop),
        // many: the instructions (16384 rows of 1024 22.4 us, 22.6 without it)
        if (kVec == 1) {
            s = warp_sum(lane < threads / 32 ? part[lane] : 0.0);
        } else {
            s = 0.0;
            for (int i = 0; i < threads / 32; ++i) s += part[i];
        }
    }
    const RowScale rs = row_scale(rstd_of(s, a.d, a.inv_d, a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = (float)rs.rstd;

    float gs = 0.0f, g6 = 0.0f, r6 = 0.0f;
    bool fast6 = false;
    if (!kMx) {
        gs = __fdiv_rn(amax_in, 2688.0f);
        g6 = __fmul_rn(6.0f, gs);
        r6 = __frcp_rn(g6);
        fast6 = div_fast_ok(g6);
        if (!kFake && m == 0 && threadIdx.x == 0) a.gs[b] = gs;
    }
    char* out = a.out.ptr + (int64_t)b * a.out.bstride + (int64_t)m * a.out.rstride;
    uint8_t* scales = kFake ? nullptr
                            : a.scale + (a.sf_mma ? (int64_t)b * a.sf_slab + mma_scale_offset(m, 0u, a.sf_ct)
                                                  : (int64_t)r * a.s_cols);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (i * threads >= a.vecs) break;   // uniform: shuffles below take whole warps
        const int k = i * threads + (int)threadIdx.x;
        const bool on = k < a.vecs;
        uint32_t mw;
        const uint4 y = normalise(v[i], wv[i], rs, mw);   // zeros past the row
        mw = hmax_abs(mw, __shfl_xor_sync(0xffffffffu, mw, 1));
        if (kMx) mw = hmax_abs(mw, __shfl_xor_sync(0xffffffffu, mw, 2));
        mw &= 0x7fff7fffu;
        const uint32_t amax = max(mw & 0xffffu, mw >> 16);
        if (kMx) {
            // scale byte e + 127 with e = min{k : amax <= 448 2^k}: 448 = 1.75 * 2^8, so a mantissa above .75
            // (96 of 128) carries into the exponent; below 2^-127 (zero and subnormal amax) the byte is 0
            const int byte8 = max((int)((amax + 31u) >> 7) - 8, 0);
            const float inv = __uint_as_float((uint32_t)(254 - byte8) << 23);   // 2^-e
            const uint64_t inv2 = f32x2(inv, inv);
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
            float2 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = f32x2_split(mul_f32x2(f32x2_bits(w[j] << 16, w[j] & 0xffff0000u), inv2));
            const uint2 c = make_uint2(e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y), e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
            if (kFake) {
                if (on) st_v4(out + 16 * (int64_t)k, fp8_dequant8(c, exp2i(byte8 - 127)));
            } else {
                if (on) st_v2(out + 8 * (int64_t)k, c);
                if (on && (k & 3) == 0) store_scale(a, scales, k >> 2, (uint32_t)byte8);
            }
        } else {
            const float am = __uint_as_float(amax << 16);
            uint32_t sb = 0u;
            if (gs != 0.0f) sb = e4m3x2(fast6 ? div_fast(am, g6, r6) : div_slow(am, g6), 0.0f) & 0xffu;
            const float d = __fmul_rn(e4m3_decode(sb), gs);
            float q[8];
            if (div_fast_ok(d)) quotients8<true>(y, d, __frcp_rn(d), q);
            else quotients8<false>(y, d, 0.0f, q);
            const uint32_t c = e2m1x8(q);
            if (kFake) {
                if (on) st_v4(out + 16 * (int64_t)k, dequant_half_h(c, e4m3x2_f16x2(sb * 0x0101u), f32x2(gs, gs)));
            } else {
                if (on) st_u32(out + 4 * (int64_t)k, c);
                if (on && (k & 1) == 0) store_scale(a, scales, k >> 1, sb);
            }
        }
    }
}

// ---------------------------------------------------------------- backward
//
// With g = dy weight, xhat = h rstd and c = sum_d g_d xhat_d / D:
//   dx = bf16(rstd (g - c xhat) + dh)      (also the residual's gradient)
//   dweight = sum over rows of dy xhat
// (the quantiser passes its gradient straight through).  A CTA walks rows
// blockIdx.x, + gridDim.x, ... and keeps its part of dweight in FP32
// registers; the parts are added in CTA order by a second launch, so the
// result does not depend on timing.  FP32 throughout: the inputs are BF16
// and no value decides a code.

// A CTA has `groups` groups of `tpr` threads, each group a row at a time.
// Rows come in through shared memory by bulk copies, `ring` rows ahead: the
// reduction's barrier, which every row has to wait for, would otherwise
// empty the memory pipe (with one row ahead in registers the kernel ran at
// two thirds of the copy rate at 8192 x 2560).

struct NormBwdArgs {
    View dy, dh, h, dx;          // dh.ptr null: no gradient of h
    const uint4* weight;
    const float* rstd;
    float* parts;                // [gridDim.x][D], null: no dweight
    FastDiv rows;
    uint32_t total_rows;
    int vecs;
    int groups, tpr, ring;
};

__device__ uint32_t g_norm_error = 0u;
constexpr uint64_t kNormWaitNs = 2000000000ull;
constexpr int kMaxRing = 4, kMaxGroups = 8;

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// kHoldW: the weight stays in registers where 122 of them fit; else it is read
// again from L1, so that nothing spills.  A row's chain of waits (its copy, its
// sums, the barrier) is what keeps the kernel from HBM's rate, hence rstd
// loaded a row ahead and several CTAs per SM where registers allow: 16384 x
// 7168 with dh takes 144 us (940 MB, 6.5 TB/s), 16384 x 4096 87 us.
template <int kVec, int kMaxThreads, int kMinCtas, bool kHoldW>
__global__ void __launch_bounds__(kMaxThreads, kMinCtas) norm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
    // 1024 threads have 64 registers each: the second pass reads the row from shared memory again
    constexpr bool kReread = kMaxThreads > 512;
    extern __shared__ __align__(128) uint8_t smem_rows[];
    __shared__ float part[2][kMaxThreads / 32];
    __shared__ __align__(8) uint64_t bars[kMaxGroups * kMaxRing];
    const int tpr = a.tpr, group = (int)threadIdx.x / tpr, t = (int)threadIdx.x - group * tpr;
    const int warps = tpr / 32, warp0 = group * warps;
    const uint32_t row_bytes = (uint32_t)a.vecs * 16u, stage = 3u * row_bytes;
    const uint32_t ring = smem_addr(smem_rows) + (uint32_t)(group * a.ring) * stage;
    const uint32_t full = smem_addr(bars) + 8u * (uint32_t)(group * kMaxRing);
    const bool has_dh = a.dh.ptr != nullptr;
    const uint32_t bytes = has_dh ? stage : 2u * row_bytes;
    const float inv_d = __fdiv_rn(1.0f, (float)(8 * a.vecs));
    const uint32_t first = blockIdx.x * (uint32_t)a.groups + (uint32_t)group, stride = gridDim.x * (uint32_t)a.groups;

    if (t == 0) {
        for (int i = 0; i < a.ring; ++i) mbar_init(full + 8u * i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    let_later_kernels_start();
    wait_for_earlier_kernels();
    const uint64_t pol = l2_policy_evict_first();
    auto fetch = [&](uint32_t r, uint32_t st) {   // one thread of the group
        const uint32_t b = fdiv(r, a.rows), m = r - b * a.rows.d;
        const uint32_t at = ring + st * stage, bar = full + 8u * st;
        mbar_arrive_expect_tx(bar, bytes);
        bulk_load(at, a.dy.ptr + (int64_t)b * a.dy.bstride + (int64_t)m * a.dy.rstride, row_bytes, bar, pol);
        bulk_load(at + row_bytes, a.h.ptr + (int64_t)b * a.h.bstride + (int64_t)m * a.h.rstride, row_bytes, bar, pol);
        if (has_dh)
            bulk_load(at + 2u * row_bytes, a.dh.ptr + (int64_t)b * a.dh.bstride + (int64_t)m * a.dh.rstride, row_bytes,
                      bar, pol);
    };
    if (t == 0)
        for (int i = 0; i < a.ring; ++i)
            if ((uint64_t)first + (uint64_t)i * stride < a.total_rows) fetch(first + (uint32_t)i * stride, (uint32_t)i);

    float dw[kVec][8];
    uint4 held[kHoldW ? kVec : 1];
    auto weight = [&](int i) {
        const int k = i * tpr + t;
        return k < a.vecs ? ld_v4(a.weight + k) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (kHoldW) held[i] = weight(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    uint32_t st = 0u, phase = 0u;
    int flip = 0;
    bool alive = true;
    int waits = a.ring;
    float rstd_next = first < a.total_rows ? ld_f32(a.rstd + first) : 0.0f;
    for (uint64_t r64 = first; r64 < a.total_rows; r64 += stride, flip ^= 1) {
        const uint32_t r = (uint32_t)r64;
        const float rstd = rstd_next;   // loaded a row ahead
        if (r64 + stride < a.total_rows) rstd_next = ld_f32(a.rstd + r + stride);
        // once a wait has given up the outputs are unspecified: no further copies, and waits only for those in flight
        if (waits > 0 && !mbar_wait_bounded(full + 8u * st, phase, kNormWaitNs)) {
            atomicOr(&g_norm_error, kErrTmaTimeout);
            alive = false;
        }
        if (!alive) --waits;
        constexpr int kKept = kReread ? 1 : kVec;
        uint4 vg[kKept], vh[kKept], vd[kKept];
        const uint32_t at = ring + st * stage + 16u * (uint32_t)t;
        auto load = [&](int i, int k, bool with_dh) {   // vector i into place k
            const bool on = i * tpr + t < a.vecs;
            const uint32_t o = at + 16u * (uint32_t)(i * tpr);
            vg[k] = on ? ld_shared_v4(o) : make_uint4(0u, 0u, 0u, 0u);
            vh[k] = on ? ld_shared_v4(o + row_bytes) : make_uint4(0u, 0u, 0u, 0u);
            vd[k] = on && with_dh ? ld_shared_v4(o + 2u * row_bytes) : make_uint4(0u, 0u, 0u, 0u);
        };
        if constexpr (!kReread) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) load(i, i, has_dh);
        }
        float c = 0.0f;
#pragma unroll
        for (int i0 = 0; i0 < kVec; ++i0) {
            const int i = kReread ? 0 : i0;
            if (kReread) load(i0, 0, false);
            const uint32_t g[4] = {vg[i].x, vg[i].y, vg[i].z, vg[i].w}, hh[4] = {vh[i].x, vh[i].y, vh[i].z, vh[i].w};
            const uint4 wv = kHoldW ? held[kHoldW ? i0 : 0] : weight(i0);
            const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float t0 = bf16_lo(g[j]) * (bf16_lo(hh[j]) * rstd), t1 = bf16_hi(g[j]) * (bf16_hi(hh[j]) * rstd);
                dw[i0][2 * j] += t0;
                dw[i0][2 * j + 1] += t1;
                c = __fmaf_rn(t0, bf16_lo(w[j]), c);
                c = __fmaf_rn(t1, bf16_hi(w[j]), c);
            }
        }
        c = warp_sum_f(c);
        if ((t & 31) == 0) part[flip][warp0 + (t >> 5)] = c;
        // every thread of the group has read the stage; the two halves of `part` alternate
        if (warps > 1) asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "r"(tpr) : "memory");
        else __syncwarp();
        const uint64_t next = r64 + (uint64_t)a.ring * stride;
        const uint32_t used = st;
        if (!kReread && t == 0 && alive && next < a.total_rows) fetch((uint32_t)next, used);
        if (++st == (uint32_t)a.ring) {
            st = 0u;
            phase ^= 1u;
        }
        if (warps > 1) {   // four chains; the loads do not wait for the additions
            float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kMaxThreads / 32; ++i)
                if (i < warps) q[i & 3] += part[flip][warp0 + i];
            c = (q[0] + q[1]) + (q[2] + q[3]);
        }
        c *= inv_d;
        const uint32_t b = fdiv(r, a.rows), m = r - b * a.rows.d;
        char* dx = a.dx.ptr + (int64_t)b * a.dx.bstride + (int64_t)m * a.dx.rstride + 16 * t;
#pragma unroll
        for (int i0 = 0; i0 < kVec; ++i0) {
            if (i0 * tpr + t >= a.vecs) continue;
            const int i = kReread ? 0 : i0;
            if (kReread) load(i0, 0, has_dh);
            const uint32_t g[4] = {vg[i].x, vg[i].y, vg[i].z, vg[i].w}, hh[4] = {vh[i].x, vh[i].y, vh[i].z, vh[i].w};
            const uint4 wv = kHoldW ? held[kHoldW ? i0 : 0] : weight(i0);
            const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w}, d[4] = {vd[i].x, vd[i].y, vd[i].z, vd[i].w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e0 = __fmaf_rn(bf16_lo(hh[j]) * rstd, -c, bf16_lo(g[j]) * bf16_lo(w[j]));
                const float e1 = __fmaf_rn(bf16_hi(hh[j]) * rstd, -c, bf16_hi(g[j]) * bf16_hi(w[j]));
                o[j] = pack_bf16x2(__fmaf_rn(e0, rstd, bf16_lo(d[j])), __fmaf_rn(e1, rstd, bf16_hi(d[j])));
            }
            st_v4(dx + (int64_t)16 * (i0 * tpr), make_uint4(o[0], o[1], o[2], o[3]));
        }
        if (kReread) {   // the stage has been read by all only now
            asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "r"(tpr) : "memory");
            if (t == 0 && alive && next < a.total_rows) fetch((uint32_t)next, used);
        }
    }
    if (!a.parts) return;
    // the groups' dweights are added in group order in shared memory (every row's copy has been read)
    float* sum = reinterpret_cast<float*>(smem_rows);
    for (int g = 0; g < a.groups; ++g) {
        __syncthreads();
        if (group != g) continue;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int k = i * tpr + t;
            if (k >= a.vecs) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (g > 0) dw[i][j] += sum[8 * k + j];
                if (g < a.groups - 1) sum[8 * k + j] = dw[i][j];
            }
            if (g == a.groups - 1) {
                float* q = a.parts + (int64_t)blockIdx.x * a.vecs * 8 + 8 * (int64_t)k;
                st_v4(q, make_uint4(__float_as_uint(dw[i][0]), __float_as_uint(dw[i][1]), __float_as_uint(dw[i][2]),
                                    __float_as_uint(dw[i][3])));
                st_v4(q + 4, make_uint4(__float_as_uint(dw[i][4]), __float_as_uint(dw[i][5]), __float_as_uint(dw[i][6]),
                                        __float_as_uint(dw[i][7])));
            }
        }
    }
}

// dweight[d] = sum of the parts in a fixed order: 32 warps take every 32nd
// part of 32 columns, eight loads in flight each, then the 32 sums are added.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* parts, int n_parts, int D, void* dweight,
                                                            int bf16_out) {
    __shared__ float s[32][33];
    let_later_kernels_start();
    wait_for_earlier_kernels();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = (int)blockIdx.x * 32 + lane;
    float v = 0.0f;
    for (int p = warp; p < n_parts; p += 8 * 32) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = d < D && p + 32 * i < n_parts ? ld_f32(parts + (int64_t)(p + 32 * i) * D + d) : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += t[i];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && d < D) {
        v = s[0][lane];
#pragma unroll
        for (int i = 1; i < 32; ++i) v += s[i][lane];
        if (bf16_out) static_cast<uint16_t*>(dweight)[d] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
        else static_cast<float*>(dweight)[d] = v;
    }
}

// Threads per row: the fewest whole warps that hold it in `vec` vectors each.
int norm_threads(int64_t D, int vec) { return (int)((D / 8 + 32 * vec - 1) / (32 * vec)) * 32; }

template <NormOut kOut, int kVec, int kMaxThreads>
cudaError_t launch_norm_out(const NormArgs& a, int threads, cudaStream_t s) {
    const unsigned pads = a.pad_words ? (unsigned)std::min<uint64_t>((a.pad_words + threads - 1) / threads, 128) : 0u;
    return launch_early(norm_kernel<kOut, kVec, kMaxThreads>, a.row_ctas + pads, (unsigned)threads, 0, s, 1u, a);
}

template <NormOut kOut>
cudaError_t launch_norm_kind(const NormArgs& a, cudaStream_t s) {
    const int64_t D = 8 * (int64_t)a.vecs;
    // few rows leave SMs idle either way: spread each over four times the threads
    if (D <= 8192 && a.total_rows <= (uint32_t)sm_count(current_device()))
        return launch_norm_out<kOut, 1, 1024>(a, norm_threads(D, 1), s);
    // five vectors per thread where they fill every lane and four do not (2560 columns, 8192 rows to MXFP8: 29.9
    // against 31.2 us; where both leave lanes over, four are faster: 3584 columns, 16384 rows 70.1 against 72.7)
    if (D <= 8192 && norm_threads(D, 5) * 5 == a.vecs && norm_threads(D, 4) * 4 > a.vecs)
        return launch_norm_out<kOut, 5, 256>(a, norm_threads(D, 5), s);
    if (D <= 8192) return launch_norm_out<kOut, 4, 256>(a, norm_threads(D, 4), s);
    return launch_norm_out<kOut, 4, 1024>(a, norm_threads(D, 4), s);
}

// Launch shape of the backward pass: two vectors per thread while 512 threads
// hold the row, four above (4096 x 12288: 94 us, 123 with two and 1024
// threads); small rows share a CTA of about 256 threads (one dweight part per
// CTA), and as many rows ahead as pay.
struct BwdShape {
    int vec, tpr, groups, ctas, ring, grid;
    size_t smem;
};
constexpr size_t kBwdSmem = 200 * 1024;   // per SM
constexpr int kBwdPairThreads = 320;
BwdShape norm_bwd_shape(int64_t rows, int64_t D) {
    BwdShape s;
    s.vec = D <= 8192 ? 2 : 4;
    s.tpr = norm_threads(D, s.vec);
    s.groups = std::max(1, std::min(kMaxGroups, 256 / s.tpr));
    const int threads = s.tpr * s.groups;
    // 512 threads of 128 registers, or two CTAs of up to 320 threads with about 100 (16384 x 4112: 94.8 us, one CTA
    // per SM 116.7; 16384 x 5120: 115 against 119)
    s.ctas = s.vec == 2 && threads > 256 && threads <= kBwdPairThreads ? 2 : std::max(1, 512 / threads);
    const size_t stage = 6 * (size_t)D * s.groups;
    // several CTAs per SM hide each other's waits: two rows each (16384 x 4096: 86.5 us, 91.6 with four); one alone
    // needs more (16384 x 7168: 143.7 us with four, 146.9 with two)
    const size_t most = s.ctas > 1 ? 2 : kMaxRing;
    s.ring = (int)std::max<size_t>(1, std::min<size_t>(most, kBwdSmem / s.ctas / stage));
    s.smem = s.ring * stage;
    s.grid = persistent_grid((rows + s.groups - 1) / s.groups, s.ctas);
    return s;
}

}  // namespace

cudaError_t launch_norm(const Norm& n, cudaStream_t s) {
    NormArgs a;
    a.x = n.x;
    a.res = n.res;
    a.h = n.h;
    a.out = n.out;
    a.weight = static_cast<const uint4*>(n.weight);
    a.eps = n.eps;
    a.d = (double)n.x.cols;
    a.inv_d = 1.0 / a.d;
    a.amax = n.amax;
    a.gs = n.gs;
    a.scale = n.scale;
    a.rstd = n.rstd;
    a.rows = make_fastdiv((uint32_t)n.x.rows);
    a.total_rows = (uint32_t)(n.x.batch * n.x.rows);
    a.vecs = (int)(n.x.cols / 8);
    a.s_cols = (int)(n.x.cols / (n.fp4 ? 16 : 32));
    a.sf_mma = n.scale_mma;
    a.sf_ct = (uint32_t)mma_scale_col_tiles(a.s_cols);
    a.sf_slab = mma_scale_slab_bytes(n.x.rows, a.s_cols);
    a.row_ctas = a.total_rows;
    a.pad_rows = n.scale_mma && !n.fake ? (uint32_t)((128 - n.x.rows % 128) % 128) : 0u;
    a.pad_words = (uint64_t)n.x.batch * a.pad_rows * a.sf_ct;
    if (n.fp4) return n.fake ? launch_norm_kind<NormOut::kNvfp4Fake>(a, s) : launch_norm_kind<NormOut::kNvfp4>(a, s);
    return n.fake ? launch_norm_kind<NormOut::kMxfp8Fake>(a, s) : launch_norm_kind<NormOut::kMxfp8>(a, s);
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    return ((size_t)norm_bwd_shape(rows, D).grid * (size_t)D * 4 + 255) / 256 * 256;
}

namespace {

template <int kVec, int kMaxThreads, int kMinCtas, bool kHoldW>
cudaError_t launch_bwd_kernel(const NormBwdArgs& a, const BwdShape& sh, cudaStream_t s) {
    static int configured[kMaxDevices] = {0};
    const void* fn = (const void*)norm_bwd_kernel<kVec, kMaxThreads, kMinCtas, kHoldW>;
    const cudaError_t e = set_smem_limit_once(configured, &fn, 1, (int)kBwdSmem);
    if (e != cudaSuccess) return e;
    return launch_early(norm_bwd_kernel<kVec, kMaxThreads, kMinCtas, kHoldW>, (unsigned)sh.grid,
                        (unsigned)(sh.tpr * sh.groups), sh.smem, s, 1u, a);
}

}  // namespace

cudaError_t read_and_clear_norm_error(uint32_t* code) {
    uint32_t zero = 0u;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_norm_error, sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(uint32_t));
}

cudaError_t launch_norm_bwd(const NormBwd& n, cudaStream_t s) {
    NormBwdArgs a;
    a.dy = n.dy;
    a.dh = n.dh;
    a.h = n.h;
    a.dx = n.dx;
    a.weight = static_cast<const uint4*>(n.weight);
    a.rstd = n.rstd;
    a.parts = n.dweight ? static_cast<float*>(n.workspace) : nullptr;
    a.rows = make_fastdiv((uint32_t)n.h.rows);
    a.total_rows = (uint32_t)(n.h.batch * n.h.rows);
    a.vecs = (int)(n.h.cols / 8);
    const BwdShape sh = norm_bwd_shape(a.total_rows, n.h.cols);
    a.groups = sh.groups;
    a.tpr = sh.tpr;
    a.ring = sh.ring;
    const int threads = sh.tpr * sh.groups;
    const cudaError_t e = sh.vec == 4  ? threads <= 512 ? launch_bwd_kernel<4, 512, 1, false>(a, sh, s)
                                                       : launch_bwd_kernel<4, 1024, 1, false>(a, sh, s)
                          : threads <= 256             ? launch_bwd_kernel<2, 256, 2, true>(a, sh, s)
                          : threads <= kBwdPairThreads ? launch_bwd_kernel<2, kBwdPairThreads, 2, false>(a, sh, s)
                                                       : launch_bwd_kernel<2, 512, 1, true>(a, sh, s);
    if (e != cudaSuccess || !n.dweight) return e;
    const int D = (int)n.h.cols;
    return launch_early(norm_dweight_kernel, (unsigned)((D + 31) / 32), 1024, 0, s, 1u, (const float*)a.parts, sh.grid, D,
                        n.dweight, n.dweight_bf16);
}

}  // namespace pwq
