// pwq_tcgen05.cuh -- 5th-generation tensor core helpers (sm_100a): tensor
// memory, shared-memory matrix descriptors, block-scaled MMA and the scale
// copies, as the PTX ISA's tcgen05 chapter defines them.
#pragma once

#include "pwq_device.cuh"

namespace pwq {

// Bit of the device error word: a wait inside a block-scaled product gave up.
constexpr uint32_t kErrMatmulTimeout = 4u;

// ---------------------------------------------------------------- barriers

// Whether the barrier's phase of that parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// ---------------------------------------------------------------- tensor memory

// Whole warp.  Writes the TMEM base address of `cols` columns (a power of
// two, 32..512) to the shared-memory word at `dst`.
template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    if (kCtas == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    if (kCtas == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Whole warp: 16 / 32 consecutive 32-bit columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
// Whole warp: 16 lanes (addr's lane and the 15 after it) x 32 columns as 8x8
// fragments: of columns 8 r .. 8 r + 7, thread T gets in v[4 r], v[4 r + 1] the
// columns 2 (T % 4), + 1 of lane T / 4, and in v[4 r + 2], v[4 r + 3] those of lane T / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
// Whole warp: four 8x8 fragments of 16-bit elements, stored transposed; lane
// 8 i + c gives the 16-byte address of column c of fragment i.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- warp-uniform roles
//
// TMA and tcgen05 instructions take their operands from uniform registers.
// A producer or issuer loop that runs in one lane of a diverged warp pays
// about 65 to 130 clocks per instruction to bring them there (measured: an
// MMA step of 12 scale copies and 4 MMAs issued in 1800 clocks); the same
// loop run by the whole converged warp, with one elected lane at the
// instructions, issues them back to back.

// The warp's index as a value that the compiler knows to be uniform.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0u;
}

// Position in a ring of barriers: stage and the parity of its current use.
struct RingPos {
    uint32_t at = 0u, phase = 0u;
    __device__ __forceinline__ void next(uint32_t stages) {
        if (++at == stages) {
            at = 0u;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ void prefetch_tensor_map(const void* map) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
}

// ---------------------------------------------------------------- descriptors

// K-major operand tile in shared memory, rows of 128 bytes in the 128-byte
// swizzle (1024-byte aligned, 8-row groups 1024 bytes apart).  Advancing
// along K by 32 bytes inside the swizzled row adds 2 to the start address.
__device__ __forceinline__ uint64_t desc_swizzle128(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// A scale tile: 32 lines of 16 contiguous bytes, no swizzle (8-line groups
// 128 bytes apart).
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// ---------------------------------------------------------------- formats of a block-scaled product

// MXFP8: E4M3 codes, K = 32 per MMA (32 bytes), one UE8M0 byte per row and
// MMA; a scale tile (four scale columns) serves the four MMAs of a 128-byte
// step.  NVFP4: packed E2M1, K = 64 per MMA (32 bytes), four E4M3 bytes per
// row and MMA; one scale tile per MMA.
enum class ProductFormat { kMxfp8, kNvfp4 };

template <ProductFormat kF>
struct ProductTraits {
    static constexpr bool kFp4 = kF == ProductFormat::kNvfp4;
    static constexpr int kScaleTiles = kFp4 ? 4 : 1;     // 512-byte scale tiles per operand band and 128-byte step
    static constexpr uint32_t kScaleBytes = 512u * kScaleTiles;
};

constexpr uint32_t kStepBytes = 128;   // bytes of a code row per pipeline step
constexpr int kMmasPerStep = 4;        // 32 bytes of K each

// Instruction descriptor for an M x N block-scaled MMA, FP32 accumulation,
// both operands K-major.  MXFP8: scale format UE8M0 (bit 23), E4M3 (type 0);
// NVFP4: scale format UE4M3, E2M1 (type 1 in bits 7 and 10).
template <ProductFormat kF>
__device__ constexpr uint32_t mma_idesc(int m, int n) {
    return (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 7) << 27 |
           (kF == ProductFormat::kNvfp4 ? (1u << 7 | 1u << 10) : 1u << 23);
}

// One thread.  D[tmem] (+)= A B^T with block scales; scale_a / scale_b are
// the TMEM addresses of the scale tiles.
template <ProductFormat kF, int kCtas>
__device__ __forceinline__ void mma_block_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t scale_a,
                                                 uint32_t scale_b, bool accumulate) {
    const uint32_t acc = accumulate ? 1u : 0u;
#define PWQ_MMA(GROUP, KIND)                                                                                     \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                               \
                 "tcgen05.mma.cta_group::" GROUP "." KIND " [%0], %1, %2, %3, [%5], [%6], p;\n\t}"               \
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(scale_a), "r"(scale_b) : "memory")
    if (kF == ProductFormat::kNvfp4) {
        if (kCtas == 1) PWQ_MMA("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
        else PWQ_MMA("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    } else {
        if (kCtas == 1) PWQ_MMA("1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
        else PWQ_MMA("2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    }
#undef PWQ_MMA
}

// One thread: a 512-byte scale tile from shared memory into four TMEM
// columns, repeated for the four warps' lanes.  Executed in order with the
// MMAs that the same thread issues after it.
template <int kCtas>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if (kCtas == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(desc) : "memory");
}

// One thread: arrives on `bar` when every tcgen05 operation issued by this
// thread so far has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

// The same for a CTA pair: arrives on the barrier at this offset in both CTAs.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .b16 both;\n\tmov.b16 both, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}"
        :: "r"(bar) : "memory");
}

// 3-D tiled TMA load into this CTA's shared memory that completes a barrier
// of either CTA of the pair (`bar`: its address in the cluster window).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}

// 3-D tiled TMA store of a shared-memory box, in this thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :: "l"(tmap), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's bulk groups still read shared memory / are still in flight.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------- clusters

// Arrives on a barrier of any CTA of the cluster (address in the cluster
// window) to say that this warp's TMEM loads have ended: registers hold the
// values, no memory is published, so the arrival is relaxed and the
// tcgen05 fences on both sides give the order (a releasing arrival here
// costs about 1000 clocks).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster (warps converged).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared-memory address `addr` of this CTA, as seen in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

}  // namespace pwq
