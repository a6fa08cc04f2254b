// tc_mx_ptx.cuh -- inline-PTX wrappers for the block-scaled tcgen05 products:
// MXFP8 (kind::mxf8f6f4, one scale per 32 elements of K) and MXFP4 (kind::mxf4),
// their scales copied from shared memory to TMEM, and what clusters need.
//
// Operand tiles are K-major rows of 128 bytes in the 128-byte swizzle, as in
// tc_ptx.cuh: 128 elements of 8 bits or 256 of 4 bits; one MMA takes 32 bytes of a
// row (K = 32 or 64).
//
// Scales of 128 rows x 4 blocks are 512 bytes, the bytes of (row, block) at
// 16 (row % 32) + 4 (row / 32) + block: 32 rows of 16 bytes, which tcgen05.cp
// 32x128b.warpx4 puts into 4 TMEM columns of every lane quarter: column row / 32,
// lane row % 32, a byte per block.  An MMA names its blocks' bytes by the scale id
// in its instruction descriptor.
#pragma once

#include "tc_ptx.cuh"

namespace gdn {
namespace tc {

// Instruction descriptor of the block-scaled kinds: e4m3 (0) or e2m1 (1) A and B,
// power-of-two scales, N >> 3 in bits 17-22, M >> 4 in bits 24-28; `id` is the
// scale byte both operands take.
__host__ __device__ constexpr uint32_t idesc_mx(bool fp4, int M, int N, int id) {
    return ((uint32_t)id << 4) | ((fp4 ? 1u : 0u) << 7) | ((fp4 ? 1u : 0u) << 10) |
           ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
           ((uint32_t)id << 29);
}

// Descriptor of a 512-byte scale tile for tcgen05.cp: no swizzle, 8-row groups of
// 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// D (+)= A B with scales; warp-collective like mma_bf16.
template <bool FP4>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                       uint32_t sb, uint32_t accumulate) {
    if (FP4)
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// A 512-byte scale tile to 4 TMEM columns; in order with the MMAs the same warp
// issues.  Warp-collective.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n"
        ".reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n"
        "}\n" ::"r"(taddr),
        "l"(desc)
        : "memory");
}

// A whole stage in one go: its scale tiles to TMEM, its four MMAs (K = 128 in 8 bits,
// 256 in 4), and the arrival on `bar` when they are done.  One election for the stage and
// operands that differ by constants: single calls take the issuing warp twice as long.
// Scale tiles lie 512 bytes apart from `scales`: A's, then B's.
template <bool FP4>
__device__ __forceinline__ void mma_mx_stage(uint32_t d, uint64_t a, uint64_t b, uint64_t scales, uint32_t sa,
                                             uint32_t sb, uint32_t idesc, uint32_t accumulate, uint64_t *bar) {
    if (FP4)                       // scale ids 0 and 2: bits 4-5 and 29-30
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            ".reg .b64 a1, a2, a3, b1, b2, b3, s1, s2, s3;\n"
            ".reg .b32 i2, ta, tb;\n"
            "setp.ne.b32 p, %7, 0;\n"
            "or.b32 i2, %6, 0x40000020;\n"
            "add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
            "add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
            "add.s64 s1, %3, 32;\n add.s64 s2, %3, 64;\n add.s64 s3, %3, 96;\n"
            "add.s32 ta, %4, 4;\n add.s32 tb, %5, 4;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %3;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], s2;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %6, [%4], [%5], p;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a1, b1, i2, [%4], [%5], 1;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [ta], s1;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [tb], s3;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a2, b2, %6, [ta], [tb], 1;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a3, b3, i2, [ta], [tb], 1;\n"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%8];\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "l"(scales), "r"(sa), "r"(sb), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar))
            : "memory");
    else                           // scale ids 0 to 3
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            ".reg .b64 a1, a2, a3, b1, b2, b3, s1;\n"
            ".reg .b32 i1, i2, i3;\n"
            "setp.ne.b32 p, %7, 0;\n"
            "or.b32 i1, %6, 0x20000010;\n or.b32 i2, %6, 0x40000020;\n or.b32 i3, %6, 0x60000030;\n"
            "add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
            "add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
            "add.s64 s1, %3, 32;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %3;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], s1;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %6, [%4], [%5], p;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, i1, [%4], [%5], 1;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, i2, [%4], [%5], 1;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, i3, [%4], [%5], 1;\n"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%8];\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "l"(scales), "r"(sa), "r"(sb), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar))
            : "memory");
}

// mbar_wait for a whole warp by plain polling: the polls of mbar_wait may put the warp to
// sleep, and waking costs a mainloop that is short of time more than polling does.  The
// same answer in every lane.
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity, long long limit, int *status) {
    for (long long i = 0; i < limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n"
            "}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
    }
    set_status(status, GDN_ERR_TIMEOUT);
    return false;
}

// Waits until the word at `p`, which other CTAs add to with add_release, is `want`; their
// writes before that may then be read by this warp's TMA loads.  The same answer in every
// lane.
__device__ __forceinline__ bool word_spin(const uint32_t *p, uint32_t want, long long limit, int *status) {
    for (long long i = 0; i < limit; ++i) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        if (__all_sync(0xffffffffu, v == want)) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            __syncwarp();
            return true;
        }
    }
    set_status(status, GDN_ERR_TIMEOUT);
    return false;
}
// Adds 1 to the word at `p` behind every write of the warp, for the readers of word_spin.
__device__ __forceinline__ void add_release(uint32_t *p) {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}

// ------------------------------------------------------------------ CTA pairs
// The same for cta_group::2: two CTAs of a cluster work on one 256-row tile.  Each
// holds its 128 rows of A, half the rows of B, and 128 lanes of D; the even CTA issues
// for both, and descriptors name the same offsets in both shared memories.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols) {  // one warp of each
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
template <bool FP4>
__device__ __forceinline__ void mma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                            uint32_t sb, uint32_t accumulate) {
    if (FP4)
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n"
        ".reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n"
        "}\n" ::"r"(taddr),
        "l"(desc)
        : "memory");
}
// Arrives on `bar` of both CTAs once every MMA issued so far has completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar) {
    asm volatile(
        "{\n"
        ".reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
        "}\n" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// A whole stage in one go: its scale tiles to TMEM, its four MMAs (K = 128 in 8 bits,
// 256 in 4), and the arrival on `bar` of both CTAs when they are done.  The issuing
// warp is what bounds a pair's mainloop: one election for the stage and operands that
// differ by constants halve its time against the single calls above.  Scale tiles lie 512
// bytes apart from `scales`: A's, then B's rows 0-127, then B's rows 128-255.
template <bool FP4>
__device__ __forceinline__ void mma_mx_stage_pair(uint32_t d, uint64_t a, uint64_t b, uint64_t scales, uint32_t sa,
                                                  uint32_t sb, uint32_t accumulate, uint64_t *bar) {
    constexpr uint32_t kId0 = idesc_mx(FP4, 256, 256, 0), kId1 = idesc_mx(FP4, 256, 256, 1),
                       kId2 = idesc_mx(FP4, 256, 256, 2), kId3 = idesc_mx(FP4, 256, 256, 3);
    if (FP4)
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            ".reg .b64 a1, a2, a3, b1, b2, b3, s1, s2, s3, s4, s5;\n"
            ".reg .b32 i0, i2, ta, t4, t8, tc;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "mov.b32 i0, %9;\n"
            "mov.b32 i2, %10;\n"
            "add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
            "add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
            "add.s64 s1, %3, 32;\n add.s64 s2, %3, 64;\n add.s64 s3, %3, 96;\n"
            "add.s64 s4, %3, 128;\n add.s64 s5, %3, 160;\n"
            "add.s32 ta, %4, 4;\n add.s32 t4, %5, 4;\n add.s32 t8, %5, 8;\n add.s32 tc, %5, 12;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%4], %3;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], s2;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t4], s4;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, i0, [%4], [%5], p;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a1, b1, i2, [%4], [%5], 1;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [ta], s1;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t8], s3;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [tc], s5;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a2, b2, i0, [ta], [t8], 1;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a3, b3, i2, [ta], [t8], 1;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%7], %8;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "l"(scales), "r"(sa), "r"(sb), "r"(accumulate), "r"(smem_u32(bar)), "h"((uint16_t)3),
            "n"(kId0), "n"(kId2)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            ".reg .b64 a1, a2, a3, b1, b2, b3, s1, s2;\n"
            ".reg .b32 i0, i1, i2, i3, t4;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "mov.b32 i0, %9;\n mov.b32 i1, %10;\n mov.b32 i2, %11;\n mov.b32 i3, %12;\n"
            "add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
            "add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
            "add.s64 s1, %3, 32;\n add.s64 s2, %3, 64;\n"
            "add.s32 t4, %5, 4;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%4], %3;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], s1;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t4], s2;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, i0, [%4], [%5], p;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, i1, [%4], [%5], 1;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, i2, [%4], [%5], 1;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, i3, [%4], [%5], 1;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%7], %8;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "l"(scales), "r"(sa), "r"(sb), "r"(accumulate), "r"(smem_u32(bar)), "h"((uint16_t)3),
            "n"(kId0), "n"(kId1), "n"(kId2), "n"(kId3)
            : "memory");
}
// One operand's tile and scale tiles into this CTA, completing on a barrier of the pair
// (`bar`: a shared::cluster address).  Warp-collective, like the MMAs and for the same
// reason: issued by one lane of divergent code, the loads of a stage took longer than its
// MMAs.
__device__ __forceinline__ void load_operand_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                                  uint32_t scales, const CUtensorMap *smap, int k, int r,
                                                  uint32_t bar) {
    asm volatile(
        "{\n"
        ".reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%8];\n"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%4], [%5, {%9, %6, %7}], [%8];\n"
        "}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(scales), "l"(reinterpret_cast<uint64_t>(smap)),
        "r"(k), "r"(r), "r"(bar), "r"(0)
        : "memory");
}
// The same for one CTA: the scale tiles as a contiguous copy, the barrier its own.
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t scales,
                                             const uint8_t *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "{\n"
        ".reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%7];\n"
        "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%4], [%5], %6, [%7];\n"
        "}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(scales), "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
// One lane arms `bar` for `bytes`, if `here`.  Warp-collective.
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes, bool here) {
    asm volatile(
        "{\n"
        ".reg .pred e, q;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.and.u32 q, %2, 0, e;\n"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
        "}\n" ::"r"(bar),
        "r"(bytes), "r"((uint32_t)here)
        : "memory");
}
// Arrives on another CTA's barrier (a shared::cluster address).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Starts the fetch of a tensor map (a kernel parameter) that a load will soon use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster meets; writes before the arrival are seen
// after the wait.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The address of `saddr` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

}  // namespace tc
}  // namespace gdn
