// tc_bf16_ptx.cuh -- inline-PTX wrappers for the bf16 products of the feed-forward block: a
// stage's loads and MMAs, of one CTA or of a pair (cta_group::2), each in one go.
//
// A stage is 64 of the contraction.  An operand tile of 128 rows is 16 KB: K-major, rows of 64
// elements (128 bytes, 128-byte swizzle); or, of a matrix whose rows run along the contraction
// (MN-major), two blocks of 64 contraction rows x 64 elements, 8 KB each.
#pragma once

#include "tc_mx_ptx.cuh"

namespace gdn {
namespace tc {

// Descriptors of a tile, and what 16 of the contraction add to them (in units of 16 bytes).
template <bool MN>
__device__ __forceinline__ uint64_t desc_tile(uint32_t saddr) {
    return MN ? desc_sw128(saddr, 8192, 1024) : desc_sw128(saddr, 0, 1024);
}
template <bool MN>
constexpr int kStepOf = MN ? 128 : 2;

// The four MMAs of a stage, and the arrival on `bar` (of both CTAs of a pair) when they are done.
// Warp-collective: one election for the stage.
template <bool A_MN, bool B_MN, bool PAIR>
__device__ __forceinline__ void mma_bf16_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                               uint64_t *bar) {
    constexpr int kA = kStepOf<A_MN>, kB = kStepOf<B_MN>;
    if (PAIR)
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            ".reg .b64 a1, a2, a3, b1, b2, b3;\n"
            "setp.ne.b32 p, %4, 0;\n"
            "add.s64 a1, %1, %7;\n add.s64 a2, a1, %7;\n add.s64 a3, a2, %7;\n"
            "add.s64 b1, %2, %8;\n add.s64 b2, b1, %8;\n add.s64 b3, b2, %8;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, 1;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, 1;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, 1;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], %6;\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar)), "h"((uint16_t)3), "n"(kA), "n"(kB)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p, e;\n"
            ".reg .b64 a1, a2, a3, b1, b2, b3;\n"
            "setp.ne.b32 p, %4, 0;\n"
            "add.s64 a1, %1, %6;\n add.s64 a2, a1, %6;\n add.s64 a3, a2, %6;\n"
            "add.s64 b1, %2, %7;\n add.s64 b2, b1, %7;\n add.s64 b3, b2, %7;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
            "}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar)), "n"(kA), "n"(kB)
            : "memory");
}

// One box into this CTA's shared memory, completing on `bar`: of the pair's CTA that issues (a
// shared::cluster address), or its own.  Warp-collective.
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    if (PAIR)
        asm volatile(
            "{\n"
            ".reg .pred e;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3}], [%4];\n"
            "}\n" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred e;\n"
            "elect.sync _|e, 0xffffffff;\n"
            "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];\n"
            "}\n" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
// ROWS (64 or 128) of an operand from `row` on, contraction k .. k + 63.
template <bool MN, bool PAIR, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int row, int k, uint32_t bar) {
    if (MN) {
        load_box<PAIR>(dst, map, row, k, bar);
        if (ROWS == 128) load_box<PAIR>(dst + 8192, map, row + 64, k, bar);
    } else {
        load_box<PAIR>(dst, map, k, row, bar);
    }
}

}  // namespace tc
}  // namespace gdn
