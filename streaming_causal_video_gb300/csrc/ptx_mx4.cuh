// Inline-PTX spellings for products of microscaled 4-bit matrices by CTA pairs.  Each function is one instruction
// or one ring stage's block of them, issued by an elected lane of a converged warp where its name says so.
#pragma once
#include <cuda.h>
#include <cstdint>

#include "tmem_io.cuh"

namespace sdv2 {

// Instruction descriptor of kind::mxf4: A and B e2m1 (1, at bits 7 and 10), scales ue8m0 (bit 23), N/8 at bit 17, M/128 at bit
// 27; `half` selects the upper two of the four scale bytes that a tensor-memory cell holds (ids 0 or 2 at bits 4 and 29).
__host__ __device__ constexpr uint32_t idesc_mx4(int M, int N, int half)
{
    return (static_cast<uint32_t>(2 * half) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 7) << 27) | (static_cast<uint32_t>(2 * half) << 29);
}

// Shared-memory descriptor of 128 rows' scales for 128 columns (512 bytes, no swizzle): 8 rows of 16 bytes lie 128 bytes
// behind the 8 before them.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// A ring stage's copies: codes of a and b (columns `k` of rows `ra`, `rb`) and their scales (from scale tile `t` of row tiles `sa`,
// `sb`) to `to` and the places behind it, counted on the barrier `full` of the pair's leader, which arms its own barrier `mine`
// for `bytes` before.  One block of instructions with one election, as what bounds small tiles is how fast a thread issues them:
// with the four copies issued by a thread on its own, a stage takes 290 ns whatever its size, with this 200 at 128 rows of b.
__device__ __forceinline__ void mx4_load_pair_warp(bool leads, uint32_t mine, uint32_t bytes, uint32_t full, const CUtensorMap* a, const CUtensorMap* b,
                                                   const CUtensorMap* as, const CUtensorMap* bs, uint32_t to_a, uint32_t to_b, uint32_t to_as,
                                                   uint32_t to_bs, int k, int ra, int rb, int t, int sa, int sb)
{
    asm volatile(
        "{\n\t.reg .pred e, f;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.and.b32 f, %0, 0, e;\n\t"
        "@f mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], %2;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%8], [%4, {%12, %13, %18}], [%3];\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%9], [%5, {%12, %14, %18}], [%3];\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%10], [%6, {%18, %15, %16}], [%3];\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%11], [%7, {%18, %15, %17}], [%3];\n\t}" ::"r"(
            static_cast<int>(leads)),
        "r"(mine), "r"(bytes), "r"(full), "l"(reinterpret_cast<uint64_t>(a)), "l"(reinterpret_cast<uint64_t>(b)), "l"(reinterpret_cast<uint64_t>(as)),
        "l"(reinterpret_cast<uint64_t>(bs)), "r"(to_a), "r"(to_b), "r"(to_as), "r"(to_bs), "r"(k), "r"(ra), "r"(rb), "r"(t), "r"(sa), "r"(sb), "r"(0)
        : "memory");
}

// The same within one CTA (4 rows at 1536 x 1536 3.6 us with a thread on its own, 3.0 with this).
__device__ __forceinline__ void mx4_load_warp(uint32_t full, uint32_t bytes, const CUtensorMap* a, const CUtensorMap* b, const CUtensorMap* as,
                                              const CUtensorMap* bs, uint32_t to_a, uint32_t to_b, uint32_t to_as, uint32_t to_bs, int k, int ra, int rb,
                                              int t, int sa, int sb)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%6], [%2, {%10, %11, %16}], [%0];\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%7], [%3, {%10, %12, %16}], [%0];\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%8], [%4, {%16, %13, %14}], [%0];\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%9], [%5, {%16, %13, %15}], [%0];\n\t}" ::"r"(full),
        "r"(bytes), "l"(reinterpret_cast<uint64_t>(a)), "l"(reinterpret_cast<uint64_t>(b)), "l"(reinterpret_cast<uint64_t>(as)),
        "l"(reinterpret_cast<uint64_t>(bs)), "r"(to_a), "r"(to_b), "r"(to_as), "r"(to_bs), "r"(k), "r"(ra), "r"(rb), "r"(t), "r"(sa), "r"(sb), "r"(0)
        : "memory");
}

// One ring stage, 256 columns, issued by one elected lane: the scales of both scale tiles of a and of b's one or two row tiles go from each
// CTA's shared memory to its own tensor memory (a: 4 columns a tile; b: 8), and four MMAs over the pair add 64 columns each to
// the sums.  One block of instructions with one election, as a single thread issues them all.
//   a, b: descriptors of the codes, a row's 64 columns 32 bytes apart; as, bs: of the scales, tiles 512 bytes apart, b's second
//   row tile 1024; i0, i1: instruction descriptors for the first and the second half of a scale tile
template <int ROW_TILES>
__device__ __forceinline__ void mx4_stage_pair_warp(uint32_t sums, uint64_t a, uint64_t b, uint64_t as, uint64_t bs, uint32_t a_scales,
                                                    uint32_t b_scales, uint32_t b_first, uint32_t i0, uint32_t i1, uint32_t accumulate)
{
    if constexpr (ROW_TILES == 2) {
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t"
            ".reg .b64 x, y;\n\t"
            ".reg .b32 t, u;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %10, 0;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], %3;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%6], %4;\n\t"
            "add.s32 t, %6, 4;\n\t"
            "add.s64 x, %4, 64;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], x;\n\t"
            "add.s32 t, %5, 4;\n\t"
            "add.s64 x, %3, 32;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], x;\n\t"
            "add.s32 u, %6, 8;\n\t"
            "add.s64 x, %4, 32;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [u], x;\n\t"
            "add.s32 u, %6, 12;\n\t"
            "add.s64 x, %4, 96;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [u], x;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %8, [%5], [%7], p;\n\t"
            "add.s64 x, %1, 2;\n\t"
            "add.s64 y, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %9, [%5], [%7], 1;\n\t"
            "add.s64 x, %1, 4;\n\t"
            "add.s64 y, %2, 4;\n\t"
            "add.s32 u, %7, 8;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %8, [t], [u], 1;\n\t"
            "add.s64 x, %1, 6;\n\t"
            "add.s64 y, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %9, [t], [u], 1;\n\t}" ::"r"(sums),
            "l"(a), "l"(b), "l"(as), "l"(bs), "r"(a_scales), "r"(b_scales), "r"(b_first), "r"(i0), "r"(i1), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t"
            ".reg .b64 x, y;\n\t"
            ".reg .b32 t, u;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %10, 0;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%5], %3;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%6], %4;\n\t"
            "add.s32 t, %5, 4;\n\t"
            "add.s64 x, %3, 32;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], x;\n\t"
            "add.s32 u, %6, 8;\n\t"
            "add.s64 x, %4, 32;\n\t"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [u], x;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %8, [%5], [%7], p;\n\t"
            "add.s64 x, %1, 2;\n\t"
            "add.s64 y, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %9, [%5], [%7], 1;\n\t"
            "add.s64 x, %1, 4;\n\t"
            "add.s64 y, %2, 4;\n\t"
            "add.s32 u, %7, 8;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %8, [t], [u], 1;\n\t"
            "add.s64 x, %1, 6;\n\t"
            "add.s64 y, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %9, [t], [u], 1;\n\t}" ::"r"(sums),
            "l"(a), "l"(b), "l"(as), "l"(bs), "r"(a_scales), "r"(b_scales), "r"(b_first), "r"(i0), "r"(i1), "r"(accumulate)
            : "memory");
    }
}

// The same within one CTA, of 128 rows of a and few rows of b, whose scales are one row tile's as well (4 columns a tile).
__device__ __forceinline__ void mx4_stage_warp(uint32_t sums, uint64_t a, uint64_t b, uint64_t as, uint64_t bs, uint32_t a_scales, uint32_t b_scales,
                                               uint32_t i0, uint32_t i1, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        ".reg .b64 x, y;\n\t"
        ".reg .b32 t, u;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %9, 0;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], %3;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%6], %4;\n\t"
        "add.s32 t, %5, 4;\n\t"
        "add.s64 x, %3, 32;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [t], x;\n\t"
        "add.s32 u, %6, 4;\n\t"
        "add.s64 x, %4, 32;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [u], x;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %7, [%5], [%6], p;\n\t"
        "add.s64 x, %1, 2;\n\t"
        "add.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %8, [%5], [%6], 1;\n\t"
        "add.s64 x, %1, 4;\n\t"
        "add.s64 y, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %7, [t], [u], 1;\n\t"
        "add.s64 x, %1, 6;\n\t"
        "add.s64 y, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %8, [t], [u], 1;\n\t}" ::"r"(sums),
        "l"(a), "l"(b), "l"(as), "l"(bs), "r"(a_scales), "r"(b_scales), "r"(i0), "r"(i1), "r"(accumulate)
        : "memory");
}

// Bytes that a barrier of this CTA was told to expect and that no copy will bring.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t cluster_addr, int32_t v)
{
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Box from shared memory to global memory; rows and columns past the tensor's end are not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1, int32_t c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// 16 or 32 columns of this thread's lane, and waits for them.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_x16_sync(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_x32_sync(taddr, r); }

}  // namespace sdv2
