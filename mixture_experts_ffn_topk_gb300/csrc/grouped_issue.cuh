// grouped_issue.cuh -- how the grouped products' tensor-core roles issue.
//
// A role keeps its whole warp in its loop, and every issue is one instruction
// predicated on a lane elected once (`on`). No branch diverges, so addresses,
// coordinates and descriptors stay in uniform registers; a loop run by one
// lane alone moves each operand there again for every instruction, which cost
// about 60 cycles per tcgen05.mma and 140 per TMA copy where a stage's four
// MMAs take 512.
#pragma once

#include "tc_ptx.cuh"

namespace moe {
namespace {

// 1 in one lane of a converged warp, always the same one.
__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

// Waits with the whole warp; true in every lane or in none.
template <int CG>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                          unsigned *status, uint64_t limit_ns)
{
    return __all_sync(0xffffffffu, mbar_wait<CG>(bar, parity, abort_flag, status, limit_ns));
}

__device__ __forceinline__ void expect_tx_on(uint32_t on, uint64_t *bar, uint32_t bytes)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
        "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], %2;\n\t}" ::"r"(on),
        "r"(smem_u32(bar)), "r"(bytes)
        : "memory");
}

__device__ __forceinline__ void arrive_on(uint32_t on, uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"(on),
        "r"(smem_u32(bar))
        : "memory");
}

// TMA copies into this CTA's shared memory, completing on the barrier at the
// shared-memory address `bar` (on a pair a cluster address, of either CTA).
template <int CG>
__device__ __forceinline__ void load_2d_on(uint32_t on, uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                           int c0, int c1)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
            "@p cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%1], [%2, {%4, %5}], [%3];\n\t}" ::"r"(on),
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
            "@p cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%1], [%2, {%4, %5}], [%3];\n\t}" ::"r"(on),
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void load_3d_on(uint32_t on, uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                           int c0, int c1, int c2)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
            "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%1], [%2, {%4, %5, %6}], [%3];\n\t}" ::"r"(on),
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
            "@p cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%1], [%2, {%4, %5, %6}], [%3];\n\t}" ::"r"(on),
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// D (+)= A B^T of one K = 16 step (see umma_f16).
template <int CG>
__device__ __forceinline__ void umma_on(uint32_t on, uint32_t d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(on),
            "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(on),
            "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// The MMAs issued so far arrive on this barrier when done (on a pair, on the
// barrier at this offset in both CTAs).
template <int CG>
__device__ __forceinline__ void commit_on(uint32_t on, uint64_t *bar)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
            "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%1], %2;\n\t}" ::"r"(
                on),
            "r"(smem_u32(bar)), "h"((uint16_t)0x3)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
            "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(on),
            "r"(smem_u32(bar))
            : "memory");
}

// 32 TMEM lanes x 16 (32) consecutive fp32 columns, written; tmem_st_wait() before
// they are read again.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 "
        "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 "
        "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Failure path only: gives this CTA's TMA copies a bounded time to land before
// its shared memory goes.
__device__ __forceinline__ void let_copies_land()
{
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000000ull) { }
}

}  // namespace
}  // namespace moe
