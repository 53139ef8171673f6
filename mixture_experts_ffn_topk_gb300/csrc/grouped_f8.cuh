// grouped_f8.cuh -- what the two forms of the 8-bit grouped product share.
#pragma once

#include <cfloat>

#include "common.cuh"
#include "grouped_issue.cuh"
#include "grouped_units.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int BK = 128;                  // k per stage: 128 bytes, one block of scales
constexpr int UK = 32;                   // k per tcgen05.mma
constexpr int W_BYTES = BM * BK;         // 16 KiB
constexpr uint64_t kDrainLimitNs = 100000000ull;

// D (+)= A B^T of one K = 32 step of e4m3 operands.
template <int CG>
__device__ __forceinline__ void umma_f8_on(uint32_t on, uint32_t d, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%1], %2, %3, %4, p;\n\t}" ::"r"(on),
            "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%1], %2, %3, %4, p;\n\t}" ::"r"(on),
            "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Arrives on a barrier of either CTA of the pair, given by its cluster address. Not
// a release: the barrier orders tensor memory alone, and tcgen05 fences on both
// sides do that; a release at cluster scope, a full memory barrier, cost a
// microsecond per block of k, and one at CTA scope some 100 cycles.
__device__ __forceinline__ void arrive_relaxed_on(uint32_t on, uint32_t cluster_addr)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
        "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%1];\n\t}" ::"r"(on),
        "r"(cluster_addr)
        : "memory");
}

// Instruction descriptor, kind::f8f6f4: FP32 accumulator, A and B e4m3 (0), MN-major
// where a_mn or b_mn (bits 15 and 16), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// warp_wait on two barriers whose phases may well be complete: both are asked at once.
__device__ __forceinline__ bool warp_wait_both(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb,
                                               volatile int *abort_flag, unsigned *status, uint64_t limit_ns)
{
    const bool ok_a = mbar_try_wait(a, pa), ok_b = mbar_try_wait(b, pb);
    if (__all_sync(0xffffffffu, ok_a && ok_b)) return true;
    return warp_wait<1>(a, pa, abort_flag, status, limit_ns) && warp_wait<1>(b, pb, abort_flag, status, limit_ns);
}

// A block's two scales as one number s and a power of two k, so that (v k) s is v times
// both, rounded once, where v is a block's sum: 0, or 2^-18 (the least product of two
// codes) to 2^25 in magnitude. k is 1 where a w is a normal number, or 0 because a scale
// is. A product below 2^-126 comes 2^100 times too large with k = 2^-100, one above
// FP32's largest the other way round: v k is exact and normal in both. From 2^228 on
// s is FP32's largest: (v k) s is infinite with all v but 0, as it should be.
// Returns -1, 0 or 1 for the three k.
constexpr float kScaleUp = 1.2676506002282294e30f, kScaleDown = 7.888609052210118e-31f;  // 2^100, 2^-100

__device__ __forceinline__ int scales_apart(float a, float w, float &s)
{
    s = a * w;
    const float lo = fabsf(a) < fabsf(w) ? a : w, hi = fabsf(a) < fabsf(w) ? w : a;
    if (fabsf(s) < FLT_MIN && lo != 0.0f) {
        s = (lo * kScaleUp) * hi;
        return -1;
    }
    if (isinf(s) && !isinf(hi)) {
        s = fminf(fmaxf((hi * kScaleDown) * lo, -FLT_MAX), FLT_MAX);
        return 1;
    }
    return 0;
}

__device__ __forceinline__ float shift_of(int which) { return which == 0 ? 1.0f : which < 0 ? kScaleDown : kScaleUp; }

// Whether the product of any two such scales is a normal number: 2^-63 <= |v| < 2^63.
__device__ __forceinline__ bool plain_scale(float v)
{
    return (__float_as_uint(v) << 1) - (64u << 24) < (126u << 24);
}

// 4 bytes of global memory into shared memory, asynchronously.
__device__ __forceinline__ void copy4_async(float *dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Bytes, row-major, of two or three dimensions, in boxes of 128 bytes by box_rows.
bool encode_bytes(CUtensorMap *m, const void *base, int rank, const uint64_t (&dims)[3],
                  const uint64_t (&strides)[2], uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t d[3] = {dims[0], dims[1], dims[2]}, st[2] = {strides[0], strides[1]};
    cuuint32_t box[3] = {128, box_rows, 1}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(base), d, st, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe
