// rows8.cuh -- what the kernels that quantize rows in blocks of columns share: eight
// columns of a row per lane, neighbouring lanes to a block, and a walk over the
// blocks of all rows.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kLaneCols = 8;     // columns a lane handles
constexpr int kRowThreads = 256; // threads of a CTA

// Item = one block of one row; a thread walks items first, first + step, ...
// as (row, blk) pairs without dividing: step = step_row * S + step_blk.
struct Walk {
    int64_t rows;            // rows of the call
    int S;                   // blocks per row
    int64_t step_row;
    int step_blk;
    const int32_t *end;      // offsets + E (rows from *end on are left alone), or nullptr
};

__device__ __forceinline__ int64_t rows_to_do(const Walk &w)
{
    if (w.end == nullptr) return w.rows;
    const int64_t e = *w.end;
    return e < 0 ? 0 : (e < w.rows ? e : w.rows);
}

// Eight consecutive columns of a row as they are stored.
template <int DT>
struct Raw8 {
    uint4 q[DT == DT_F32 ? 2 : 1];

    __device__ __forceinline__ float at(int i) const
    {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
        if constexpr (DT == DT_F32) return __uint_as_float(w[i]);
        const uint32_t h = w[i >> 1];
        if constexpr (DT == DT_BF16) return __uint_as_float(i & 1 ? h & 0xffff0000u : h << 16);
        return __half2float(__ushort_as_half((unsigned short)(i & 1 ? h >> 16 : h)));
    }
};

// VEC: rows start on 16 bytes. A piece that is not whole (the end of a row, or
// any piece without VEC) is read by element; columns past `left` read 0.
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> load8(const void *row, int col, int left)
{
    using T = typename Elem<DT>::T;
    const T *p = static_cast<const T *>(row) + col;
    Raw8<DT> r;
    if (VEC && left >= 8) {
#pragma unroll
        for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) r.q[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) r.q[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) reinterpret_cast<T *>(&r)[i] = p[i];
    }
    return r;
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(void *row, int col, int left, const float (&v)[8])
{
    using T = typename Elem<DT>::T;
    T *p = static_cast<T *>(row) + col;
    if (VEC && left >= 8) {
        if constexpr (DT == DT_F32) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            Vec16 q;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q.w[i] = DT == DT_BF16 ? float2_to_bf16x2(v[2 * i], v[2 * i + 1])
                                       : float2_to_f16x2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(p) = q.u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = Elem<DT>::from_f(v[i]);
    }
}

// t = 1 / (1 + exp(-g)) and 1 - t, from z = exp(-|g|) <= 1: nothing overflows,
// and where t is tiny it fades through FP32's subnormals instead of dropping
// to 0 at exp(89). FP32 outputs take the full exponential and division; the
// 16-bit ones the hardware's approximations (errors of about 2^-21 (1 + |g|), far
// below their rounding), of exp(-|g| / 2), whose square fades as it should
// where the approximation itself, which knows no subnormals, would be 0.
template <int DT>
__device__ __forceinline__ void sigmoid_of(float g, float &t, float &not_t)
{
    float z, r;
    if constexpr (DT == DT_F32) {
        z = expf(-fabsf(g));
        r = 1.0f / (1.0f + z);
    } else {
        float w;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fabsf(g) * -0.72134752f));   // -log2(e) / 2
        z = w * w;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + z));
    }
    const float zr = z * r;
    t = g >= 0.0f ? r : zr;
    not_t = g >= 0.0f ? zr : r;
}

// Largest magnitude of this lane's eight values as FP32 bits; FINITE: of the
// finite ones only. 16-bit values are compared two at a time.
template <int DT, bool FINITE>
__device__ __forceinline__ uint32_t top8(const Raw8<DT> &v)
{
    if constexpr (DT == DT_F32 || FINITE) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = __float_as_uint(v.at(i)) & 0x7fffffffu;
            top = max(top, !FINITE || a < 0x7f800000u ? a : 0u);
        }
        return top;
    } else {
        constexpr uint32_t M = 0x7fff7fffu;
        uint32_t m = __vimax3_u16x2(v.q[0].x & M, v.q[0].y & M, v.q[0].z & M);
        m = __vimax3_u16x2(m, v.q[0].w & M, m);
        m = max(m & 0xffffu, m >> 16);
        if constexpr (DT == DT_BF16) return m << 16;
        // F16 infinities and NaN stay at or above FP32's infinity
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    }
}

// Where a thread is in the walk.
struct Place {
    int64_t row;
    int blk;

    __device__ __forceinline__ void advance(const Walk &w)
    {
        row += w.step_row;
        blk += w.step_blk;
        if (blk >= w.S) { blk -= w.S; ++row; }
    }
};

// LANES: lanes of a block.
template <int LANES>
__device__ __forceinline__ Place first_place(const Walk &w)
{
    const int64_t item = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) / LANES;
    Place p;
    p.row = item / w.S;
    p.blk = (int)(item - p.row * w.S);
    return p;
}

// At least 8 CTAs per SM (the whole work, if less), more where each thread
// would walk over 16 blocks: with 4 lanes to a block, 32768 x
// 14336 values took the SwiGLU checkpoint 645, 637 and 634 us at 8, 16 and 64 per
// SM (its backward 769, 760, 743), 24576 x 1408 53, 57, 60.
template <int LANES>
Walk make_walk(int64_t rows, int64_t I, const int32_t *end, unsigned *grid)
{
    Walk w;
    w.rows = rows;
    w.S = (int)((I + LANES * kLaneCols - 1) / (LANES * kLaneCols));
    w.end = end;
    const int64_t per = kRowThreads / LANES, items = rows * w.S;
    const int64_t want = (items + per - 1) / per, fill = (int64_t)device_sm_count() * 8;
    int64_t n = want / 16 > fill ? want / 16 : want < fill ? want : fill;
    if (n > 0x7fffffff) n = 0x7fffffff;
    *grid = (unsigned)n;
    const int64_t step = n * per;
    w.step_row = step / w.S;
    w.step_blk = (int)(step % w.S);
    return w;
}

bool rows16(const void *p, int64_t ld_bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld_bytes % 16 == 0;
}

}  // namespace
}  // namespace moe
