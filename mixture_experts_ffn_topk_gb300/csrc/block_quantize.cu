// block_quantize.cu -- rows, expert matrices and SwiGLU activations in 8 bits with
// an FP32 scale per block of 128 columns (matrices: 128 x 128).
//
// With m the largest magnitude of a block's finite values, 2^-100 at least:
// scale s = m / 448 (448 is e4m3's largest), and a value v is stored as
// e4m3(v * (448 / m)), round to nearest even. The product is off by at most
// 2^-23 of itself (the quotient's rounding and its own), so code * s lies within
// (2^-4 + 2^-22) |v| of v, or 2^-10 s where the code is subnormal. 2^-100 keeps
// 448 / m finite; below it codes shrink instead of the scale, and the error stays
// within 2^-10 s. Infinities and NaN are stored as e4m3's NaN and take no part in m.
// SwiGLU: v = g / (1 + exp(-g)) * u in FP32, not rounded before.
//
// All are bound by HBM: 3 bytes per 16-bit value (SwiGLU 5). Sixteen lanes share a
// row's block, 8 columns each: 16-byte loads of 16-bit rows, 8-byte stores of
// codes, four shuffles for the maximum. What is left next to HBM is instructions: the
// divisions of a thread's blocks, 448 / m and m / 448, are one, spread over lanes
// (SwiGLU, 32767 x 14336 in BF16: 458 -> 380 us; 6 CTAs per SM: 368 us, 95 % of the
// copy bandwidth; 24576 x 1408: 33 us, 78 %). A matrix's block is one CTA's, 64
// values per thread in registers between the maximum and the codes (64 x 1408 x
// 2048: 91 us, 90 %).
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kBlock = 128;
constexpr int kLanes = kBlock / kLaneCols;
constexpr float kTopLeast = 7.888609052210118e-31f;      // 2^-100
// Blocks a thread has in flight at once (SwiGLU, as above: 1 398, 2 381, 3 419, 4 433 us).
constexpr int kItems = 2;
constexpr int kMatrixRows = kBlock / (kRowThreads / kLanes);     // rows of a block per thread

// A lane's eight columns of a block: consecutive where rows are read in vectors,
// else every 16th, so that the lanes' elements are neighbours.
template <bool VEC>
__device__ __forceinline__ int column(int lane, int i)
{
    return VEC ? lane * kLaneCols + i : lane + i * kLanes;
}

// Of the row's block at `row` (left columns to its end; 0 or less: none).
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> load_columns(const void *row, int lane, int left)
{
    if constexpr (VEC) {
        return load8<DT, true>(row, lane * kLaneCols, left - lane * kLaneCols);
    } else {
        using T = typename Elem<DT>::T;
        Raw8<DT> r;
#pragma unroll
        for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) r.q[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (column<false>(lane, i) < left)
                reinterpret_cast<T *>(&r)[i] = static_cast<const T *>(row)[column<false>(lane, i)];
        return r;
    }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t *row, int lane, int left, uint2 c)
{
    if (VEC && left >= (lane + 1) * kLaneCols) {
        __stcs(reinterpret_cast<uint2 *>(row + lane * kLaneCols), c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (column<VEC>(lane, i) < left)
                row[column<VEC>(lane, i)] = (uint8_t)((i < 4 ? c.x : c.y) >> (i & 3) * 8);
    }
}

// Largest finite magnitude of eight values (a maximum passes over NaN; INF: and
// over infinities).
template <bool INF>
__device__ __forceinline__ float top_of(const float (&v)[8])
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (!INF || fabsf(v[i]) != INFINITY) top = fmaxf(top, fabsf(v[i]));
    return top;
}

// Largest of the sixteen lanes of a block; of numbers >= 0, not NaN.
__device__ __forceinline__ float block_max(float v)
{
    uint32_t m = __float_as_uint(v);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __uint_as_float(m);
}

// r: 448 over the block's largest finite magnitude; odd: some value may be infinite.
__device__ __forceinline__ uint2 encode(const float (&v)[8], float r, bool odd)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = make_float2(v[2 * i] * r, v[2 * i + 1] * r);
        if (odd) {
            // the conversion saturates infinities; they are to come back as NaN
            if (isinf(v[2 * i])) f.x = __uint_as_float(0x7fffffffu);
            if (isinf(v[2 * i + 1])) f.y = __uint_as_float(0x7fffffffu);
        }
        c[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// SiLU(g) u. FP32 rows take the full exponential and division; 16-bit ones the
// hardware's approximations (relative errors of about 2^-21 (1 + |g|)), which
// take 1 / (1 + exp(-g)) below 2^-126 for 0.
template <int DT>
__device__ __forceinline__ float swiglu(float g, float u)
{
    if constexpr (DT == DT_F32) return g / (1.0f + expf(-g)) * u;
    float z, t;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(1.0f + z));
    return g * t * u;
}

// SWIGLU: the rows are g's, and the values SiLU(g) u. All lanes of a warp stay
// together: the shuffles always have every lane.
template <int DT, bool VEC, bool SWIGLU>
__global__ void __launch_bounds__(kRowThreads, DT == DT_F32 ? 3 : 6)
quantize_rows_kernel(const void *__restrict__ g, const void *__restrict__ u, int64_t ld_bytes, int K,
                     Walk w, uint8_t *__restrict__ codes, int64_t ldc, float *__restrict__ scales)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t rows = rows_to_do(w);
    const int lane = threadIdx.x & (kLanes - 1);
    Place at = first_place<kLanes>(w);
    while (__any_sync(0xffffffffu, at.row < rows)) {
        Place p[kItems];
        Raw8<DT> a[kItems], b[SWIGLU ? kItems : 1];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            p[k] = at;
            at.advance(w);
            const int left = p[k].row < rows ? K - p[k].blk * kBlock : 0;
            const int64_t off = left > 0 ? p[k].row * ld_bytes + (int64_t)p[k].blk * kBlock * sizeof(typename Elem<DT>::T) : 0;
            a[k] = load_columns<DT, VEC>(static_cast<const uint8_t *>(g) + off, lane, left);
            if constexpr (SWIGLU) b[k] = load_columns<DT, VEC>(static_cast<const uint8_t *>(u) + off, lane, left);
        }
        float v[kItems][8], m[kItems];
        bool odd[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = SWIGLU ? swiglu<DT>(a[k].at(i), b[SWIGLU ? k : 0].at(i)) : a[k].at(i);
            m[k] = block_max(top_of<false>(v[k]));
            odd[k] = __any_sync(0xffffffffu, m[k] == INFINITY);      // rare
            if (odd[k]) m[k] = block_max(top_of<true>(v[k]));
            m[k] = fmaxf(m[k], kTopLeast);
        }
        // one division for all: lane k of a block's sixteen has 448 / m of item k, lane
        // kItems + k the scale m / 448
        float top = m[0];
#pragma unroll
        for (int k = 1; k < kItems; ++k) top = lane % kItems == k ? m[k] : top;
        const float quotient = (lane < kItems ? 448.0f : top) / (lane < kItems ? top : 448.0f);
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const float r = __shfl_sync(0xffffffffu, quotient, k, kLanes);
            if (p[k].row >= rows) continue;
            store_codes<VEC>(codes + p[k].row * ldc + (int64_t)p[k].blk * kBlock, lane,
                             K - p[k].blk * kBlock, encode(v[k], r, odd[k]));
            if (lane == kItems + k) scales[p[k].row * w.S + p[k].blk] = quotient;
        }
    }
}

// One CTA per block of 128 x 128; blocks run along a matrix's rows first.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kRowThreads, DT == DT_F32 ? 2 : 4)
quantize_matrices_kernel(const void *__restrict__ w, int64_t N, int64_t K, int64_t n_blocks,
                         int64_t k_blocks, uint8_t *__restrict__ codes, float *__restrict__ scales)
{
    __shared__ uint32_t warp_top[kRowThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t kb = blockIdx.x % k_blocks, nb = blockIdx.x / k_blocks % n_blocks,
                  e = blockIdx.x / k_blocks / n_blocks;
    const int lane = threadIdx.x & (kLanes - 1), first = threadIdx.x / kLanes;
    const int left = (int)(K - kb * kBlock < kBlock ? K - kb * kBlock : kBlock);
    const int tall = (int)(N - nb * kBlock < kBlock ? N - nb * kBlock : kBlock);
    const int64_t at = (e * N + nb * kBlock) * K + kb * kBlock;
    Raw8<DT> a[kMatrixRows];
#pragma unroll
    for (int j = 0; j < kMatrixRows; ++j) {
        const int r = first + j * (kRowThreads / kLanes);
        a[j] = load_columns<DT, VEC>(static_cast<const typename Elem<DT>::T *>(w) + at + (r < tall ? r * K : 0),
                                     lane, r < tall ? left : 0);
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kMatrixRows; ++j) top = max(top, top8<DT, false>(a[j]));
    auto over_all = [&](uint32_t v) {
        v = __reduce_max_sync(0xffffffffu, v);
        if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x / 32] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowThreads / 32; ++i) v = max(v, warp_top[i]);
        return v;
    };
    top = over_all(top);
    const bool odd = top >= 0x7f800000u;                 // the same in all threads
    if (odd) {
        top = 0;
#pragma unroll
        for (int j = 0; j < kMatrixRows; ++j) top = max(top, top8<DT, true>(a[j]));
        __syncthreads();
        top = over_all(top);
    }
    const float m = fmaxf(__uint_as_float(top), kTopLeast);
#pragma unroll
    for (int j = 0; j < kMatrixRows; ++j) {
        const int r = first + j * (kRowThreads / kLanes);
        if (r >= tall) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = a[j].at(i);
        store_codes<VEC>(codes + at + r * K, lane, left, encode(v, 448.0f / m, odd));
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = m / 448.0f;
}

bool rows8(const void *p, int64_t ld_bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 7u) == 0 && ld_bytes % 8 == 0;
}

template <int DT, bool SWIGLU>
cudaError_t rows_dt(const void *g, const void *u, int64_t ld, int64_t rows, int64_t K, const int32_t *end,
                    uint8_t *codes, int64_t ldc, float *scales, cudaStream_t s)
{
    const int64_t eb = sizeof(typename Elem<DT>::T);
    unsigned grid;
    const Walk w = make_walk<kLanes>(rows, K, end, &grid);
    const bool vec = rows16(g, ld * eb) && (!SWIGLU || rows16(u, ld * eb)) && rows8(codes, ldc);
    auto k = vec ? quantize_rows_kernel<DT, true, SWIGLU> : quantize_rows_kernel<DT, false, SWIGLU>;
    return launch_pdl(k, dim3(grid), dim3(kRowThreads), 0, s, g, u, ld * eb, (int)K, w, codes, ldc, scales);
}

template <int DT>
cudaError_t matrices_dt(const void *w, int64_t E, int64_t N, int64_t K, uint8_t *codes, float *scales,
                        cudaStream_t s)
{
    const int64_t eb = sizeof(typename Elem<DT>::T);
    const int64_t nb = (N + kBlock - 1) / kBlock, kb = (K + kBlock - 1) / kBlock;
    const bool vec = rows16(w, K * eb) && rows8(codes, K);
    auto k = vec ? quantize_matrices_kernel<DT, true> : quantize_matrices_kernel<DT, false>;
    return launch_pdl(k, dim3((unsigned)(E * nb * kb)), dim3(kRowThreads), 0, s, w, N, K, nb, kb, codes, scales);
}

}  // namespace

cudaError_t launch_quantize_rows(int dt, const void *x, int64_t ld, const int32_t *end, int64_t rows,
                                 int64_t K, uint8_t *codes, int64_t ldc, float *scales, cudaStream_t s)
{
    if (dt == DT_F32) return rows_dt<DT_F32, false>(x, nullptr, ld, rows, K, end, codes, ldc, scales, s);
    if (dt == DT_BF16) return rows_dt<DT_BF16, false>(x, nullptr, ld, rows, K, end, codes, ldc, scales, s);
    return rows_dt<DT_F16, false>(x, nullptr, ld, rows, K, end, codes, ldc, scales, s);
}

cudaError_t launch_swiglu_quantize(int dt, const void *g, const void *u, int64_t ld, const int32_t *end,
                                   int64_t rows, int64_t I, uint8_t *codes, int64_t ldc, float *scales,
                                   cudaStream_t s)
{
    if (dt == DT_F32) return rows_dt<DT_F32, true>(g, u, ld, rows, I, end, codes, ldc, scales, s);
    if (dt == DT_BF16) return rows_dt<DT_BF16, true>(g, u, ld, rows, I, end, codes, ldc, scales, s);
    return rows_dt<DT_F16, true>(g, u, ld, rows, I, end, codes, ldc, scales, s);
}

cudaError_t launch_quantize_weights(int dt, const void *w, int64_t E, int64_t N, int64_t K,
                                    uint8_t *codes, float *scales, cudaStream_t s)
{
    if (dt == DT_F32) return matrices_dt<DT_F32>(w, E, N, K, codes, scales, s);
    if (dt == DT_BF16) return matrices_dt<DT_BF16>(w, E, N, K, codes, scales, s);
    return matrices_dt<DT_F16>(w, E, N, K, codes, scales, s);
}

}  // namespace moe
