// swiglu_checkpoint.cu -- SwiGLU with an 8-bit checkpoint, and its backward.
//
// Forward, per value: h = SiLU(g) * u = g / (1 + exp(-g)) * u in FP32, rounded
// once to the rows' dtype, and g and u kept in 8 bits for the backward: a block
// of 32 columns of a row shares the smallest power of two s = 2^x, -127 <= x <=
// 119, with max |v| <= 448 s over its finite values (448 is e4m3's largest);
// each value is stored as e4m3(v / s), round to nearest even, and x + 127 as a
// byte. v / s is exact (a change of exponent; what falls below FP32's normal
// range is far below e4m3's smallest step), so a value is rounded once, by at
// most 2^-4 of itself or 2^-10 s. Infinities and NaN are stored as e4m3's NaN and take
// no part in the block's scale. x stops at 119 because 256 * 2^120 is FP32's
// infinity: magnitudes above 1.75 * 2^127 come back as 1.75 * 2^127.
//
// Backward, with g and u read back (exact in FP32) and t = 1 / (1 + exp(-g)):
// grad_g = grad_h u t (1 + g (1 - t)), grad_u = grad_h g t, h = g t u.
//
// Both are bound by HBM: in 16 bits the forward reads 4 and writes 4.06 bytes
// per value, the backward reads 4.06 and writes 6. Four lanes share a block, 8
// columns each (16-byte loads of 16-bit rows, 8-byte stores of codes, two
// shuffles for the block's maximum), so a warp touches whole 32-byte sectors
// of every plane and no shared memory is needed. A thread keeps two blocks
// (backward: three) in flight. At 32768 x 14336 in BF16 the forward takes
// 0.62 ms (91 % of the measured copy bandwidth), the backward 0.71 ms (100 %). Rows
// that do not all start on 16 bytes are read and written by element, and bound by
// that: 24576 x 1408, BF16, forward 52 -> 88 us, backward 65 -> 279; FP32 84 -> 108
// and 117 -> 377.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kBlock = 32;       // columns that share a scale
constexpr int kLanes = kBlock / kLaneCols;
// Blocks a thread has in flight at once: on 32768 x 14336 values in BF16, 1, 2 and
// 3 take the forward 614, 619 and 632 us (24576 x 1408: 58, 53, 55), the backward
// 771, 737 and 707.
constexpr int kForwardItems = 2;
constexpr int kBackwardItems = 3;

// The block's scale byte from its largest finite magnitude's bits, which all
// four lanes of the block hold: 1.75 * 2^8 = 448.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    const int b = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)min(max(b, 0), 246);
}

// Codes of this lane's eight values, and the block's scale byte. All lanes of
// the warp call.
template <int DT>
__device__ __forceinline__ uint2 encode8(const Raw8<DT> &v, uint32_t &sb)
{
    uint32_t top = top8<DT, false>(v);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool odd = __any_sync(0xffffffffu, top >= 0x7f800000u);     // infinities or NaN: rare
    if (odd) {
        top = top8<DT, true>(v);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    }
    sb = scale_byte(top);
    const float inv = __uint_as_float((254u - sb) << 23);       // 2^-x, normal for every byte
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = make_float2(v.at(2 * i) * inv, v.at(2 * i + 1) * inv);
        if (odd) {
            // the conversion saturates infinities; they are to come back as NaN
            if (isinf(v.at(2 * i))) f.x = __uint_as_float(0x7fffffffu);
            if (isinf(v.at(2 * i + 1))) f.y = __uint_as_float(0x7fffffffu);
        }
        c[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

__device__ __forceinline__ void decode8(uint2 c, uint32_t sb, float (&v)[8])
{
    // 2^(sb - 127); 2^-127 is subnormal
    const float s = __uint_as_float(sb == 0 ? 0x00400000u : sb << 23);
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
swiglu_checkpoint_kernel(const void *__restrict__ g, const void *__restrict__ u, int64_t ld_bytes,
                         int I, Walk w, void *__restrict__ h, int64_t ldh_bytes,
                         uint8_t *__restrict__ codes_g, uint8_t *__restrict__ codes_u,
                         uint8_t *__restrict__ scales_g, uint8_t *__restrict__ scales_u)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t rows = rows_to_do(w);
    const int part = (threadIdx.x & 3) * kLaneCols;
    Place at = first_place<kLanes>(w);
    // the four lanes of a block stay together; a warp leaves when all its
    // blocks are done, so the shuffles always have every lane
    while (__any_sync(0xffffffffu, at.row < rows)) {
        Place p[kForwardItems];
        Raw8<DT> a[kForwardItems], b[kForwardItems];
#pragma unroll
        for (int k = 0; k < kForwardItems; ++k) {
            p[k] = at;
            at.advance(w);
            const int col = p[k].blk * kBlock + part;
            const int left = p[k].row < rows ? I - col : 0;
            const int64_t off = left > 0 ? p[k].row * ld_bytes : 0;
            a[k] = load8<DT, VEC>(static_cast<const uint8_t *>(g) + off, col, left);
            b[k] = load8<DT, VEC>(static_cast<const uint8_t *>(u) + off, col, left);
        }
#pragma unroll
        for (int k = 0; k < kForwardItems; ++k) {
            uint32_t sa, sb;
            const uint2 ca = encode8<DT>(a[k], sa), cb = encode8<DT>(b[k], sb);
            if (p[k].row >= rows) continue;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t, not_t;
                sigmoid_of<DT>(a[k].at(i), t, not_t);
                o[i] = a[k].at(i) * t * b[k].at(i);
            }
            const int col = p[k].blk * kBlock + part;
            const int64_t block = p[k].row * w.S + p[k].blk;
            *reinterpret_cast<uint2 *>(codes_g + block * kBlock + part) = ca;
            *reinterpret_cast<uint2 *>(codes_u + block * kBlock + part) = cb;
            if (part == 0) {
                scales_g[block] = (uint8_t)sa;
                scales_u[block] = (uint8_t)sb;
            }
            store8<DT, VEC>(static_cast<uint8_t *>(h) + p[k].row * ldh_bytes, col, I - col, o);
        }
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
swiglu_checkpoint_backward_kernel(const void *__restrict__ grad_h, int64_t ld_bytes,
                                  const uint8_t *__restrict__ codes_g,
                                  const uint8_t *__restrict__ codes_u,
                                  const uint8_t *__restrict__ scales_g,
                                  const uint8_t *__restrict__ scales_u, int I, Walk w,
                                  void *__restrict__ grad_g, void *__restrict__ grad_u,
                                  int64_t ldg_bytes, void *__restrict__ h, int64_t ldh_bytes)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t rows = rows_to_do(w);
    const int part = (threadIdx.x & 3) * kLaneCols;
    Place at = first_place<kLanes>(w);
    while (at.row < rows) {
        Place p[kBackwardItems];
        Raw8<DT> d[kBackwardItems];
        uint2 cg[kBackwardItems], cu[kBackwardItems];
        uint32_t sg[kBackwardItems], su[kBackwardItems];
#pragma unroll
        for (int k = 0; k < kBackwardItems; ++k) {
            p[k] = at;
            at.advance(w);
            if (p[k].row >= rows) continue;
            const int col = p[k].blk * kBlock + part;
            const int64_t block = p[k].row * w.S + p[k].blk;
            d[k] = load8<DT, VEC>(static_cast<const uint8_t *>(grad_h) + p[k].row * ld_bytes, col, I - col);
            cg[k] = __ldcs(reinterpret_cast<const uint2 *>(codes_g + block * kBlock + part));
            cu[k] = __ldcs(reinterpret_cast<const uint2 *>(codes_u + block * kBlock + part));
            sg[k] = scales_g[block];
            su[k] = scales_u[block];
        }
#pragma unroll
        for (int k = 0; k < kBackwardItems; ++k) {
            if (p[k].row >= rows) continue;
            float g[8], u[8], dg[8], du[8], o[8];
            decode8(cg[k], sg[k], g);
            decode8(cu[k], su[k], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t, not_t;
                sigmoid_of<DT>(g[i], t, not_t);
                const float gt = g[i] * t, x = d[k].at(i);
                dg[i] = x * (u[i] * (t * (1.0f + g[i] * not_t)));
                du[i] = x * gt;
                o[i] = gt * u[i];
            }
            const int col = p[k].blk * kBlock + part, left = I - col;
            store8<DT, VEC>(static_cast<uint8_t *>(grad_g) + p[k].row * ldg_bytes, col, left, dg);
            store8<DT, VEC>(static_cast<uint8_t *>(grad_u) + p[k].row * ldg_bytes, col, left, du);
            if (h != nullptr)
                store8<DT, VEC>(static_cast<uint8_t *>(h) + p[k].row * ldh_bytes, col, left, o);
        }
    }
}

template <int DT>
cudaError_t forward_dt(const void *g, const void *u, int64_t ld, int64_t rows, int64_t I,
                       const int32_t *end, void *h, int64_t ldh, uint8_t *cg, uint8_t *cu,
                       uint8_t *sg, uint8_t *su, cudaStream_t s)
{
    const int64_t eb = sizeof(typename Elem<DT>::T);
    unsigned grid;
    const Walk w = make_walk<kLanes>(rows, I, end, &grid);
    const bool vec = rows16(g, ld * eb) && rows16(u, ld * eb) && rows16(h, ldh * eb);
    auto k = vec ? swiglu_checkpoint_kernel<DT, true> : swiglu_checkpoint_kernel<DT, false>;
    return launch_pdl(k, dim3(grid), dim3(kRowThreads), 0, s, g, u, ld * eb, (int)I, w, h, ldh * eb,
                      cg, cu, sg, su);
}

template <int DT>
cudaError_t backward_dt(const void *gh, int64_t ld, const uint8_t *cg, const uint8_t *cu,
                        const uint8_t *sg, const uint8_t *su, int64_t rows, int64_t I,
                        const int32_t *end, void *dg, void *du, int64_t ldg, void *h, int64_t ldh,
                        cudaStream_t s)
{
    const int64_t eb = sizeof(typename Elem<DT>::T);
    unsigned grid;
    const Walk w = make_walk<kLanes>(rows, I, end, &grid);
    const bool vec = rows16(gh, ld * eb) && rows16(dg, ldg * eb) && rows16(du, ldg * eb) &&
                     (h == nullptr || rows16(h, ldh * eb));
    auto k = vec ? swiglu_checkpoint_backward_kernel<DT, true>
                 : swiglu_checkpoint_backward_kernel<DT, false>;
    return launch_pdl(k, dim3(grid), dim3(kRowThreads), 0, s, gh, ld * eb, cg, cu, sg, su, (int)I, w,
                      dg, du, ldg * eb, h, ldh * eb);
}

}  // namespace

SwigluCheckpointPlanes swiglu_checkpoint_planes(int64_t rows, int64_t I)
{
    const size_t S = (size_t)((I + kBlock - 1) / kBlock);
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    SwigluCheckpointPlanes p;
    p.row_codes = S * kBlock;
    p.row_scales = S;
    p.gate_codes = 0;
    p.up_codes = up((size_t)rows * p.row_codes);
    p.gate_scales = p.up_codes + up((size_t)rows * p.row_codes);
    p.up_scales = p.gate_scales + up((size_t)rows * S);
    p.total = p.up_scales + up((size_t)rows * S);
    return p;
}

cudaError_t launch_swiglu_checkpoint(int dt, const void *g, const void *u, int64_t ld,
                                     const int32_t *end, int64_t rows, int64_t I, void *h,
                                     int64_t ldh, void *ckpt, cudaStream_t s)
{
    const SwigluCheckpointPlanes p = swiglu_checkpoint_planes(rows, I);
    uint8_t *c = static_cast<uint8_t *>(ckpt);
    uint8_t *cg = c + p.gate_codes, *cu = c + p.up_codes, *sg = c + p.gate_scales, *su = c + p.up_scales;
    if (dt == DT_F32) return forward_dt<DT_F32>(g, u, ld, rows, I, end, h, ldh, cg, cu, sg, su, s);
    if (dt == DT_BF16) return forward_dt<DT_BF16>(g, u, ld, rows, I, end, h, ldh, cg, cu, sg, su, s);
    return forward_dt<DT_F16>(g, u, ld, rows, I, end, h, ldh, cg, cu, sg, su, s);
}

cudaError_t launch_swiglu_checkpoint_backward(int dt, const void *grad_h, int64_t ld,
                                              const void *ckpt, const int32_t *end, int64_t rows,
                                              int64_t I, void *grad_g, void *grad_u, int64_t ldg,
                                              void *h, int64_t ldh, cudaStream_t s)
{
    const SwigluCheckpointPlanes p = swiglu_checkpoint_planes(rows, I);
    const uint8_t *c = static_cast<const uint8_t *>(ckpt);
    const uint8_t *cg = c + p.gate_codes, *cu = c + p.up_codes, *sg = c + p.gate_scales,
                  *su = c + p.up_scales;
    if (dt == DT_F32)
        return backward_dt<DT_F32>(grad_h, ld, cg, cu, sg, su, rows, I, end, grad_g, grad_u, ldg, h, ldh, s);
    if (dt == DT_BF16)
        return backward_dt<DT_BF16>(grad_h, ld, cg, cu, sg, su, rows, I, end, grad_g, grad_u, ldg, h, ldh, s);
    return backward_dt<DT_F16>(grad_h, ld, cg, cu, sg, su, rows, I, end, grad_g, grad_u, ldg, h, ldh, s);
}

}  // namespace moe
