// few.cuh -- the whole layer for a few tokens in two kernels: routing, the gate and
// up products and SwiGLU in the first, routing again, the down product and the
// weighted combine in the second.
//
//   p = softmax(logits[t]); the top_k experts by logit, lower id first among equal
//   ones; w = p (over its sum where renormalized), rounded to the logits' type;
//   h[t, j] = SiLU(x[t] Wg[e]^T) * (x[t] Wu[e]^T), rounded to x's type;
//   y[t] = sum over j, in slot order, of w[t, j] * (h[t, j] Wd[e]^T).
// 8-bit weights: Wg[e][n, k] = code * scale of the block (n / 128, k / 128); the sums
// of a block's 128 products are multiplied by its scale and added up in FP32.
//
// The layer reads the matrices of the touched experts once and does 2 flops per
// pair for each of their values: bound by HBM for up to some 8 tokens per expert and
// more. So both kernels are a stream of weights, and all else is arranged around it.
// Every CTA (one per SM, 16 warps) routes all tokens by itself, in shared memory: a
// microsecond or two, and no kernel or grid barrier in between. The (token, slot)
// pairs are sorted by expert and cut into chunks of at most 8 NT pairs of one expert.
//
// A tile is 16 weight rows against a chunk: the M = 16 side of mma.sync m16n8k16,
// with the chunk's tokens on the N = 8 side (NT of them); a tensor-memory MMA would
// take 128 rows, and these sums need no more than a few percent of the pipe. In the
// first kernel rows 0-7 are gate rows and 8-15 the up rows of the same columns, so
// that a thread holds both factors of its h; in the second 16 rows of down. Lane
// (g, t) = (lane / 4, lane % 4) loads 16 bytes of rows g and g + 8 as they lie: the
// order of k within an MMA is free as long as both operands have the same one, and
// x is read in that order too (from L1). FP32 runs on FFMA in the same layout.
//
// A CTA's tiles x k-steps form one sequence, cut into 16 equal contiguous pieces, one
// per warp, so that all warps stream for the whole time; a warp keeps kDepth steps of
// 2 x 128 bytes per row in flight in registers, across tile borders. Tiles cut by a
// border leave partial sums in shared memory, which the warp that has the tile's
// beginning adds up in order: results do not depend on timing.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewPairs = kFewMaxTokens * kFewMaxTopK;
constexpr int kDepth = 4;                 // steps in flight per warp
constexpr int kStepBytes = 128;           // of each row per step
constexpr uint16_t kNoExpert = 0xffff;
constexpr unsigned kFull = 0xffffffffu;

// What a CTA knows of the routing.
struct alignas(16) FewPlan {
    uint16_t ids[kFewPairs];              // expert of pair t * top_k + j
    float w[kFewPairs];                   // its weight
    uint16_t order[kFewPairs];            // pairs by expert
    struct { uint16_t e, first, count, pad; } chunk[kFewPairs];
    uint32_t starts[kFewPairs / 32];      // bit i: order[i] starts a chunk
    int chunks;
};

// Routes one token with a warp; lane i holds logits i, i + 32, ...
template <int EPL>
__device__ __forceinline__ void few_route_token(const FewArgs &a, int t, FewPlan &S)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[EPL];                    // larger key, larger logit; 0: none or taken
    int bad = 0, some = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0;
        if (e >= a.E) continue;
        const float l = load_as_float(a.logits, a.ldt, (int64_t)t * a.E + e);
        bad |= isnan(l) || l == INFINITY;
        some |= l != -INFINITY;
        const uint32_t b = l == 0.0f ? 0u : __float_as_uint(l);      // -0 and +0 are equal
        key[i] = b & 0x80000000u ? ~b : b | 0x80000000u;
    }
    const bool invalid = __any_sync(kFull, bad) || !__any_sync(kFull, some);
    auto logit = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); };
    constexpr float kLog2e = 1.4426950408889634f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = max(top, key[i]);
    const float m = logit(__reduce_max_sync(kFull, top));
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (key[i] != 0) s += exp2f((logit(key[i]) - m) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    const float inv_s = 1.0f / s;
    float z = 0.0f, mine = 0.0f;
    int id = 0;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(kFull, best);
        int e = 0x7fffffff;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
            if (key[i] == best) e = lane + 32 * i;
        e = __reduce_min_sync(kFull, e);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == lane + 32 * i) key[i] = 0;
        const float p = exp2f((logit(best) - m) * kLog2e) * inv_s;
        z += p;
        if (lane == j) { mine = p; id = e; }
    }
    if (lane < a.top_k) {
        float w = invalid ? __uint_as_float(0x7fc00000u) : a.renormalize ? mine / z : mine;
        if (a.ldt == DT_BF16) w = __bfloat162float(__float2bfloat16_rn(w));
        else if (a.ldt == DT_F16) w = __half2float(__float2half_rn(w));
        S.ids[t * a.top_k + lane] = (uint16_t)(invalid ? lane : id);
        S.w[t * a.top_k + lane] = w;
    }
}

// Fills the plan; all threads call.
__device__ __forceinline__ void few_plan(const FewArgs &a, int chunk_max, FewPlan &S)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pairs = a.T * a.top_k;
    if (a.logits != nullptr) {
        for (int t = warp; t < a.T; t += kFewWarps) {
            if (a.E <= 64) few_route_token<2>(a, t, S);
            else if (a.E <= 256) few_route_token<8>(a, t, S);
            else few_route_token<32>(a, t, S);
        }
    } else {
        for (int i = threadIdx.x; i < pairs; i += kFewThreads) {
            const uint32_t e = a.indices[i];
            const bool ok = e < (uint32_t)a.E;
            if (!ok && blockIdx.x == 0) atomicOr(a.status, ST_BAD_INDEX);
            S.ids[i] = ok ? (uint16_t)e : kNoExpert;
            // a token with a slot that has no expert is NaN
            S.w[i] = ok ? load_as_float(a.weights, a.wdt, i) : __uint_as_float(0x7fc00000u);
        }
    }
    __syncthreads();
    // position of each pair in the order by (expert, pair); pairs without an
    // expert come last and start no chunk
    bool start[kFewPairs / kFewThreads];
    int at[kFewPairs / kFewThreads], before[kFewPairs / kFewThreads], same[kFewPairs / kFewThreads];
#pragma unroll
    for (int r = 0; r < kFewPairs / kFewThreads; ++r) {
        const int i = threadIdx.x + r * kFewThreads;
        start[r] = false;
        at[r] = i;
        if (i >= pairs) continue;
        const int e = S.ids[i];
        int less = 0;
        before[r] = same[r] = 0;
        for (int k = 0; k < pairs; ++k) {
            const int f = S.ids[k];
            less += f < e;
            same[r] += f == e;
            before[r] += f == e && k < i;
        }
        at[r] = less + before[r];
        S.order[at[r]] = (uint16_t)i;
        start[r] = e != kNoExpert && before[r] % chunk_max == 0;
    }
    if (threadIdx.x < kFewPairs / 32) S.starts[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFewPairs / kFewThreads; ++r)
        if (start[r]) atomicOr(&S.starts[at[r] >> 5], 1u << (at[r] & 31));
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFewPairs / kFewThreads; ++r) {
        if (!start[r]) continue;
        int c = __popc(S.starts[at[r] >> 5] & ((1u << (at[r] & 31)) - 1u));
        for (int i = 0; i < at[r] >> 5; ++i) c += __popc(S.starts[i]);
        const int left = same[r] - before[r];
        S.chunk[c].e = S.ids[threadIdx.x + r * kFewThreads];
        S.chunk[c].first = (uint16_t)at[r];
        S.chunk[c].count = (uint16_t)(left < chunk_max ? left : chunk_max);
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int i = 0; i < kFewPairs / 32; ++i) n += __popc(S.starts[i]);
        S.chunks = n;
    }
    (void)lane;
    __syncthreads();
}

// 16 bytes of weights, read once.
__device__ __forceinline__ uint4 load_weights(const uint8_t *p)
{
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}

// 16 bytes of x or h. Not the read-only path: h was written by the kernel before,
// which this one may have started under.
__device__ __forceinline__ uint4 load_x(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int DT>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1)
{
    if constexpr (DT == DT_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 codes as two values of x's type (exact; NaN stays NaN).
template <int DT>
__device__ __forceinline__ uint32_t two_codes(uint32_t codes)
{
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    if constexpr (DT == DT_F16) return (uint32_t)r.x | (uint32_t)r.y << 16;
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
    return float2_to_bf16x2(f.x, f.y);
}

// DOWN: the second kernel. `rows`: of down per CTA, in tiles of `tile_rows`; `pass`:
// tiles whose outputs fit in shared memory at once.
template <int DT, bool F8, int NT, bool DOWN>
__global__ void __launch_bounds__(kFewThreads, 1)
few_kernel(const FewArgs a, int rows, int tile_rows, int pass)
{
    using T = typename Elem<DT>::T;
    static_assert(!F8 || DT != DT_F32, "8-bit weights meet 16-bit activations");
    constexpr int WB = F8 ? 1 : (int)sizeof(T);          // bytes per weight
    constexpr int EPC = 16 / WB;                         // weights in 16 bytes
    constexpr int STEP = kStepBytes / WB;                // k per step
    constexpr int NC = 8 * NT;                           // tokens of a chunk at most
    extern __shared__ uint8_t smem[];
    FewPlan &S = *reinterpret_cast<FewPlan *>(smem);
    float4 *pieces = reinterpret_cast<float4 *>(smem + sizeof(FewPlan));     // [warp][2][NT][32]
    float *out = reinterpret_cast<float *>(pieces + kFewWarps * 2 * NT * 32);    // DOWN: [pair][row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int K = DOWN ? a.I : a.H;                      // summed over
    const int steps = (K + STEP - 1) / STEP;
    const int kb = (K + 127) / 128;

    // the first kernel starts here under whatever made its inputs; by the time it
    // lets the second one start, those are complete
    if constexpr (!DOWN) {
        pdl_wait();
        pdl_launch_dependents();
    }
    few_plan(a, NC, S);

    const int row_begin = DOWN ? (int)blockIdx.x * rows : 0;
    const int row_end = DOWN ? min(row_begin + rows, a.H) : a.I;
    const int row_tiles = DOWN ? (row_end - row_begin + tile_rows - 1) / tile_rows : (a.I + 7) / 8;

    bool waited = !DOWN;
    for (int pass0 = 0; pass0 < (DOWN ? row_tiles : 1); pass0 += pass) {
        const int per_chunk = DOWN ? min(pass, row_tiles - pass0) : row_tiles;
        const int64_t all = (int64_t)S.chunks * per_chunk;
        const int tile0 = DOWN ? 0 : (int)(all * blockIdx.x / gridDim.x);
        const int tile1 = DOWN ? (int)all : (int)(all * (blockIdx.x + 1) / gridDim.x);
        const int64_t work = (int64_t)(tile1 - tile0) * steps;
        auto begin_of = [&](int w) { return work * w / kFewWarps; };
        const int64_t begin = begin_of(warp), end = begin_of(warp + 1);

        // what is loaded: rows p0, p1 of a tile from step `m` on, n steps of it
        struct Group { int tile, m, n; };
        auto group_at = [&](int64_t at) {
            Group r;
            const int local = (int)(at / steps);
            r.tile = tile0 + local;
            r.m = (int)(at - (int64_t)local * steps);
            const int64_t n = min((int64_t)(steps - r.m), end - at);
            r.n = (int)min((int64_t)kDepth, max(n, (int64_t)0));
            return r;
        };
        const uint8_t *p0 = nullptr, *p1 = nullptr;
        const float *s0 = nullptr, *s1 = nullptr;
        int loading = -1;
        auto point = [&](int tile) {
            if (tile == loading) return;
            loading = tile;
            const int c = tile / per_chunk, r = tile - c * per_chunk;
            const int64_t e = S.chunk[c].e;
            if constexpr (DOWN) {
                const int first = row_begin + (pass0 + r) * tile_rows;
                const int top = min(first + tile_rows, row_end), r0 = first + g, r1 = r0 + 8;
                const uint8_t *base = static_cast<const uint8_t *>(a.down) + t * 16;
                p0 = r0 < top ? base + (e * a.H + r0) * K * WB : nullptr;
                p1 = r1 < top ? base + (e * a.H + r1) * K * WB : nullptr;
                if constexpr (F8) {
                    const int64_t nb = (a.H + 127) / 128;
                    s0 = a.down_scales + (e * nb + (r0 < top ? r0 : first) / 128) * kb;
                    s1 = a.down_scales + (e * nb + (r1 < top ? r1 : first) / 128) * kb;
                }
            } else {
                const int row = r * 8 + g;
                const int64_t off = (e * a.I + row) * K * WB + t * 16;
                p0 = row < a.I ? static_cast<const uint8_t *>(a.gate) + off : nullptr;
                p1 = row < a.I ? static_cast<const uint8_t *>(a.up) + off : nullptr;
                if constexpr (F8) {
                    const int64_t at = (e * ((a.I + 127) / 128) + r * 8 / 128) * kb;
                    s0 = a.gate_scales + at;
                    s1 = a.up_scales + at;
                }
            }
        };
        uint4 buf[kDepth][2][2];                          // [step][half][row]
        float scale[kDepth][2];
        auto issue = [&](int i, const Group &r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (r.m + i) * STEP + h * (STEP / 2) + t * EPC;
                const int64_t off = (int64_t)(r.m + i) * kStepBytes + h * (kStepBytes / 2);
                const bool in = i < r.n && k < K;
                buf[i][h][0] = in && p0 != nullptr ? load_weights(p0 + off) : make_uint4(0u, 0u, 0u, 0u);
                buf[i][h][1] = in && p1 != nullptr ? load_weights(p1 + off) : make_uint4(0u, 0u, 0u, 0u);
            }
            if constexpr (F8) {
                scale[i][0] = i < r.n ? __ldg(s0 + r.m + i) : 0.0f;
                scale[i][1] = i < r.n ? __ldg(s1 + r.m + i) : 0.0f;
            }
        };
        Group now = group_at(begin);
        if (begin < end) {
            point(now.tile);
#pragma unroll
            for (int i = 0; i < kDepth; ++i) issue(i, now);
        }
        // h comes from the first kernel
        if (!waited) {
            pdl_wait();
            waited = true;
        }

        const uint8_t *px[NT];
        int computing = -1;
        float c[NT][4];
        constexpr int FR = DT == DT_F32 ? NC : 1;
        float f[FR][2];                                   // FP32: this lane's part of rows g, g + 8
        (void)f;
        auto clear = [&] {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[n][i] = 0.0f;
#pragma unroll
            for (int n = 0; n < FR; ++n) f[n][0] = f[n][1] = 0.0f;
        };
        clear();
        // a tile's sums: c[n][0..1] row g, tokens 8 n + 2 t and the next; c[n][2..3] row g + 8
        auto finish = [&](int tile, const float (&v)[NT][4]) {
            const int ch = tile / per_chunk, r = tile - ch * per_chunk;
            const int first = S.chunk[ch].first, count = S.chunk[ch].count;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int tok = n * 8 + 2 * t + q;
                    if (tok >= count) continue;
                    const int pair = S.order[first + tok];
                    if constexpr (DOWN) {
                        float *o = out + pair * (pass * tile_rows) + r * tile_rows;
                        if (g < tile_rows) o[g] = v[n][q];
                        if (g + 8 < tile_rows) o[g + 8] = v[n][2 + q];
                    } else {
                        const int row = r * 8 + g;
                        const float z = v[n][q], h = z / (1.0f + expf(-z)) * v[n][2 + q];
                        if (row < a.I) static_cast<T *>(a.h)[(int64_t)pair * a.I + row] = Elem<DT>::from_f(h);
                    }
                }
        };
        int64_t at = begin;
        while (at < end) {
            // the next group's loads take the places of this one's
            const int64_t then = at + now.n;
            const Group next = then < end ? group_at(then) : Group{now.tile, 0, 0};
            const int ch = now.tile / per_chunk;
            if (ch != computing) {
                computing = ch;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int tok = n * 8 + g;
                    px[n] = nullptr;
                    if (DT != DT_F32 && tok < S.chunk[ch].count) {
                        const int pair = S.order[S.chunk[ch].first + tok];
                        px[n] = DOWN ? static_cast<const uint8_t *>(a.h) + (int64_t)pair * K * sizeof(T)
                                     : static_cast<const uint8_t *>(a.x) + (int64_t)(pair / a.top_k) * K * sizeof(T);
                    }
                }
            }
            const int count = S.chunk[ch].count;
            point(next.tile);
#pragma unroll
            for (int i = 0; i < kDepth; ++i) {
                float part[F8 ? NT : 1][4];
                if constexpr (F8) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q) part[n][q] = 0.0f;
                }
                if (i < now.n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = (now.m + i) * STEP + h * (STEP / 2) + t * EPC;
                        const uint32_t w0[4] = {buf[i][h][0].x, buf[i][h][0].y, buf[i][h][0].z, buf[i][h][0].w};
                        const uint32_t w1[4] = {buf[i][h][1].x, buf[i][h][1].y, buf[i][h][1].z, buf[i][h][1].w};
                        if constexpr (DT == DT_F32) {
                            const int first = S.chunk[ch].first;
#pragma unroll
                            for (int n = 0; n < NC; ++n) {
                                if (n >= count) continue;
                                const int pair = S.order[first + n];
                                const float *row = DOWN ? static_cast<const float *>(a.h) + (int64_t)pair * K
                                                        : static_cast<const float *>(a.x) + (int64_t)(pair / a.top_k) * K;
                                Vec16 xv;
                                xv.u = k < K ? load_x(reinterpret_cast<const uint8_t *>(row + k)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    f[n][0] = fmaf(__uint_as_float(w0[q]), xv.f[q], f[n][0]);
                                    f[n][1] = fmaf(__uint_as_float(w1[q]), xv.f[q], f[n][1]);
                                }
                            }
                        } else {
                            uint32_t w0x[F8 ? 8 : 4], w1x[F8 ? 8 : 4];
                            if constexpr (F8) {
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    w0x[2 * q] = two_codes<DT>(w0[q] & 0xffffu);
                                    w0x[2 * q + 1] = two_codes<DT>(w0[q] >> 16);
                                    w1x[2 * q] = two_codes<DT>(w1[q] & 0xffffu);
                                    w1x[2 * q + 1] = two_codes<DT>(w1[q] >> 16);
                                }
                            } else {
#pragma unroll
                                for (int q = 0; q < 4; ++q) { w0x[q] = w0[q]; w1x[q] = w1[q]; }
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (n * 8 >= count) continue;
#pragma unroll
                                for (int v = 0; v < (F8 ? 2 : 1); ++v) {
                                    const uint4 xv = px[n] != nullptr && k < K
                                                         ? load_x(px[n] + (int64_t)k * sizeof(T) + v * 16)
                                                         : make_uint4(0u, 0u, 0u, 0u);
                                    float (&acc)[4] = F8 ? part[n] : c[n];
                                    mma16<DT>(acc, w0x[4 * v], w1x[4 * v], w0x[4 * v + 1], w1x[4 * v + 1], xv.x, xv.y);
                                    mma16<DT>(acc, w0x[4 * v + 2], w1x[4 * v + 2], w0x[4 * v + 3], w1x[4 * v + 3], xv.z, xv.w);
                                }
                            }
                        }
                    }
                    if constexpr (F8) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            c[n][0] = fmaf(part[n][0], scale[i][0], c[n][0]);
                            c[n][1] = fmaf(part[n][1], scale[i][0], c[n][1]);
                            c[n][2] = fmaf(part[n][2], scale[i][1], c[n][2]);
                            c[n][3] = fmaf(part[n][3], scale[i][1], c[n][3]);
                        }
                    }
                }
                issue(i, next);
            }
            const bool done = now.m + now.n == steps;
            if (done || then == end) {
                if constexpr (DT == DT_F32) {
                    // the quad's lanes hold sums over their own k
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            f[n][r] += __shfl_xor_sync(kFull, f[n][r], 1);
                            f[n][r] += __shfl_xor_sync(kFull, f[n][r], 2);
                            if (n % 8 / 2 == t) c[n / 8][r * 2 + n % 2] = f[n][r];
                        }
                }
                const int64_t tile_begin = (int64_t)(now.tile - tile0) * steps;
                if (done && begin <= tile_begin) {
                    finish(now.tile, c);
                } else {
                    // part of a tile: 1 has its beginning, 0 has not
                    float4 *to = pieces + ((warp * 2 + (begin <= tile_begin)) * NT) * 32 + lane;
#pragma unroll
                    for (int n = 0; n < NT; ++n) to[n * 32] = make_float4(c[n][0], c[n][1], c[n][2], c[n][3]);
                }
                clear();
            }
            at = then;
            now = next;
        }
        __syncthreads();
        if (begin < end) {
            // a tile that begins here and goes on in later warps
            const int last = (int)((end - 1) / steps);
            const int64_t tile_begin = (int64_t)last * steps, tile_end = tile_begin + steps;
            if (begin <= tile_begin && tile_end > end) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 v = pieces[((warp * 2 + 1) * NT + n) * 32 + lane];
                    c[n][0] = v.x; c[n][1] = v.y; c[n][2] = v.z; c[n][3] = v.w;
                }
                for (int w = warp + 1; w < kFewWarps && begin_of(w) < tile_end; ++w) {
                    if (begin_of(w) == begin_of(w + 1)) continue;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 v = pieces[((w * 2) * NT + n) * 32 + lane];
                        c[n][0] += v.x; c[n][1] += v.y; c[n][2] += v.z; c[n][3] += v.w;
                    }
                }
                finish(tile0 + last, c);
            }
        }
        if constexpr (DOWN) {
            __syncthreads();
            if (pass0 + pass >= row_tiles) pdl_launch_dependents();
            const int first = row_begin + pass0 * tile_rows, n = min(per_chunk * tile_rows, row_end - first);
            for (int i = threadIdx.x; i < a.T * n; i += kFewThreads) {
                const int tok = i / n, r = i - tok * n;
                float y = 0.0f;
                for (int j = 0; j < a.top_k; ++j) {
                    const int pair = tok * a.top_k + j;
                    // NaN where the slot has no expert
                    y = S.ids[pair] == kNoExpert ? S.w[pair] : fmaf(S.w[pair], out[pair * (pass * tile_rows) + r], y);
                    if (S.ids[pair] == kNoExpert) break;
                }
                static_cast<T *>(a.y)[(int64_t)tok * a.H + first + r] = Elem<DT>::from_f(y);
            }
            __syncthreads();
        }
    }
}

template <int DT, bool F8, int NT>
cudaError_t launch_few_nt(const FewArgs &a, cudaStream_t s)
{
    auto up = few_kernel<DT, F8, NT, false>, down = few_kernel<DT, F8, NT, true>;
    const size_t fixed = sizeof(FewPlan) + (size_t)kFewWarps * 2 * NT * 32 * sizeof(float4);
    const int pairs = a.T * a.top_k, sms = device_sm_count();
    // equal shares of down's rows, in equal tiles of at most 16
    const int rows = (a.H + sms - 1) / sms, tiles = (rows + 15) / 16, tile_rows = (rows + tiles - 1) / tiles;
    const int fit = (int)((kFewSharedBytes - fixed) / ((size_t)pairs * tile_rows * sizeof(float)));
    const int pass = fit < tiles ? fit : tiles;
    const size_t smem = fixed + (size_t)pairs * pass * tile_rows * sizeof(float);
    cudaError_t err = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fixed);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSharedBytes);
    if (err != cudaSuccess) return err;
    const int64_t up_tiles = (int64_t)pairs * ((a.I + 7) / 8);
    err = launch_pdl(up, dim3((unsigned)(up_tiles < sms ? up_tiles : sms)), dim3(kFewThreads), fixed, s, a, 0, 0, 1);
    if (err != cudaSuccess) return err;
    return launch_pdl(down, dim3((unsigned)((a.H + rows - 1) / rows)), dim3(kFewThreads), smem, s, a, rows,
                      tile_rows, pass);
}

template <int DT, bool F8>
cudaError_t launch_few_form(const FewArgs &a, cudaStream_t s)
{
    if (a.T <= 8) return launch_few_nt<DT, F8, 1>(a, s);
    if (a.T <= 16) return launch_few_nt<DT, F8, 2>(a, s);
    return launch_few_nt<DT, F8, 4>(a, s);
}

}  // namespace
}  // namespace moe
