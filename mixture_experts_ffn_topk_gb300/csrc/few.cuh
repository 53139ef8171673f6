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
// The layer reads the matrices of the touched experts and does 2 flops per pair for
// each of their values: bound by HBM. So both kernels are a stream of weights, and all
// else is arranged around it. Every CTA (one per SM, 16 warps) routes all tokens by
// itself, in shared memory: a microsecond or two, and no kernel or grid barrier in
// between. The (token, slot) pairs are sorted by expert and cut into chunks of at most
// 8 NT pairs of one expert (NT: 2 for 16-bit weights where experts have four pairs and
// more on average, else 1).
//
// Each chunk is a pass of its own over its expert's matrices: an expert with more than
// 8 NT pairs is read from memory once per chunk. 8 experts of 4096 x 4096, top_k 2,
// e4m3: 80 us for 16 tokens (no expert with more than 8 pairs: 8 passes, 59 us of
// bytes), 91 for 17 (9 passes), 120 for 32 (12). Below that every byte is read once.
//
// A tile is 16 weight rows against a chunk: the M = 16 side of mma.sync m16n8k16,
// with the chunk's tokens on the N = 8 side (NT of them); a tensor-memory MMA would
// take 128 rows, and these sums need no more than a few percent of the pipe. In the
// first kernel rows 0-7 are gate rows and 8-15 the up rows of the same columns, so
// that a thread holds both factors of its h; in the second 16 rows of down. Lane
// (g, t) = (lane / 4, lane % 4) loads 32 bytes of rows g and g + 8 as they lie: the
// order of k within an MMA is free as long as both operands have the same one, and
// x is read in that order too (from L1). FP32 runs on FFMA in the same layout.
//
// A CTA's tiles x k-steps form one sequence, cut into 16 equal contiguous pieces, one
// per warp, so that all warps stream for the whole time; a warp keeps kDepth steps of
// 16 rows x 128 bytes in flight in registers, across tile borders. Tiles cut by a
// border leave partial sums in shared memory, which the warp that has the tile's
// beginning adds up in order: results do not depend on timing.
//
// What the rest costs is latency: x is loaded for a whole group of steps before its
// products (one wait instead of one per product: 973 -> 754 us for 8 tokens on 256
// experts of 7168 x 2048), and the code that finishes a tile is there once, since
// weights that pass through L2 evict the kernel and each launch fetches its code from
// memory anew; for the same reason weights are read evict-first (where all rows start
// on 32 bytes). Deeper groups (4
// steps) cost 8-bit weights their registers (528 us against 409), and a ring of
// asynchronous copies in shared memory an issue slot per 16 bytes (1106 us).
// 8 tokens, 256 experts, BF16: 0.74 to 0.78 ms, the touched weights at the copy
// bandwidth; e4m3: 0.41 to 0.43 ms (90 %). One token, 64 experts of 2048 x 1408: 26 us, of which 15
// stream; the routing in each kernel takes 2, the first loads after it 2.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kFewWarps = 16;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kDepth = 2;                 // steps of a warp in flight
constexpr int kStepBytes = 128;           // of each row per step
constexpr uint16_t kNoExpert = 0xffff;
constexpr unsigned kFull = 0xffffffffu;

// What a CTA knows of the routing, in shared memory: `n` pairs.
struct FewPlan {
    float *w;                             // weight of pair t * top_k + j
    uint16_t *ids;                        // its expert
    uint16_t *order;                      // pairs by expert
    uint16_t *len;                        // of the chunk that starts at order[i], or 0
    uint16_t *chunk_e, *chunk_first, *chunk_len;
    int *chunks;

    __host__ __device__ static constexpr size_t bytes(int n) { return 16 + (size_t)((n + 7) & ~7) * 16; }

    __device__ __forceinline__ FewPlan(uint8_t *at, int n)
    {
        n = (n + 7) & ~7;
        chunks = reinterpret_cast<int *>(at);
        w = reinterpret_cast<float *>(at + 16);
        ids = reinterpret_cast<uint16_t *>(w + n);
        order = ids + n;
        len = order + n;
        chunk_e = len + n;
        chunk_first = chunk_e + n;
        chunk_len = chunk_first + n;
    }
};

// Routes one token with a warp; lane i holds logits i, i + 32, ...
template <int EPL>
__device__ __forceinline__ void few_route_token(const FewArgs &a, int t, const FewPlan &S)
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
__device__ __forceinline__ void few_plan(const FewArgs &a, int chunk_max, const FewPlan &S)
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
    for (int i = threadIdx.x; i < pairs; i += kFewThreads) {
        const int e = S.ids[i];
        int less = 0, before = 0, same = 0;
        for (int k = 0; k < pairs; ++k) {
            const int f = S.ids[k];
            less += f < e;
            same += f == e;
            before += f == e && k < i;
        }
        S.order[less + before] = (uint16_t)i;
        const int left = same - before;
        S.len[less + before] = e != kNoExpert && before % chunk_max == 0 ? (uint16_t)min(left, chunk_max) : 0;
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int i0 = 0; i0 < pairs; i0 += 32) {
            const int i = i0 + lane, len = i < pairs ? S.len[i] : 0;
            const unsigned starts = __ballot_sync(kFull, len != 0);
            if (len != 0) {
                const int c = n + __popc(starts & ((1u << lane) - 1u));
                S.chunk_e[c] = S.ids[S.order[i]];
                S.chunk_first[c] = (uint16_t)i;
                S.chunk_len[c] = (uint16_t)len;
            }
            n += __popc(starts);
        }
        if (lane == 0) *S.chunks = n;
    }
    __syncthreads();
}

// 32 bytes of weights, read once. WIDE: at once, or in two loads of 16 (rows that do
// not all start on 32 bytes; the second half may lie behind the row).
struct Raw32 {
    uint32_t w[8];
};

__device__ __forceinline__ void load_weights32(Raw32 &v, const uint8_t *p)
{
    asm("ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
          "=r"(v.w[7])
        : "l"(p));
}

__device__ __forceinline__ void load_weights16(uint32_t *w, const uint8_t *p)
{
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
        : "l"(p));
}

// 16 bytes of x or h. Not the read-only path: h was written by the kernel before,
// which this one may have started under.
__device__ __forceinline__ uint4 load_x(const void *p)
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
// tiles whose outputs fit in shared memory at once. WIDE: rows of weights start on 32
// bytes.
template <int DT, bool F8, int NT, bool DOWN, bool WIDE>
__global__ void __launch_bounds__(kFewThreads, 1)
few_kernel(const FewArgs a, int rows, int tile_rows, int pass)
{
    using T = typename Elem<DT>::T;
    static_assert(!F8 || DT != DT_F32, "8-bit weights meet 16-bit activations");
    constexpr int WB = F8 ? 1 : (int)sizeof(T);          // bytes per weight
    constexpr int EPC = 16 / WB;                         // weights in 16 bytes
    constexpr int STEP = kStepBytes / WB;                // k per step
    constexpr int NC = 8 * NT;                           // tokens of a chunk at most
    // x of so many half steps is loaded before their products, in at most 32 registers
    constexpr int XV = F8 ? 2 : 1, XH = NT * XV <= 2 ? 4 : NT * XV == 4 ? 2 : 1;
    extern __shared__ __align__(16) uint8_t smem[];
    const int pairs = a.T * a.top_k;
    const FewPlan S(smem, pairs);
    float4 *pieces = reinterpret_cast<float4 *>(smem + FewPlan::bytes(pairs));   // [warp][2][NT][32]
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
        // kFewMaxDim keeps all of this within 31 bits
        const int all = *S.chunks * per_chunk, share = all / (int)gridDim.x, rest = all - share * (int)gridDim.x;
        auto tile_of = [&](int b) { return share * b + rest * b / (int)gridDim.x; };
        const int tile0 = DOWN ? 0 : tile_of(blockIdx.x), tile1 = DOWN ? all : tile_of(blockIdx.x + 1);
        const int work = (tile1 - tile0) * steps;
        auto begin_of = [&](int w) { return (int)((int64_t)work * w / kFewWarps); };
        const int begin = begin_of(warp), end = begin_of(warp + 1);
        const int skipped = begin / steps, first_tile = tile0 + skipped, first_m = begin - skipped * steps;

        // steps m .. m + n of a tile, loaded together
        struct Group {
            int tile, m, n;
        };
        int ungrouped = end - begin;
        auto group_at = [&](int tile, int m) {
            Group r{tile, m, min(min(kDepth, steps - m), ungrouped)};
            ungrouped -= r.n;
            return r;
        };
        const uint8_t *p0 = nullptr, *p1 = nullptr;      // this lane's rows g, g + 8, or NULL
        const float *s0 = nullptr, *s1 = nullptr;        // their scales
        int loading = -1;
        auto point = [&](int tile) {
            if (tile == loading) return;
            loading = tile;
            const int c = tile / per_chunk, r = tile - c * per_chunk;
            const int64_t e = S.chunk_e[c], row_bytes = (int64_t)K * WB;
            if constexpr (DOWN) {
                const int first = row_begin + (pass0 + r) * tile_rows;
                const int top = min(first + tile_rows, row_end), r0 = first + g, r1 = r0 + 8;
                const uint8_t *base = static_cast<const uint8_t *>(a.down) + e * a.H * row_bytes + t * 32;
                p0 = r0 < top ? base + r0 * row_bytes : nullptr;
                p1 = r1 < top ? base + r1 * row_bytes : nullptr;
                if constexpr (F8) {
                    const int64_t nb = (a.H + 127) / 128;
                    s0 = a.down_scales + (e * nb + (r0 < top ? r0 : first) / 128) * kb;
                    s1 = a.down_scales + (e * nb + (r1 < top ? r1 : first) / 128) * kb;
                }
            } else {
                const int row = r * 8 + g;
                const int64_t off = (e * a.I + row) * row_bytes + t * 32;
                p0 = row < a.I ? static_cast<const uint8_t *>(a.gate) + off : nullptr;
                p1 = row < a.I ? static_cast<const uint8_t *>(a.up) + off : nullptr;
                if constexpr (F8) {
                    const int64_t at = (e * ((a.I + 127) / 128) + r * 8 / 128) * kb;
                    s0 = a.gate_scales + at;
                    s1 = a.up_scales + at;
                }
            }
        };
        Raw32 buf[kDepth][2];                              // [step][row]
        float scale[F8 ? kDepth : 1][2];
        (void)scale;
        auto issue = [&](int i, const Group &r) {
            const int k = (r.m + i) * STEP + t * 2 * EPC;
            const int64_t off = (int64_t)(r.m + i) * kStepBytes;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint8_t *p = b ? p1 : p0;
                const bool in = i < r.n && p != nullptr;
#pragma unroll
                for (int q = 0; q < 8; ++q) buf[i][b].w[q] = 0;
                if constexpr (WIDE) {
                    if (in && k < K) load_weights32(buf[i][b], p + off);
                } else {
                    if (in && k < K) load_weights16(buf[i][b].w, p + off);
                    if (in && k + EPC < K) load_weights16(buf[i][b].w + 4, p + off + 16);
                }
            }
            if constexpr (F8) {
                scale[i][0] = i < r.n ? __ldg(s0 + r.m + i) : 0.0f;
                scale[i][1] = i < r.n ? __ldg(s1 + r.m + i) : 0.0f;
            }
        };
        Group now = group_at(first_tile, first_m);
        if (now.n > 0) {
            point(now.tile);
#pragma unroll
            for (int i = 0; i < kDepth; ++i) issue(i, now);
        }
        // h comes from the first kernel
        if (!waited) {
            pdl_wait();
            waited = true;
        }

        const uint8_t *px[NT];                           // x (h) of this lane's tokens
        int x_off = 0, count = 0;                        // FP32: of token `lane`
        float c[NT][4];
        constexpr int FR = DT == DT_F32 ? NC : 1;
        float f[FR][2];                                  // FP32: this lane's part of rows g, g + 8
        (void)f;
        int split = -1;                                  // a tile that begins here and goes on in later warps
        // once over the groups, then once more for a split tile: one copy of the
        // code that finishes a tile, which comes from memory on every launch
#pragma unroll 1
        for (int round = 0; round < 2; ++round) {
            bool fresh = true;
#pragma unroll 1
            while (round == 0 ? now.n > 0 : split >= 0) {
                int tile;
                bool whole;
                if (round == 0) {
                    tile = now.tile;
                    if (fresh) {
                        // another tile
                        fresh = false;
                        const int ch = tile / per_chunk, first = S.chunk_first[ch];
                        count = S.chunk_len[ch];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int tok = n * 8 + g;
                            px[n] = nullptr;
                            if (DT != DT_F32 && tok < count) {
                                const int pair = S.order[first + tok];
                                px[n] = DOWN ? static_cast<const uint8_t *>(a.h) + (int64_t)pair * K * sizeof(T)
                                             : static_cast<const uint8_t *>(a.x) + (int64_t)(pair / a.top_k) * K * sizeof(T);
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) c[n][q] = 0.0f;
                        }
                        if constexpr (DT == DT_F32) {
                            const int pair = S.order[first + min(lane, count - 1)];
                            x_off = (DOWN ? pair : pair / a.top_k) * K;
#pragma unroll
                            for (int n = 0; n < FR; ++n) f[n][0] = f[n][1] = 0.0f;
                        }
                    }
                    // the next group's loads take the places of this one's
                    const bool done = now.m + now.n == steps;
                    const Group next = group_at(done ? tile + 1 : tile, done ? 0 : now.m + now.n);
                    if (next.n > 0) point(next.tile);
                    float part[F8 ? NT : 1][4];
                    uint4 xs[XH][DT == DT_F32 ? 1 : NT][XV];
                    (void)part;
                    (void)xs;
#pragma unroll
                    for (int hs = 0; hs < 2 * kDepth; ++hs) {
                        const int i = hs / 2, h = hs % 2;                // step, half of the 32 bytes
                        if constexpr (DT != DT_F32) {
                            if (hs % XH == 0) {
#pragma unroll
                                for (int j = 0; j < XH; ++j)
#pragma unroll
                                    for (int n = 0; n < NT; ++n)
#pragma unroll
                                        for (int v = 0; v < XV; ++v) {
                                            const int at = now.m + (hs + j) / 2;
                                            const int k = at * STEP + t * 2 * EPC + (hs + j) % 2 * EPC;
                                            xs[j][n][v] = px[n] != nullptr && (hs + j) / 2 < now.n && k < K
                                                              ? load_x(px[n] + (int64_t)k * sizeof(T) + v * 16)
                                                              : make_uint4(0u, 0u, 0u, 0u);
                                        }
                            }
                        }
                        if constexpr (F8) {
                            if (h == 0) {
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int q = 0; q < 4; ++q) part[n][q] = 0.0f;
                            }
                        }
                        const uint32_t *u0 = buf[i][0].w + 4 * h, *u1 = buf[i][1].w + 4 * h;
                        if constexpr (DT == DT_F32) {
                            // both halves of the step, four tokens at a time
                            const float *x = static_cast<const float *>(DOWN ? a.h : a.x);
                            const int k = (now.m + i) * STEP + t * 2 * EPC;
#pragma unroll
                            for (int n0 = 0; n0 < NC; n0 += 4) {
                                if (n0 >= count || i >= now.n || h == 1) continue;
                                Vec16 xv[4][2];
#pragma unroll
                                for (int n = 0; n < 4; ++n) {
                                    const int off = __shfl_sync(kFull, x_off, n0 + n);
                                    xv[n][0].u = k < K ? load_x(x + off + k) : make_uint4(0u, 0u, 0u, 0u);
                                    xv[n][1].u = k + EPC < K ? load_x(x + off + k + EPC) : make_uint4(0u, 0u, 0u, 0u);
                                }
#pragma unroll
                                for (int n = 0; n < 4; ++n)
#pragma unroll
                                    for (int q = 0; q < 8; ++q) {
                                        f[n0 + n][0] = fmaf(__uint_as_float(u0[q]), xv[n][q / 4].f[q % 4], f[n0 + n][0]);
                                        f[n0 + n][1] = fmaf(__uint_as_float(u1[q]), xv[n][q / 4].f[q % 4], f[n0 + n][1]);
                                    }
                            }
                        } else if (i < now.n) {
                            uint32_t v0[F8 ? 8 : 4], v1[F8 ? 8 : 4];
                            if constexpr (F8) {
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    v0[2 * q] = two_codes<DT>(u0[q] & 0xffffu);
                                    v0[2 * q + 1] = two_codes<DT>(u0[q] >> 16);
                                    v1[2 * q] = two_codes<DT>(u1[q] & 0xffffu);
                                    v1[2 * q + 1] = two_codes<DT>(u1[q] >> 16);
                                }
                            } else {
#pragma unroll
                                for (int q = 0; q < 4; ++q) { v0[q] = u0[q]; v1[q] = u1[q]; }
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (n * 8 >= count) continue;
                                float (&acc)[4] = F8 ? part[n] : c[n];
#pragma unroll
                                for (int v = 0; v < XV; ++v) {
                                    const uint4 xv = xs[hs % XH][n][v];
                                    mma16<DT>(acc, v0[4 * v], v1[4 * v], v0[4 * v + 1], v1[4 * v + 1], xv.x, xv.y);
                                    mma16<DT>(acc, v0[4 * v + 2], v1[4 * v + 2], v0[4 * v + 3], v1[4 * v + 3], xv.z, xv.w);
                                }
                            }
                            if constexpr (F8) {
                                if (h == 1) {
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        c[n][0] = fmaf(part[n][0], scale[i][0], c[n][0]);
                                        c[n][1] = fmaf(part[n][1], scale[i][0], c[n][1]);
                                        c[n][2] = fmaf(part[n][2], scale[i][1], c[n][2]);
                                        c[n][3] = fmaf(part[n][3], scale[i][1], c[n][3]);
                                    }
                                }
                            }
                        }
                        if (h == 1) issue(i, next);
                    }
                    now = next;
                    if (!done && next.n > 0) continue;
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
                    const bool begun = tile != first_tile || first_m == 0;       // here, not in an earlier warp
                    whole = done && begun;
                    if (!whole) {
                        // part of a tile: 1 has its beginning, 0 has not
                        if (begun) split = tile;
                        float4 *to = pieces + ((warp * 2 + begun) * NT) * 32 + lane;
#pragma unroll
                        for (int n = 0; n < NT; ++n) to[n * 32] = make_float4(c[n][0], c[n][1], c[n][2], c[n][3]);
                    }
                    fresh = true;
                } else {
                    whole = true;
                    tile = split;
                    split = -1;
                    count = S.chunk_len[tile / per_chunk];
                    const int tile_end = (tile - tile0 + 1) * steps;
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
                }
                if (whole) {
                    // c[n][0..1]: row g, tokens 8 n + 2 t and the next; c[n][2..3]: row g + 8
                    const int ch = tile / per_chunk, r = tile - ch * per_chunk, first = S.chunk_first[ch];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int tok = n * 8 + 2 * t + q;
                            if (tok >= count) continue;
                            const int pair = S.order[first + tok];
                            if constexpr (DOWN) {
                                float *o = out + pair * (pass * tile_rows) + r * tile_rows;
                                if (g < tile_rows) o[g] = c[n][q];
                                if (g + 8 < tile_rows) o[g + 8] = c[n][2 + q];
                            } else {
                                const int row = r * 8 + g;
                                const float z = c[n][q], h = z / (1.0f + expf(-z)) * c[n][2 + q];
                                if (row < a.I) static_cast<T *>(a.h)[(int64_t)pair * a.I + row] = Elem<DT>::from_f(h);
                            }
                        }
                }
            }
            if (round == 0) __syncthreads();
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

template <int DT, bool F8, int NT, bool WIDE>
cudaError_t launch_few_wide(const FewArgs &a, cudaStream_t s)
{
    static std::atomic<int> opted[kCachedDevices];
    auto up = few_kernel<DT, F8, NT, false, WIDE>, down = few_kernel<DT, F8, NT, true, WIDE>;
    const int pairs = a.T * a.top_k, ctas = device_sm_count();
    const size_t fixed = FewPlan::bytes(pairs) + (size_t)kFewWarps * 2 * NT * 32 * sizeof(float4);
    // equal shares of down's rows, in equal tiles of at most 16
    const int rows = (a.H + ctas - 1) / ctas, tiles = (rows + 15) / 16, tile_rows = (rows + tiles - 1) / tiles;
    const int fit = (int)((kFewSharedBytes - fixed) / ((size_t)pairs * tile_rows * sizeof(float)));
    const int pass = fit < tiles ? fit : tiles;
    const size_t smem = fixed + (size_t)pairs * pass * tile_rows * sizeof(float);
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kCachedDevices;
    if (!cached || opted[dev].load() == 0) {
        err = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSharedBytes);
        if (err == cudaSuccess) err = cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSharedBytes);
        if (err != cudaSuccess) return err;
        if (cached) opted[dev].store(1);
    }
    const int64_t up_tiles = (int64_t)pairs * ((a.I + 7) / 8);
    err = launch_pdl(up, dim3((unsigned)(up_tiles < ctas ? up_tiles : ctas)), dim3(kFewThreads), fixed, s, a, 0, 0, 1);
    if (err != cudaSuccess) return err;
    return launch_pdl(down, dim3((unsigned)((a.H + rows - 1) / rows)), dim3(kFewThreads), smem, s, a, rows,
                      tile_rows, pass);
}

template <int DT, bool F8, int NT>
cudaError_t launch_few_nt(const FewArgs &a, cudaStream_t s)
{
    const uint64_t wb = F8 ? 1 : sizeof(typename Elem<DT>::T);
    const uint64_t at = reinterpret_cast<uintptr_t>(a.gate) | reinterpret_cast<uintptr_t>(a.up) |
                        reinterpret_cast<uintptr_t>(a.down) | (uint64_t)a.H * wb | (uint64_t)a.I * wb;
    return at % 32 == 0 ? launch_few_wide<DT, F8, NT, true>(a, s) : launch_few_wide<DT, F8, NT, false>(a, s);
}

template <int DT, bool F8>
cudaError_t launch_few_form(const FewArgs &a, cudaStream_t s)
{
    // Two blocks of eight tokens per tile where experts have four and more on average:
    // 8 experts of 4096 x 4096, top_k 2, us for 12, 24, 32 tokens: one block 131 142
    // 163, two 134 136 137. 8-bit and FP32 weights take one: a second costs registers
    // (8 bits: 80 94 112 against 103 113 117; FP32: 406 517 652 against 535 893 950).
    if constexpr (!F8 && DT != DT_F32)
        if (a.T * a.top_k >= 4 * a.E) return launch_few_nt<DT, F8, 2>(a, s);
    return launch_few_nt<DT, F8, 1>(a, s);
}

}  // namespace
}  // namespace moe
