// grouped_f8.cu -- grouped products of e4m3 rows and matrices with FP32 scales per
// block of 128, on tcgen05 tensor cores.
//
// For the rows r of expert e, with b running over the blocks of 128 of K:
//   out[r, n] = sum_b sa[r, b] sw[e, n / 128, b] * (sum_{k in b} a[r, k] w[e][n, k])
// (MOE_WEIGHT_NK), or w[e][k, n] and sw[e, b, n / 128] (MOE_WEIGHT_KN).
// The inner sums run on the tensor cores (kind::f8f6f4, FP32 accumulator); each
// block's is multiplied by its two scales and added up in FP32 registers, so no
// sum in the accumulator has more than 128 terms.
//
// Two forms. Experts of many rows: grouped_f8_wide.cu. This file's is for few rows,
// where the kernel streams weights. It is transposed as in grouped_tc.cu, out^T =
// w a^T: the weights' n on the MMA's fixed side (M = 128), the expert's rows, at most
// 64, on the other (N = 16 .. 64), so that one or two rows per expert cost a
// 16-wide MMA. A weight tile of 128 n has one scale per block, a row (a column of the
// accumulator) its own.
//
// Per CTA (one per SM, 384 threads, persistent over the units):
//   warp 0   TMA producer of the weights: 128 n x 128 k (16 KiB) per stage;
//   warp 2   TMA producer of the unit's rows x 128 k, into the same stages;
//   warp 1   tcgen05.mma issuer, K = 32 per instruction, one accumulator of 64
//            columns per block, four in turn;
//   warp 3   products of the rows' scales and the weights', four blocks at a time;
//   warps 4-7, 8-11  epilogue, 32 columns each: TMEM is read in 8 x 8 blocks, in
//            which a thread meets two of every eight columns, so that it fetches a
//            quarter of the scales; sums stay in registers until the last block.
// Few units: a cluster of 2, 4 or 8 CTAs shares each unit's k (SPLIT), every
// CTA with its own blocks; the FP32 partial sums meet through distributed shared
// memory, each CTA adding its share of the rows in rank order.
//
// Bound by HBM where experts have few rows: 1024 rows on 256 experts of 7168 x 2048
// 540 us, the copy bandwidth. Many small matrices cost more than their bytes: 64
// experts of 2048 x 2048, 4 rows each, 48 us for 40 of bytes.
//
// Every wait is bounded (wait_ns); on expiry the kernel records ST_TIMEOUT, stops
// issuing work, drains its own copies and MMAs, frees TMEM and exits.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "grouped.cuh"
#include "grouped_f8.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int RING_BYTES = 192 << 10;
constexpr int MAX_STAGES = 10;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int STG_ROWS = 8;              // rows staged at a time
constexpr int STG_F32_ROW = 528;         // bytes of a staged row: 16 more than 128 FP32 values
constexpr int STG_BYTES = STG_ROWS * STG_F32_ROW;    // a group's buffer; in 16 bits two halves of it
constexpr int CAP = 64;                  // rows of a unit at most
constexpr int SCALE_STAGES = 3, SCALE_KB = 4;        // scales are staged for four blocks at a time
constexpr int ACCS = 4, TMEM_COLS = ACCS * CAP;
constexpr int PARTIAL_BYTES = CAP * BM * 4;

struct __align__(1024) Smem {
    uint8_t ring[RING_BYTES];
    uint8_t stg[2][STG_BYTES];           // one per group of epilogue warps
    float scale[SCALE_STAGES][SCALE_KB][CAP];            // a row's times the weights'
    int8_t shift[SCALE_STAGES][SCALE_KB][CAP];           // (scales_apart) where plain is 0
    int plain[SCALE_STAGES];                             // these products need no shift
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full[ACCS];
    uint64_t acc_empty[ACCS];
    uint64_t scale_full[SCALE_STAGES];
    uint64_t scale_empty[SCALE_STAGES];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int warp_sum[THREADS / 32];
    Segments seg;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;       // + alignment slack
static_assert(kSmemBytes <= 232448, "one CTA's shared memory");

struct F8Params {
    const int32_t *offsets;
    const float *a_scales;   // [rows, KB]
    const float *w_scales;   // [E, NB, KB] or [E, KB, NB]
    int E, rows, N, K;
    int w_tiles;             // weight tiles of 128 columns
    int tok_cap;             // rows per unit at most
    int row_block;           // row units per block
    int slot_bytes;          // ring slot: W_BYTES + the rows of a full unit
    int stages;
    int split;               // SPLIT: CTAs that share a unit's k
    int out_bf16;            // 16-bit outputs: BF16 or F16
    uint8_t *out;
    int64_t out_row_bytes;
    int vec;                 // rows of out start on 16 bytes
    unsigned *status;
    uint64_t wait_ns;
};

// Three maps of the rows, for boxes of 64, 32 and 16 of them.
struct RowMaps {
    CUtensorMap m[3];
};

// sum += v * s of two FP32 values in one register pair.
__device__ __forceinline__ void fma2(uint64_t &sum, uint32_t v0, uint32_t v1, uint64_t s)
{
    asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\tfma.rn.f32x2 %0, a, %3, %0;\n\t}"
        : "+l"(sum)
        : "r"(v0), "r"(v1), "l"(s));
}

__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// 16 TMEM lanes x 32 consecutive fp32 columns as blocks of 8 x 8: thread T holds
// lanes T / 4 (r[4 i], r[4 i + 1]) and T / 4 + 8 (r[4 i + 2], r[4 i + 3]), columns
// 8 i + 2 (T % 4) and the next.
__device__ __forceinline__ void tmem_ld_blocks32(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Stores four 8 x 8 blocks of 16-bit values, one register each, transposed; the
// lanes 8 m .. 8 m + 7 give the addresses of block m's eight rows of 16 bytes.
__device__ __forceinline__ void store_blocks_transposed(uint32_t saddr, uint32_t r0, uint32_t r1, uint32_t r2,
                                                        uint32_t r3)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r0),
                 "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

template <bool KN, bool OUT_F32, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
grouped_f8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_a,
                  const F8Params p)
{
    extern __shared__ uint8_t smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int ways = SPLIT ? p.split : 1;            // CTAs per unit
    const int unit0 = (int)blockIdx.x / ways, unit_step = (int)gridDim.x / ways;
    // this CTA's blocks of k
    const int all_kb = (p.K + BK - 1) / BK, slice = SPLIT ? (int)cluster_ctarank() : 0;
    const int kb_begin = SPLIT ? all_kb * slice / ways : 0;
    const int kb_end = SPLIT ? all_kb * (slice + 1) / ways : all_kb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) { mbar_init(&S.full[s], 1); mbar_init(&S.empty[s], 1); }
        for (int a = 0; a < ACCS; ++a) { mbar_init(&S.acc_full[a], 1); mbar_init(&S.acc_empty[a], EPI_WARPS); }
        for (int s = 0; s < SCALE_STAGES; ++s) { mbar_init(&S.scale_full[s], 1); mbar_init(&S.scale_empty[s], EPI_WARPS); }
        mbar_init(&S.drain, 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc<1>(&S.tmem_base, TMEM_COLS);
        tmem_relinquish<1>();
    }
    pdl_wait();
    pdl_launch_dependents();
    load_segments<THREADS>(S.seg, S.warp_sum, p.offsets, p.E, p.rows, p.status,
                           [&](int cnt) { return (cnt + p.tok_cap - 1) / p.tok_cap * p.w_tiles; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = S.tmem_base;
    const int total = S.seg.unit[p.E];
    volatile int *abort_flag = &S.abort;
    UnitWalk<1, F8Params> walk(S.seg, p, 0);

    if (warp < 4) {
        if (warp == 0) {
            // ------------------------------------------- TMA producer: weights
            const uint32_t on = elect_lane();
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const uint32_t bytes = W_BYTES + u.mma_n * BK;
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    ok = warp_wait<1>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&S.full[stage]);
                    expect_tx_on(on, &S.full[stage], bytes);
                    if constexpr (KN) load_3d_on<1>(on, ring + stage * p.slot_bytes, &map_w, bar, u.w0, kb * BK, u.e);
                    else load_3d_on<1>(on, ring + stage * p.slot_bytes, &map_w, bar, kb * BK, u.w0, u.e);
                    if (++stage == p.stages) { stage = 0; phase ^= 1u; }
                }
            }
        } else if (warp == 2) {
            // ------------------------------------------- TMA producer: rows
            const uint32_t on = elect_lane();
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const int mine = u.mma_n;
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    ok = warp_wait<1>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    const uint32_t sa = ring + stage * p.slot_bytes + W_BYTES, bar = smem_u32(&S.full[stage]);
                    auto load = [&](int box, int at) {
                        load_2d_on<1>(on, sa + at * BK, &map_a.m[box], bar, kb * BK, u.row0 + at);
                    };
                    int at = 0;
                    if (mine & 64) { load(0, at); at += 64; }
                    if (mine & 32) { load(1, at); at += 32; }
                    if (mine & 16) load(2, at);
                    if (++stage == p.stages) { stage = 0; phase ^= 1u; }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            constexpr uint32_t idesc0 = idesc_e4m3(BM, 0, KN, false);
            const uint32_t on = elect_lane();
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const uint32_t idesc = idesc0 | ((uint32_t)(u.mma_n >> 3) << 17);
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    ok = warp_wait_both(&S.acc_empty[acc], acc_phase ^ 1u, &S.full[stage], phase, abort_flag,
                                        p.status, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(acc * CAP);
                    const uint32_t w = ring + stage * p.slot_bytes, a = w + W_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / UK; ++k)
                        umma_f8_on<1>(on, d, KN ? sdesc_mn_sw128(w + k * UK * 128, W_BYTES) : sdesc_k_sw128(w + k * UK),
                                       sdesc_k_sw128(a + k * UK), idesc, k ? 1u : 0u);
                    commit_on<1>(on, &S.empty[stage]);
                    commit_on<1>(on, &S.acc_full[acc]);
                    if (++stage == p.stages) { stage = 0; phase ^= 1u; }
                    if (++acc == ACCS) { acc = 0; acc_phase ^= 1u; }
                }
            }
            // every MMA issued must finish before TMEM is released, also where
            // another role has given up
            if (on) {
                umma_commit<1>(&S.drain);
                mbar_wait(&S.drain, 0, nullptr, p.status, kDrainLimitNs);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ------------------------------------------------------ scales
            // of the unit's rows times the weights', four blocks at a time: four lanes to a row
            const int n_blocks = (p.N + BM - 1) / BM, k = lane & 3;
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const int nb = u.w0 / BM < n_blocks ? u.w0 / BM : 0;     // columns past N are not stored
                for (int kb = kb_begin; kb < kb_end; kb += SCALE_KB) {
                    float a[CAP / 8], w = 1.0f;
                    const bool in = kb + k < kb_end;
                    const float *src = p.a_scales + (int64_t)(u.row0 + lane / 4) * all_kb + kb + k;
#pragma unroll
                    for (int i = 0; i < CAP / 8; ++i, src += 8 * all_kb) a[i] = in && lane / 4 + 8 * i < u.rows ? __ldg(src) : 1.0f;
                    if (in)
                        w = __ldg(p.w_scales + (KN ? ((int64_t)u.e * all_kb + kb + k) * n_blocks + nb
                                                   : ((int64_t)u.e * n_blocks + nb) * all_kb + kb + k));
                    ok = warp_wait<1>(&S.scale_empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    bool plain = plain_scale(w);
#pragma unroll
                    for (int i = 0; i < CAP / 8; ++i) {
                        plain = plain && plain_scale(a[i]);
                        S.scale[stage][k][lane / 4 + 8 * i] = a[i] * w;
                    }
                    plain = __all_sync(0xffffffffu, plain);
                    if (!plain) {                // rare: the products themselves
                        plain = true;
                        src -= CAP * all_kb;
#pragma unroll 1
                        for (int r = lane / 4; r < CAP; r += 8, src += 8 * all_kb) {
                            const float v = in && r < u.rows ? __ldg(src) : 1.0f;
                            const int which = scales_apart(v, w, S.scale[stage][k][r]);
                            S.shift[stage][k][r] = (int8_t)which;
                            plain = plain && which == 0;
                        }
                        plain = __all_sync(0xffffffffu, plain);
                    }
                    if (lane == 0) S.plain[stage] = plain;
                    __syncwarp();
                    arrive_on(lane == 0, &S.scale_full[stage]);
                    if (++stage == SCALE_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                          // TMEM lane quadrant of this warp
        const int group = warp >= 8 ? 1 : 0;
        const int tid = threadIdx.x - (group ? 256 : 128);    // 0..127 in the group
        int acc = 0, stage = 0;
        uint32_t acc_phase = 0, phase = 0;
        const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16) + group * 32;
        for (int unit = unit0; unit < total; unit += unit_step) {
            const Unit u = walk.at(unit);
            // this group's columns: 32 of the accumulator's 64. A thread has lanes
            // lane / 4 + 8 m (m = 2 h + e) and columns 8 i + 2 (lane % 4) and the next:
            // sums[h][2 i + e], a pair each
            uint64_t sums[2][8];
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[i / 8][i % 8] = 0;
            bool ok = true;
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                const int k = (kb - kb_begin) % SCALE_KB;
                ok = warp_wait<1>(&S.acc_full[acc], acc_phase, abort_flag, p.status, p.wait_ns);
                if (k == 0) ok = ok && warp_wait<1>(&S.scale_full[stage], phase, abort_flag, p.status, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                if (u.rows > group * 32) {
                    const uint32_t tbase = tlane + (uint32_t)(acc * CAP);
                    const float *sc = S.scale[stage][k] + group * 32 + 2 * (lane & 3);
                    const int plain = S.plain[stage];
                    uint32_t v[2][16];
                    tmem_ld_blocks32(tbase, v[0]);
                    tmem_ld_blocks32(tbase + (16u << 16), v[1]);
                    uint64_t s2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) s2[i] = *reinterpret_cast<const uint64_t *>(sc + i * 8);
                    tmem_ld_wait16(v[0]);
                    tmem_ld_wait16(v[1]);
                    if (!plain) {
                        const int8_t *shift = S.shift[stage][k] + group * 32 + 2 * (lane & 3);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float f = shift_of(shift[i / 4 * 8 + (i & 1)]);
                            v[0][i] = __float_as_uint(__uint_as_float(v[0][i]) * f);
                            v[1][i] = __float_as_uint(__uint_as_float(v[1][i]) * f);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            fma2(sums[h][2 * i], v[h][4 * i], v[h][4 * i + 1], s2[i]);
                            fma2(sums[h][2 * i + 1], v[h][4 * i + 2], v[h][4 * i + 3], s2[i]);
                        }
                }
                tc_fence_before();
                __syncwarp();
                const bool last = k == SCALE_KB - 1 || kb + 1 == kb_end;
                if (lane == 0) {
                    mbar_arrive(&S.acc_empty[acc]);
                    if (last) mbar_arrive(&S.scale_empty[stage]);
                }
                if (last && ++stage == SCALE_STAGES) { stage = 0; phase ^= 1u; }
                if (++acc == ACCS) { acc = 0; acc_phase ^= 1u; }
            }
            if constexpr (SPLIT) {
                // the partial sums stay here, [row][n] in FP32
                float *mine = reinterpret_cast<float *>(S.ring + RING_BYTES - PARTIAL_BYTES) + q * 32 + lane / 4;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = group * 32 + i / 2 * 8 + 2 * (lane & 3), n = h * 16 + (i & 1) * 8;
                        mine[t * BM + n] = low(sums[h][i]);
                        mine[(t + 1) * BM + n] = high(sums[h][i]);
                    }
                continue;
            }
            // a group's warps leave together: none may wait at a barrier for
            // one that has given up
            if (!epi_all(1 + group, ok)) break;
            constexpr int ESZ = OUT_F32 ? 4 : 2, PIECES = BM * ESZ / 16, PER_IT = 128 / PIECES;
            const int piece = tid % PIECES, col = u.w0 + piece * (16 / ESZ);
            uint8_t *out0 = p.out + (int64_t)u.row0 * p.out_row_bytes + (int64_t)col * ESZ;
            const bool whole = p.vec && col + 16 / ESZ <= p.N;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t0 = group * 32 + i * 8;
                if (t0 >= u.rows) continue;
                // eight rows through shared memory. 16 bits: the halves of the buffer
                // take turns, and who passes the barrier has read the other one; the
                // 16-byte pieces of row t are permuted by t, so that a block's eight
                // rows meet no bank twice
                uint8_t *stg = S.stg[group] + (OUT_F32 ? 0 : (i & 1) * (STG_ROWS * BM * 2));
                if constexpr (OUT_F32) {
                    epi_sync(1 + group);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint64_t two = sums[m / 2][2 * i + (m & 1)];
                        uint8_t *to = stg + 2 * (lane & 3) * STG_F32_ROW + (q * 32 + m * 8 + lane / 4) * 4;
                        *reinterpret_cast<float *>(to) = low(two);
                        *reinterpret_cast<float *>(to + STG_F32_ROW) = high(two);
                    }
                } else {
                    auto block = [&](int m) {
                        const uint64_t two = sums[m / 2][2 * i + (m & 1)];
                        return p.out_bf16 ? float2_to_bf16x2(low(two), high(two)) : float2_to_f16x2(low(two), high(two));
                    };
                    const int t = lane & 7, at = q * 4 + (lane >> 3);
                    store_blocks_transposed(smem_u32(stg + t * (BM * 2) + ((at ^ t) << 4)), block(0), block(1),
                                            block(2), block(3));
                }
                epi_sync(1 + group);
#pragma unroll
                for (int r = 0; r < STG_ROWS / PER_IT; ++r) {
                    const int t = r * PER_IT + tid / PIECES;
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        stg + (OUT_F32 ? t * STG_F32_ROW + piece * 16 : t * (BM * 2) + ((piece ^ (t & 7)) << 4)));
                    if (t0 + t >= u.rows) continue;
                    uint8_t *dst = out0 + (int64_t)(t0 + t) * p.out_row_bytes;
                    if (whole) {
                        *reinterpret_cast<uint4 *>(dst) = v;
                    } else {
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int c = 0; c < 16 / ESZ; ++c) {
                            if (col + c >= p.N) continue;
                            if constexpr (OUT_F32) reinterpret_cast<uint32_t *>(dst)[c] = w[c];
                            else reinterpret_cast<uint16_t *>(dst)[c] = (uint16_t)(w[c / 2] >> (c & 1) * 16);
                        }
                    }
                }
            }
        }
    }

    if constexpr (SPLIT) {
        // every CTA's partial sums are written; each adds its rows
        __syncwarp();
        cluster_sync();
        if (unit0 < total) {
            const Unit u = UnitWalk<1, F8Params>(S.seg, p, 0).at(unit0);
            const uint32_t partial = smem_u32(S.ring + RING_BYTES - PARTIAL_BYTES);
            for (int i = threadIdx.x; ; i += THREADS) {
                const int t = i / BM * ways + slice, n = i % BM;
                if (t >= u.rows) break;
                float sum = 0.0f;
                for (int r = 0; r < ways; ++r) {
                    float v;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(v) : "r"(mapa_shared(partial + (t * BM + n) * 4, r)) : "memory");
                    sum += v;
                }
                if (u.w0 + n >= p.N) continue;
                uint8_t *dst = p.out + (int64_t)(u.row0 + t) * p.out_row_bytes;
                if constexpr (OUT_F32) reinterpret_cast<float *>(dst)[u.w0 + n] = sum;
                else if (p.out_bf16) reinterpret_cast<__nv_bfloat16 *>(dst)[u.w0 + n] = __float2bfloat16_rn(sum);
                else reinterpret_cast<__half *>(dst)[u.w0 + n] = __float2half_rn(sum);
            }
        }
        cluster_sync();             // nobody leaves while its sums are read
    }
    // ------------------------------------------------------------ teardown
    __syncthreads();
    if (*abort_flag) let_copies_land();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, TMEM_COLS);
    }
}

// ---- host side ---------------------------------------------------------------

template <bool KN, bool OUT_F32, bool SPLIT>
cudaError_t launch_kernel(int64_t units, const CUtensorMap &mw, const RowMaps &ma, const F8Params &p,
                          cudaStream_t s)
{
    static std::atomic<int> cache[kCachedDevices];
    auto kernel = grouped_f8_kernel<KN, OUT_F32, SPLIT>;
    int ctas = 0;
    cudaError_t err = prepare_kernel(kernel, 1, THREADS, kSmemBytes, cache, &ctas);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    const int ways = SPLIT ? p.split : 1;
    cfg.gridDim = dim3((unsigned)(SPLIT || ways * units < ctas ? ways * units : ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ways;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ways > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, mw, ma, p);
}

template <bool SPLIT>
cudaError_t launch_form(const GroupedF8 &g, int split, unsigned *status, cudaStream_t s)
{
    const uint64_t N = (uint64_t)g.N, K = (uint64_t)g.K, E = (uint64_t)g.E;
    CUtensorMap mw;
    RowMaps ma;
    bool ok = g.transposed ? encode_bytes(&mw, g.w, 3, {N, K, E}, {N, N * K}, BK)
                           : encode_bytes(&mw, g.w, 3, {K, N, E}, {K, N * K}, BM);
    for (int i = 0; i < 3; ++i)
        ok = ok && encode_bytes(&ma.m[i], g.a, 2, {K, (uint64_t)g.rows, 1}, {(uint64_t)g.lda, 0}, 64u >> i);
    if (!ok) return cudaErrorInvalidValue;
    F8Params p{};
    p.offsets = g.offsets;
    p.a_scales = g.a_scales;
    p.w_scales = g.w_scales;
    p.E = g.E;
    p.rows = (int)g.rows;
    p.N = (int)g.N;
    p.K = (int)g.K;
    p.w_tiles = (int)((g.N + BM - 1) / BM);
    p.tok_cap = CAP;
    const int64_t block = kRowBlockBytes / (CAP * g.K), most = (g.rows + CAP - 1) / CAP;
    p.row_block = (int)(block < 1 ? 1 : block > most ? most : block);
    p.slot_bytes = W_BYTES + CAP * BK;
    const int slots = (RING_BYTES - (SPLIT ? PARTIAL_BYTES : 0)) / p.slot_bytes;
    p.stages = slots < MAX_STAGES ? slots : MAX_STAGES;
    p.split = split;
    p.out_bf16 = g.out_dt == DT_BF16;
    p.out = static_cast<uint8_t *>(g.out);
    p.out_row_bytes = g.ldo * (g.out_dt == DT_F32 ? 4 : 2);
    p.vec = p.out_row_bytes % 16 == 0;
    p.status = status;
    // a wait may last one unit's whole reduction, a producer's as many short units
    // as the ring has stages
    p.wait_ns = wait_limit_ns() + work_ns(2 * (uint64_t)((g.K + BK - 1) / BK + p.stages), (uint64_t)p.stages);
    // an upper bound: every expert adds at most one unit that is not full
    const int64_t units = (g.rows / CAP + (g.rows < g.E ? g.rows : g.E)) * p.w_tiles;
    if (g.out_dt == DT_F32)
        return g.transposed ? launch_kernel<true, true, SPLIT>(units, mw, ma, p, s)
                            : launch_kernel<false, true, SPLIT>(units, mw, ma, p, s);
    return g.transposed ? launch_kernel<true, false, SPLIT>(units, mw, ma, p, s)
                        : launch_kernel<false, false, SPLIT>(units, mw, ma, p, s);
}

}  // namespace

cudaError_t launch_grouped_gemm_f8(const GroupedF8 &g, unsigned *status, cudaStream_t s)
{
    // Few units (of the single form's 64 rows by 128 columns): split k over as
    // many CTAs, 2 to 8, as the GPU has room for and as leave each two blocks.
    const int64_t units = (g.rows / CAP + (g.rows < g.E ? g.rows : g.E)) * ((g.N + BM - 1) / BM);
    const int64_t num_kb = (g.K + BK - 1) / BK, sms = device_sm_count();
    int split = 1;
    while (split < 8 && units * split * 2 <= sms && num_kb >= split * 2 * 2) split *= 2;
    if (split > 1) return launch_form<true>(g, split, status, s);
    // The two forms, by the average rows of an expert, each row's expert drawn evenly:
    // us at 32, 48, 56, 64, 72, 96 rows, on 64 experts of N = K = 2048 (16 of N = K =
    // 4096): this one 50 51 57 74 87 93 (54 55 54 73 83 84), the wide one 65 65 65 66
    // 66 66 (65 66 66 66 66 67). It is units of more than 64 rows that cost this form a
    // second pass over the weights: with exactly 64 rows in each expert it takes 52 (55).
    if (g.rows >= 64 * (int64_t)g.E) return launch_grouped_gemm_f8_wide(g, status, s);
    return launch_form<false>(g, 1, status, s);
}

}  // namespace moe
