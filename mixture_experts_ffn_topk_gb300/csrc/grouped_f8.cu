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
// Transposed as in grouped_tc.cu, out^T = w a^T: the weights' n on the MMA's
// fixed side (M = 128 per CTA), the expert's rows on the other (N = 16 .. 256).
// A weight tile of 128 n has one scale per block, a row (a column of the
// accumulator) its own: one product of scales per column and block, the same in
// all lanes of a warp.
//
// Per CTA (one per SM, 384 threads, persistent over the units):
//   warp 0   TMA producer of the weights: 128 n x 128 k (16 KiB) per stage;
//   warp 2   TMA producer of the unit's rows x 128 k, into the same stages;
//   warp 1   tcgen05.mma issuer, K = 32 per instruction, one accumulator per block,
//            two of 256 columns (pairs) or four of 64 in turn;
//   warp 3   the products of scales of each block, into a ring of their own;
//   warps 4-7, 8-11  two groups that take every second 16 columns of each
//            accumulator: TMEM lane = n, column = row of the segment; sums stay in
//            registers until the last block.
// CTA pairs (CG = 2): M = 256, each CTA holds its 128 weight columns and half of
// the unit's rows; the even CTA issues the MMAs for both.
// Few units: a cluster of 2, 4 or 8 single CTAs shares each unit's k (SPLIT), every
// CTA with its own blocks; the FP32 partial sums meet through distributed shared
// memory, each CTA adding its share of the rows in rank order.
//
// Every wait is bounded (wait_ns); on expiry the kernel records ST_TIMEOUT, stops
// issuing work, drains its own copies and MMAs, frees TMEM and exits.
#include <atomic>

#include "common.cuh"
#include "grouped.cuh"
#include "grouped_issue.cuh"
#include "grouped_units.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int BK = 128;                  // k per stage: 128 bytes, one block of scales
constexpr int UK = 32;                   // k per tcgen05.mma
constexpr int W_BYTES = BM * BK;         // 16 KiB
constexpr int RING_BYTES = 192 << 10;
constexpr int MAX_STAGES = 10;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int STG_BYTES = 4096;          // one epilogue staging buffer
constexpr int PAIR_CAP = 256, SINGLE_CAP = 64;       // rows of a unit at most
constexpr int SCALE_STAGES = 4;
constexpr int MAX_ACCS = 4;
constexpr int PARTIAL_BYTES = SINGLE_CAP * BM * 4;
constexpr uint64_t kDrainLimitNs = 100000000ull;

struct __align__(1024) Smem {
    uint8_t ring[RING_BYTES];
    uint8_t stg[2][2][STG_BYTES];        // two per group of epilogue warps
    float scale[SCALE_STAGES][PAIR_CAP];
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full[MAX_ACCS];
    uint64_t acc_empty[MAX_ACCS];
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
    int w_tiles;             // weight tiles of 128 * CG columns
    int tok_cap;             // rows per unit at most
    int row_block;           // row units per block
    int slot_bytes;          // ring slot: W_BYTES + this CTA's rows of a full unit
    int stages;
    int split;               // SPLIT: CTAs that share a unit's k
    int out_bf16;            // 16-bit outputs: BF16 or F16
    uint8_t *out;
    int64_t out_row_bytes;
    int vec;                 // rows of out start on 16 bytes
    unsigned *status;
    uint64_t wait_ns;
};

// Four maps of the rows, for boxes of 128, 64, 32 and 16 of them.
struct RowMaps {
    CUtensorMap m[4];
};

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

// Instruction descriptor, kind::f8f6f4: FP32 accumulator, A and B e4m3 (0), A
// MN-major where a_mn, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn)
{
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// sum += v * s of two FP32 values in one register pair.
__device__ __forceinline__ void fma2(uint64_t &sum, uint32_t v0, uint32_t v1, uint64_t s)
{
    asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\tfma.rn.f32x2 %0, a, %3, %0;\n\t}"
        : "+l"(sum)
        : "r"(v0), "r"(v1), "l"(s));
}

__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

template <int CG, bool KN, bool OUT_F32, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
grouped_f8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_a,
                  const F8Params p)
{
    extern __shared__ uint8_t smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    static_assert(!SPLIT || CG == 1, "a split unit runs on single CTAs");
    constexpr int CAP = CG == 2 ? PAIR_CAP : SINGLE_CAP;
    constexpr int ACCS = CG == 2 ? 2 : 4, TMEM_COLS = ACCS * CAP;
    const int ways = SPLIT ? p.split : CG;           // CTAs per unit
    const int unit0 = (int)blockIdx.x / ways, unit_step = (int)gridDim.x / ways;
    // this CTA's blocks of k
    const int all_kb = (p.K + BK - 1) / BK, slice = SPLIT ? (int)cluster_ctarank() : 0;
    const int kb_begin = SPLIT ? all_kb * slice / ways : 0;
    const int kb_end = SPLIT ? all_kb * (slice + 1) / ways : all_kb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) { mbar_init(&S.full[s], 1); mbar_init(&S.empty[s], 1); }
        for (int a = 0; a < ACCS; ++a) { mbar_init(&S.acc_full[a], 1); mbar_init(&S.acc_empty[a], EPI_WARPS * CG); }
        for (int s = 0; s < SCALE_STAGES; ++s) { mbar_init(&S.scale_full[s], 1); mbar_init(&S.scale_empty[s], EPI_WARPS); }
        mbar_init(&S.drain, 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc<CG>(&S.tmem_base, TMEM_COLS);
        tmem_relinquish<CG>();
    }
    pdl_wait();
    pdl_launch_dependents();
    load_segments<THREADS>(S.seg, S.warp_sum, p.offsets, p.E, p.rows, p.status,
                           [&](int cnt) { return (cnt + p.tok_cap - 1) / p.tok_cap * p.w_tiles; });
    tc_fence_before();
    // a pair also makes each CTA's barrier initialisation visible to the
    // other before any copy or arrival targets it
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = S.tmem_base;
    const int total = S.seg.unit[p.E];
    volatile int *abort_flag = &S.abort;
    UnitWalk<CG, F8Params> walk(S.seg, p, rank);

    // 384 threads start with 168 registers each: 128 * (88 + 2 * 208) is the same
    if (warp < 4) {
        if constexpr (CG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            // ------------------------------------------- TMA producer: weights
            const uint32_t on = elect_lane(), arm = leader ? on : 0u;
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                // both CTAs' copies of weights and rows complete on the leader's
                // barrier, which expects them all
                const uint32_t bytes = CG * (W_BYTES + u.mma_n / CG * BK);
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    ok = warp_wait<CG>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    const uint32_t here = smem_u32(&S.full[stage]), bar = CG == 2 ? mapa_shared(here, 0) : here;
                    expect_tx_on(arm, &S.full[stage], bytes);
                    if constexpr (KN) load_3d_on<CG>(on, ring + stage * p.slot_bytes, &map_w, bar, u.w0, kb * BK, u.e);
                    else load_3d_on<CG>(on, ring + stage * p.slot_bytes, &map_w, bar, kb * BK, u.w0, u.e);
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
                const int mine = u.mma_n / CG;               // rows this CTA loads
                const int row0 = u.row0 + rank * mine;
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    ok = warp_wait<CG>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    const uint32_t sa = ring + stage * p.slot_bytes + W_BYTES, here = smem_u32(&S.full[stage]);
                    const uint32_t bar = CG == 2 ? mapa_shared(here, 0) : here;
                    auto load = [&](int box, int at) {
                        load_2d_on<CG>(on, sa + at * BK, &map_a.m[box], bar, kb * BK, row0 + at);
                    };
                    int at = 0;
                    for (; mine - at >= 128; at += 128) load(0, at);
                    if (mine & 64) { load(1, at); at += 64; }
                    if (mine & 32) { load(2, at); at += 32; }
                    if (mine & 16) load(3, at);
                    if (++stage == p.stages) { stage = 0; phase ^= 1u; }
                }
            }
        } else if (warp == 1 && leader) {
            // ------------------------------------------------------ MMA issuer
            constexpr uint32_t idesc0 = idesc_e4m3(BM * CG, 0, KN);
            const uint32_t on = elect_lane();
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const uint32_t idesc = idesc0 | ((uint32_t)(u.mma_n >> 3) << 17);
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    ok = warp_wait<CG>(&S.acc_empty[acc], acc_phase ^ 1u, abort_flag, p.status, p.wait_ns) &&
                         warp_wait<CG>(&S.full[stage], phase, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(acc * CAP);
                    const uint32_t w = ring + stage * p.slot_bytes, a = w + W_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / UK; ++k)
                        umma_f8_on<CG>(on, d, KN ? sdesc_mn_sw128(w + k * UK * 128, W_BYTES) : sdesc_k_sw128(w + k * UK),
                                       sdesc_k_sw128(a + k * UK), idesc, k ? 1u : 0u);
                    commit_on<CG>(on, &S.empty[stage]);
                    commit_on<CG>(on, &S.acc_full[acc]);
                    if (++stage == p.stages) { stage = 0; phase ^= 1u; }
                    if (++acc == ACCS) { acc = 0; acc_phase ^= 1u; }
                }
            }
            // every MMA issued must finish before TMEM is released, also where
            // another role has given up
            if (on) {
                umma_commit<CG>(&S.drain);
                mbar_wait(&S.drain, 0, nullptr, p.status, kDrainLimitNs);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ------------------------------------------------------ scales
            constexpr int PER = CAP / 32;
            const int n_blocks = (p.N + BM - 1) / BM;
            int unit = unit0, kb = kb_begin, stage = 0;
            uint32_t phase = 0;
            Unit u = {};
            // the scales of the next block: one block is loaded ahead of the one stored
            auto next = [&](float (&v)[PER], float &w) {
                if (kb >= kb_end) { kb = kb_begin; unit += unit_step; }
                if (unit >= total || kb >= kb_end) return false;
                if (kb == kb_begin) u = walk.at(unit);
                const int nb = u.w0 / BM;
                w = nb < n_blocks
                        ? __ldg(p.w_scales + (KN ? ((int64_t)u.e * all_kb + kb) * n_blocks + nb
                                                 : ((int64_t)u.e * n_blocks + nb) * all_kb + kb))
                        : 0.0f;
                const float *s = p.a_scales + (int64_t)u.row0 * all_kb + kb;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    v[i] = i * 32 + lane < u.rows ? __ldg(s + (int64_t)(i * 32 + lane) * all_kb) : 0.0f;
                ++kb;
                return true;
            };
            auto put = [&](const float (&v)[PER], float w) {
                if (!warp_wait<1>(&S.scale_empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns)) return false;
#pragma unroll
                for (int i = 0; i < PER; ++i) S.scale[stage][i * 32 + lane] = v[i] * w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.scale_full[stage]);
                if (++stage == SCALE_STAGES) { stage = 0; phase ^= 1u; }
                return true;
            };
            float v0[PER], v1[PER], w0, w1;
            bool more = next(v0, w0);
            while (more) {
                const bool second = next(v1, w1);
                if (!put(v0, w0) || !second) break;
                more = next(v0, w0);
                if (!put(v1, w1)) break;
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        if constexpr (CG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int q = warp & 3;                          // TMEM lane quadrant of this warp
        const int group = warp >= 8 ? 1 : 0;
        const int tid = threadIdx.x - (group ? 256 : 128);    // 0..127 in the group
        constexpr int CHUNKS = CAP / 32;                 // 16 columns each
        constexpr int CH = OUT_F32 ? 8 : 16;             // rows per staging buffer
        constexpr int ESZ = OUT_F32 ? 4 : 2;
        constexpr int ROW_BYTES = BM * ESZ;              // staged bytes per row: 512 / 256
        constexpr int PIECES = ROW_BYTES / 16, PER_IT = 128 / PIECES;
        int acc = 0, stage = 0, buf = 0;
        uint32_t acc_phase = 0, phase = 0;
        const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
        for (int unit = unit0; unit < total; unit += unit_step) {
            const Unit u = walk.at(unit);
            // this group's chunks: rows [16 (2 j + group), + 16)
            const int chunks = u.rows > group * 16 ? (u.rows - group * 16 + 31) / 32 : 0;
            uint64_t sums[CHUNKS][8];                  // two rows each
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) sums[j][i] = 0;
            bool ok = true;
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                ok = warp_wait<CG>(&S.acc_full[acc], acc_phase, abort_flag, p.status, p.wait_ns) &&
                     warp_wait<1>(&S.scale_full[stage], phase, abort_flag, p.status, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t tbase = tlane + (uint32_t)(acc * CAP + group * 16);
                const float *sc = S.scale[stage] + group * 16;
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2 && !leader) mbar_arrive_cluster(mapa_shared(smem_u32(&S.acc_empty[acc]), 0));
                        else mbar_arrive(&S.acc_empty[acc]);
                    }
                };
                // a chunk is on its way while the one before is added up
                uint32_t v[2][16];
                if (chunks > 0) tmem_ld16(tbase, v[0]);
                else release();
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    if (j >= chunks) continue;
                    tmem_ld_wait16(v[j & 1]);
                    if (j + 1 < CHUNKS && j + 1 < chunks) tmem_ld16(tbase + (j + 1) * 32, v[(j + 1) & 1]);
                    else release();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const ulonglong2 s = *reinterpret_cast<const ulonglong2 *>(sc + j * 32 + i * 4);
                        fma2(sums[j][2 * i], v[j & 1][4 * i], v[j & 1][4 * i + 1], s.x);
                        fma2(sums[j][2 * i + 1], v[j & 1][4 * i + 2], v[j & 1][4 * i + 3], s.y);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.scale_empty[stage]);
                if (++stage == SCALE_STAGES) { stage = 0; phase ^= 1u; }
                if (++acc == ACCS) { acc = 0; acc_phase ^= 1u; }
            }
            if constexpr (SPLIT) {
                // the partial sums stay here, [row][n] in FP32
                float *mine = reinterpret_cast<float *>(S.ring + RING_BYTES - PARTIAL_BYTES) + q * 32 + lane;
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = j * 32 + group * 16 + 2 * i;
                        mine[t * BM] = low(sums[j][i]);
                        mine[(t + 1) * BM] = high(sums[j][i]);
                    }
                continue;
            }
            // a group's warps leave together: none may wait at a barrier for
            // one that has given up
            if (!epi_all(1 + group, ok)) break;
            const int piece = tid % PIECES, col = u.w0 + piece * (16 / ESZ);
            uint8_t *out0 = p.out + (int64_t)u.row0 * p.out_row_bytes + (int64_t)col * ESZ;
            const bool whole = p.vec && col + 16 / ESZ <= p.N;
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) {
#pragma unroll
                for (int h = 0; h < 16 / CH; ++h) {
                    const int t0 = j * 32 + group * 16 + h * CH;
                    if (t0 >= u.rows) continue;
                    // CH rows through shared memory: a barrier per buffer, who passes
                    // it has read the other one
                    uint8_t *stg = S.stg[group][buf], *mine = stg + (q * 32 + lane) * ESZ;
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const uint64_t two = sums[j][(h * CH + i) / 2];
                        const float f = i & 1 ? high(two) : low(two);
                        if constexpr (OUT_F32) {
                            *reinterpret_cast<float *>(mine + i * ROW_BYTES) = f;
                        } else if (p.out_bf16) {
                            *reinterpret_cast<__nv_bfloat16 *>(mine + i * ROW_BYTES) = __float2bfloat16_rn(f);
                        } else {
                            *reinterpret_cast<__half *>(mine + i * ROW_BYTES) = __float2half_rn(f);
                        }
                    }
                    epi_sync(1 + group);
#pragma unroll
                    for (int i = 0; i < CH / PER_IT; ++i) {
                        const int t = i * PER_IT + tid / PIECES;
                        const uint4 v = *reinterpret_cast<const uint4 *>(stg + t * ROW_BYTES + piece * 16);
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
                    buf ^= 1;
                }
            }
        }
    }

    if constexpr (SPLIT) {
        // every CTA's partial sums are written; each adds its rows
        __syncwarp();
        cluster_sync();
        if (unit0 < total) {
            const Unit u = UnitWalk<CG, F8Params>(S.seg, p, rank).at(unit0);
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
    // a pair keeps both CTAs (their shared memory is read by the leader's
    // MMAs and signalled by its commits) until both are done
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, TMEM_COLS);
    }
}

// ---- host side ---------------------------------------------------------------

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

template <int CG, bool KN, bool OUT_F32, bool SPLIT>
cudaError_t launch_kernel(int64_t units, const CUtensorMap &mw, const RowMaps &ma, const F8Params &p,
                          cudaStream_t s)
{
    static std::atomic<int> cache[kCachedDevices];
    auto kernel = grouped_f8_kernel<CG, KN, OUT_F32, SPLIT>;
    int ctas = 0;
    cudaError_t err = prepare_kernel(kernel, CG, THREADS, kSmemBytes, cache, &ctas);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    const int ways = SPLIT ? p.split : CG;
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

template <int CG, bool SPLIT>
cudaError_t launch_form(const GroupedF8 &g, int split, unsigned *status, cudaStream_t s)
{
    constexpr int CAP = CG == 2 ? PAIR_CAP : SINGLE_CAP;
    const uint64_t N = (uint64_t)g.N, K = (uint64_t)g.K, E = (uint64_t)g.E;
    CUtensorMap mw;
    RowMaps ma;
    bool ok = g.transposed ? encode_bytes(&mw, g.w, 3, {N, K, E}, {N, N * K}, BK)
                           : encode_bytes(&mw, g.w, 3, {K, N, E}, {K, N * K}, BM);
    for (int i = 0; i < 4; ++i)
        ok = ok && encode_bytes(&ma.m[i], g.a, 2, {K, (uint64_t)g.rows, 1}, {(uint64_t)g.lda, 0}, 128u >> i);
    if (!ok) return cudaErrorInvalidValue;
    F8Params p{};
    p.offsets = g.offsets;
    p.a_scales = g.a_scales;
    p.w_scales = g.w_scales;
    p.E = g.E;
    p.rows = (int)g.rows;
    p.N = (int)g.N;
    p.K = (int)g.K;
    p.w_tiles = (int)((g.N + BM * CG - 1) / (BM * CG));
    p.tok_cap = CAP;
    const int64_t block = kRowBlockBytes / (CAP * g.K), most = (g.rows + CAP - 1) / CAP;
    p.row_block = (int)(block < 1 ? 1 : block > most ? most : block);
    p.slot_bytes = W_BYTES + CAP / CG * BK;
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
        return g.transposed ? launch_kernel<CG, true, true, SPLIT>(units, mw, ma, p, s)
                            : launch_kernel<CG, false, true, SPLIT>(units, mw, ma, p, s);
    return g.transposed ? launch_kernel<CG, true, false, SPLIT>(units, mw, ma, p, s)
                        : launch_kernel<CG, false, false, SPLIT>(units, mw, ma, p, s);
}

}  // namespace

cudaError_t launch_grouped_gemm_f8(const GroupedF8 &g, unsigned *status, cudaStream_t s)
{
    // Few units (of the single form's 64 rows by 128 columns): split k over as
    // many CTAs, 2 to 8, as the GPU has room for and as leave each two blocks.
    const int64_t units = (g.rows / SINGLE_CAP + (g.rows < g.E ? g.rows : g.E)) * ((g.N + BM - 1) / BM);
    const int64_t num_kb = (g.K + BK - 1) / BK, sms = device_sm_count();
    int split = 1;
    while (split < 8 && units * split * 2 <= sms && num_kb >= split * 2 * 2) split *= 2;
    if (split > 1) return launch_form<1, true>(g, split, status, s);
    if (g.rows >= 64 * (int64_t)g.E) return launch_form<2, false>(g, 1, status, s);
    return launch_form<1, false>(g, 1, status, s);
}

}  // namespace moe
