// grouped_tc.cu -- grouped products of BF16 / F16 rows on tcgen05 tensor cores.
//
// For the rows r of expert e (offsets[e] <= r < offsets[e + 1]):
//   out[r, n] = sum_k a[r, k] w[e][n, k]   (MOE_WEIGHT_NK), or w[e][k, n].
// The product is computed transposed, out^T = w a^T: the weights' n, whose
// extent is the same for every expert, takes the MMA's fixed side (M = 128 per
// CTA), and the expert's rows take the side whose width is chosen per
// instruction (N = 16, 32, ..., 256). So a ragged segment wastes at most 15 (on
// a pair 31) columns of one instruction instead of most of a 128-row tile,
// and a decode step's one or two rows per expert cost a 16-wide MMA over a
// weight tile that is loaded whole: the kernel streams weights.
//
// Per CTA (one per SM, 352 threads, persistent over the units):
//   warp 0     TMA producer of the weights: 128 columns x 64 k (16 KiB; one box
//              of K-major rows, or two MN-major boxes of 64 n for [E, K, N])
//              per stage of a ring of 192 KiB;
//   warp 6     TMA producer of the unit's rows x 64 k, into the same stages;
//   warp 1     tcgen05.mma issuer, K = 16 per instruction, two accumulators of
//              256 TMEM columns in turn;
//   warps 2-5, 7-10  epilogue, two groups that take turns: TMEM lane = n,
//              column = row of the segment. 16 rows (8 of FP32) at a time are
//              rounded, transposed through shared memory and stored as 256
//              (512) consecutive bytes per row.
// CTA pairs (CG = 2): M = 256, each CTA holds its 128 weight columns and half
// of the unit's rows; the even CTA issues the MMAs for both.
// Few units (a few rows, a narrow N): a cluster of 2, 4 or 8 single CTAs shares
// each unit's k (SPLIT), every CTA with its own slice and accumulator; the FP32
// partial sums meet through distributed shared memory, each CTA adding its
// share of the rows in rank order, so the result does not depend on timing.
// An expert's rows are cut into units of equal width, at most tok_cap; units
// run over (expert, block of row units, weight tile, row unit), the row unit
// fastest, so that CTAs at work share a weight tile in L2; a block's rows are
// held to what stays in L2 while all weight tiles pass.
//
// Outputs are summed in parts, of kPartStages stages (FP32 outputs) or
// kLongPartStages (16-bit ones), each in an accumulator of its own. The epilogue
// adds the parts of FP32 outputs in registers (PARTS, units of 128 rows at most)
// while the next one is summed, and, SPLIT, all parts in shared memory. Otherwise
// (TOTAL) the total stays in the accumulator of the first part, and the later
// ones, all in the other accumulator, wait until the part before is added.
//
// Every wait is bounded (wait_ns); on expiry the kernel records ST_TIMEOUT,
// stops issuing work, drains its own copies and MMAs, frees TMEM and exits.
#include <atomic>

#include "common.cuh"
#include "grouped.cuh"
#include "grouped_issue.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int BM = 128;                  // weight columns per CTA
constexpr int BK = 64;                   // k per stage: 128 bytes
constexpr int UK = 16;                   // k per tcgen05.mma
constexpr int W_BYTES = BM * BK * 2;     // 16 KiB
constexpr int RING_BYTES = 192 << 10;
constexpr int MAX_STAGES = 10;
constexpr int ACC_COLS = 256;
constexpr int TMEM_COLS = 2 * ACC_COLS;
constexpr int THREADS = 352;
constexpr int EPI_WARPS = 8;             // two groups of four: 2-5 and 7-10
constexpr int STG_BYTES = 4096;          // one epilogue staging buffer
constexpr int SPLIT_CAP = 64;            // rows of a split unit at most
constexpr int PARTS_CAP = 128;           // rows of a unit whose parts are added in registers
constexpr int PARTIAL_BYTES = SPLIT_CAP * BM * 4;
constexpr uint64_t kDrainLimitNs = 100000000ull;
// Bytes of rows a block of row units may cover, well inside the 129 MB L2
// that also carries the streamed weights and the output.
constexpr int64_t kRowBlockBytes = 48ll << 20;

struct __align__(1024) Smem {
    uint8_t ring[RING_BYTES];
    uint8_t stg[2][2][STG_BYTES];        // two per group of epilogue warps
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int warp_sum[THREADS / 32];
    Segments seg;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;       // + alignment slack
static_assert(kSmemBytes <= 232448, "one CTA's shared memory");

struct GemmParams {
    const int32_t *offsets;
    int E, rows, N, K;
    int w_tiles;             // weight tiles of 128 * CG columns
    int tok_cap;             // rows per unit at most (a multiple of 16 * CG)
    int row_block;           // row units per block
    int slot_bytes;          // ring slot: W_BYTES + this CTA's rows of a full unit
    int stages;
    int split;               // SPLIT: CTAs that share a unit's k
    int part_kb;             // k-blocks summed in one accumulator: kPartStages or kLongPartStages
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

struct Unit {
    int e;
    int row0;        // first row (in the dispatched matrix)
    int rows;        // rows to store
    int mma_n;       // the same rounded up to the MMA's width
    int w0;          // first weight column of this CTA
};

// Walks a CTA's units in order. What depends on the expert alone is kept, and
// the common case divides once: with five divisions and a search per unit the
// MMA warp spent a thousand cycles between short units.
template <int CG>
struct UnitWalk {
    const Segments &S;
    const GemmParams &p;
    int rank, e, cnt, n_units, each;

    __device__ __forceinline__ UnitWalk(const Segments &seg, const GemmParams &params, int r)
        : S(seg), p(params), rank(r), e(-1), cnt(0), n_units(1), each(1) {}

    __device__ __forceinline__ Unit at(int unit)
    {
        if (e < 0 || unit >= S.unit[e + 1]) {
            e = expert_of(S, p.E, unit);
            cnt = S.count[e];
            n_units = (cnt + p.tok_cap - 1) / p.tok_cap;
            // equal widths: at most tok_cap, which is a multiple of the
            // quantum, so that none of the n_units comes out empty
            constexpr int Q = 16 * CG;
            each = ((cnt + n_units - 1) / n_units + Q - 1) / Q * Q;
        }
        Unit u;
        u.e = e;
        const int local = unit - S.unit[e];
        int wt, j;
        if (n_units <= p.row_block) {
            wt = local / n_units;
            j = local - wt * n_units;
        } else {
            const int span = p.row_block * p.w_tiles;
            const int b = local / span, rem = local - b * span;
            const int left = n_units - b * p.row_block, width = left < p.row_block ? left : p.row_block;
            wt = rem / width;
            j = b * p.row_block + rem - wt * width;
        }
        const int at = j * each;
        u.rows = cnt - at < each ? cnt - at : each;
        u.row0 = S.first[e] + at;
        u.mma_n = (u.rows + 16 * CG - 1) / (16 * CG) * (16 * CG);
        u.w0 = (wt * CG + rank) * BM;
        return u;
    }
};

// Barrier over the four warps of an epilogue group (id: 1 or 2).
__device__ __forceinline__ void epi_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// The same, true in all of them if `ok` is in all.
__device__ __forceinline__ bool epi_all(int id, bool ok)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "r"(id)
        : "memory");
    return r != 0;
}

// 32 TMEM lanes x 8 consecutive fp32 columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&r)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]));
}

// 16 TMEM lanes x 16 consecutive fp32 columns as four 8 x 8 blocks: thread T
// holds lanes T / 4 (r[0], r[1], r[4], r[5]) and T / 4 + 8 (the others), columns
// 2 (T % 4) and the next, of columns 0-7 (r[0..3]) and 8-15 (r[4..7]).
__device__ __forceinline__ void tmem_ld_blocks(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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

template <int DT, int CG, bool KN, bool OUT_F32, bool SPLIT, bool PARTS>
__global__ void __launch_bounds__(THREADS, 1)
grouped_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_a,
                    const GemmParams p)
{
    extern __shared__ uint8_t smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    static_assert(!SPLIT || CG == 1, "a split unit runs on single CTAs");
    static_assert(!PARTS || (OUT_F32 && !SPLIT), "sums of parts in registers");
    constexpr bool TOTAL = !OUT_F32 && !SPLIT;       // an FP32 sum of several parts is PARTS or SPLIT
    const int ways = SPLIT ? p.split : CG;           // CTAs per unit
    const int unit0 = (int)blockIdx.x / ways, unit_step = (int)gridDim.x / ways;
    // this CTA's k-blocks
    const int all_kb = (p.K + BK - 1) / BK, slice = SPLIT ? (int)cluster_ctarank() : 0;
    const int kb_begin = SPLIT ? all_kb * slice / ways : 0;
    const int kb_end = SPLIT ? all_kb * (slice + 1) / ways : all_kb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) { mbar_init(&S.full[s], 1); mbar_init(&S.empty[s], 1); }
        for (int a = 0; a < 2; ++a) { mbar_init(&S.acc_full[a], 1); mbar_init(&S.acc_empty[a], EPI_WARPS * CG); }
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
    UnitWalk<CG> walk(S.seg, p, rank);

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
            // barrier, which expects them all; they may land before it is
            // armed (the phase cannot complete while the arrival is pending)
            const uint32_t bytes = CG * (W_BYTES + u.mma_n / CG * BK * 2);
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                ok = warp_wait<CG>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                if (!ok) break;
                const uint32_t sw = ring + stage * p.slot_bytes, here = smem_u32(&S.full[stage]);
                const uint32_t bar = CG == 2 ? mapa_shared(here, 0) : here;
                expect_tx_on(arm, &S.full[stage], bytes);
                if constexpr (KN) {
                    load_3d_on<CG>(on, sw, &map_w, bar, u.w0, kb * BK, u.e);
                    load_3d_on<CG>(on, sw + W_BYTES / 2, &map_w, bar, u.w0 + 64, kb * BK, u.e);
                } else {
                    load_3d_on<CG>(on, sw, &map_w, bar, kb * BK, u.w0, u.e);
                }
                if (++stage == p.stages) { stage = 0; phase ^= 1u; }
            }
        }
    } else if (warp == 6) {
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
                    load_2d_on<CG>(on, sa + at * BK * 2, &map_a.m[box], bar, kb * BK, row0 + at);
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
        constexpr uint32_t idesc0 = idesc_f16_major<DT>(BM * CG, 0, KN, false);
        const uint32_t on = elect_lane();
        const uint32_t ring = smem_u32(S.ring);
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t used = 0;                               // parity of each accumulator's uses so far
        bool ok = true;
        for (int unit = unit0; unit < total && ok; unit += unit_step) {
            const Unit u = walk.at(unit);
            const uint32_t idesc = idesc0 | ((uint32_t)(u.mma_n >> 3) << 17);
            for (int kb0 = kb_begin; kb0 < kb_end && ok; kb0 += p.part_kb) {
                const int kb1 = kb_end - kb0 < p.part_kb ? kb_end : kb0 + p.part_kb;
                ok = warp_wait<CG>(&S.acc_empty[acc], (used >> acc & 1u) ^ 1u, abort_flag, p.status, p.wait_ns);
                if (!ok) break;
                used ^= 1u << acc;
                const uint32_t d = tmem_base + (uint32_t)(acc * ACC_COLS);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = warp_wait<CG>(&S.full[stage], phase, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t w = ring + stage * p.slot_bytes, a = w + W_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / UK; ++k)
                        umma_on<CG>(on, d, KN ? sdesc_mn_sw128(w + k * UK * 128, W_BYTES / 2) : sdesc_k_sw128(w + k * UK * 2),
                                    sdesc_k_sw128(a + k * UK * 2), idesc, (kb - kb0) | k ? 1u : 0u);
                    commit_on<CG>(on, &S.empty[stage]);
                    if (++stage == p.stages) { stage = 0; phase ^= 1u; }
                }
                if (ok) commit_on<CG>(on, &S.acc_full[acc]);
                acc = next_acc<TOTAL>(acc, kb0 != kb_begin, kb1 == kb_end);
            }
        }
        // every MMA issued must finish before TMEM is released, also where
        // another role has given up
        if (on) {
            umma_commit<CG>(&S.drain);
            mbar_wait(&S.drain, 0, nullptr, p.status, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp >= 2) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                          // TMEM lane quadrant of this warp
        const int group = warp >= 7 ? 1 : 0;             // takes every second chunk of rows
        const int tid = threadIdx.x - (group ? 224 : 64);     // 0..127 in the group
        constexpr int CH = OUT_F32 ? 8 : 16;             // rows per staging buffer
        constexpr int ESZ = OUT_F32 ? 4 : 2;
        constexpr int ROW_BYTES = BM * ESZ;              // staged bytes per row: 512 / 256
        constexpr int PIECES = ROW_BYTES / 16, PER_IT = 128 / PIECES;
        int next = 0, buf = 0, unit = unit0, kb0 = kb_begin;
        uint32_t used = 0;
        Unit u = {};
        // an accumulator is read: another part may have it
        auto release = [&](int acc) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2 && !leader) mbar_arrive_cluster(mapa_shared(smem_u32(&S.acc_empty[acc]), 0));
                else mbar_arrive(&S.acc_empty[acc]);
            }
        };
        float sums[PARTS ? PARTS_CAP / 32 : 1][16];        // PARTS: of this lane's n and the group's rows
        (void)sums;
        // unit by unit, part by part (kb0: the part's first k-block)
        for (; unit < total; kb0 += p.part_kb) {
            if (kb0 >= kb_end) {
                kb0 = kb_begin;
                unit += unit_step;
                if (unit >= total) break;
            }
            if (kb0 == kb_begin) u = walk.at(unit);
            const bool more = kb0 != kb_begin, last = kb_end - kb0 <= p.part_kb;  // adds to the earlier parts; ends the sum
            const int acc = next;
            const uint32_t acc_phase = used >> acc & 1u;
            used ^= 1u << acc;
            next = next_acc<TOTAL>(acc, more, last);
            // a group's warps leave together: none may wait at a barrier for
            // one that has given up
            if (!epi_all(1 + group, mbar_wait<CG>(&S.acc_full[acc], acc_phase, abort_flag, p.status, p.wait_ns))) break;
            tc_fence_after();
            auto tmem_of = [&](int a) { return tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * ACC_COLS); };
            int held = acc;                                  // the accumulator that holds the sum
            if constexpr (TOTAL) {
                // a later part is added to the first one, which stays where it is
                if (more) {
                    held = acc ^ 1;
                    for (int t0 = group * CH; t0 < u.rows; t0 += 2 * CH) {
                        uint32_t v[16], sum[16];
                        tmem_ld16(tmem_of(acc) + t0, v);
                        tmem_ld16(tmem_of(held) + t0, sum);
                        tmem_ld_wait16(v);
                        tmem_ld_wait16(sum);
                        add_to(sum, v);
                        tmem_st16(tmem_of(held) + t0, sum);
                    }
                    tmem_st_wait();
                    release(acc);
                }
                if (!last) continue;
            }
            const uint32_t tbase = tmem_of(held);
            const int piece = tid % PIECES, col = u.w0 + piece * (16 / ESZ);
            uint8_t *out0 = p.out + (int64_t)u.row0 * p.out_row_bytes + (int64_t)col * ESZ;
            const bool whole = p.vec && col + 16 / ESZ <= p.N;
            if constexpr (SPLIT) {
                // the partial sums stay here, [row][n] in FP32
                float *mine = reinterpret_cast<float *>(S.ring + RING_BYTES - PARTIAL_BYTES) + q * 32 + lane;
                for (int t0 = group * 16; t0 < u.rows; t0 += 32) {
                    uint32_t v[16];
                    tmem_ld16(tbase + t0, v);
                    tmem_ld_wait16(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        mine[(t0 + i) * BM] = more ? mine[(t0 + i) * BM] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
                }
            }
            // Stores CH staged rows from row t0 of the unit on; all four warps
            // of the group call, with their part of the rows in the buffer.
            auto store_rows = [&](const uint8_t *stg, int t0) {
                // one barrier per buffer: who passes it has read the other one
                epi_sync(1 + group);
#pragma unroll
                for (int i = 0; i < CH / PER_IT; ++i) {
                    const int t = i * PER_IT + tid / PIECES;
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        stg + t * ROW_BYTES + (OUT_F32 ? piece : piece ^ (t & 7)) * 16);
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
            };
            auto stage_fp32 = [&](const float *v, int t0) {
                uint8_t *stg = S.stg[group][buf], *mine = stg + (q * 32 + lane) * ESZ;
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<float *>(mine + i * ROW_BYTES) = v[i];
                store_rows(stg, t0);
                buf ^= 1;
            };
            if constexpr (PARTS) {
                // this group's rows: 16 of every 32, at most 64
#pragma unroll
                for (int j = 0; j < PARTS_CAP / 32; ++j) {
                    const int t0 = j * 32 + group * 16;
                    if (t0 >= u.rows) continue;
                    uint32_t v[16];
                    tmem_ld16(tbase + t0, v);
                    tmem_ld_wait16(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sums[j][i] = more ? sums[j][i] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
                }
                release(acc);
                if (!last) continue;
#pragma unroll
                for (int j = 0; j < PARTS_CAP / 32; ++j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t0 = j * 32 + group * 16 + h * 8;
                        if (t0 < u.rows) stage_fp32(&sums[j][h * 8], t0);
                    }
                }
            } else {
                for (int t0 = group * CH; !SPLIT && t0 < u.rows; t0 += 2 * CH) {
                    if constexpr (OUT_F32) {
                        uint32_t v[8];
                        tmem_ld8(tbase + t0, v);
                        tmem_ld_wait8(v);
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i]);
                        stage_fp32(f, t0);
                    } else {
                        // blocks of 8 n by 8 rows, rounded, leave transposed; the 16-byte
                        // pieces of row t are permuted by t % 8, so that a block's eight
                        // rows (256 bytes apart) meet no bank twice
                        const uint8_t *stg = S.stg[group][buf];
                        uint32_t lo[8], hi[8];               // lanes 0-15, 16-31 of the quadrant
                        tmem_ld_blocks(tbase + t0, lo);
                        tmem_ld_blocks(tbase + (16u << 16) + t0, hi);
                        tmem_ld_wait8(lo);
                        tmem_ld_wait8(hi);
                        const int t = lane & 7, at = q * 4 + (lane >> 3);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            auto block = [&](const uint32_t (&v)[8], int i) {
                                return pack2<DT>(__uint_as_float(v[c * 4 + i]), __uint_as_float(v[c * 4 + i + 1]));
                            };
                            store_blocks_transposed(smem_u32(stg + (c * 8 + t) * ROW_BYTES + ((at ^ t) << 4)),
                                                    block(lo, 0), block(lo, 2), block(hi, 0), block(hi, 2));
                        }
                        store_rows(stg, t0);
                        buf ^= 1;
                    }
                }
                release(held);
            }
        }
    }

    if constexpr (SPLIT) {
        // every CTA's partial sums are written; each adds its rows
        __syncwarp();
        cluster_sync();
        if (unit0 < total) {
            const Unit u = UnitWalk<CG>(S.seg, p, rank).at(unit0);
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
                else reinterpret_cast<typename Elem<DT>::T *>(dst)[u.w0 + n] = Elem<DT>::from_f(sum);
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

// Opts this kernel instance in to its shared memory, and (pairs) asks how many
// clusters the GPU holds at once, once per device.
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kernel, int cg, std::atomic<int> *cache, int *ctas)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kCachedDevices;
    int n = cached ? cache[dev].load() : 0;
    if (n == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (err != cudaSuccess) return err;
        n = device_sm_count();
        if (cg == 2) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(n & ~1));
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = kSmemBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int pairs = 0;
            err = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
            if (err != cudaSuccess) return err;
            if (pairs < 1) return cudaErrorInvalidConfiguration;
            n = 2 * pairs;
        }
        if (cached) cache[dev].store(n);
    }
    *ctas = n;
    return cudaSuccess;
}

template <int DT, int CG, bool KN, bool OUT_F32, bool SPLIT, bool PARTS>
cudaError_t launch_kernel(int64_t units, const CUtensorMap &mw, const RowMaps &ma, const GemmParams &p,
                          cudaStream_t s)
{
    static std::atomic<int> cache[kCachedDevices];
    auto kernel = grouped_gemm_kernel<DT, CG, KN, OUT_F32, SPLIT, PARTS>;
    int ctas = 0;
    cudaError_t err = prepare_kernel(kernel, CG, cache, &ctas);
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

template <int DT, int CG, bool SPLIT>
cudaError_t launch_cg(const void *a, int64_t lda, const int32_t *offsets, int64_t rows, const void *w,
                      int E, int64_t N, int64_t K, bool kn, void *out, int64_t ldo, bool out_f32,
                      int tok_cap, int split, unsigned *status, cudaStream_t s)
{
    const CUtensorMapDataType tdt =
        DT == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap mw;
    RowMaps ma;
    bool ok = kn ? encode_3d(&mw, tdt, w, (uint64_t)N, (uint64_t)K, (uint64_t)E, 64, BK)
                 : encode_3d(&mw, tdt, w, (uint64_t)K, (uint64_t)N, (uint64_t)E, BK, BM);
    for (int i = 0; i < 4; ++i)
        ok = ok && encode_2d_strided(&ma.m[i], tdt, a, (uint64_t)K, (uint64_t)rows, (uint64_t)lda * 2, BK, 128u >> i);
    if (!ok) return cudaErrorInvalidValue;
    GemmParams p{};
    p.offsets = offsets;
    p.E = E;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.w_tiles = (int)((N + BM * CG - 1) / (BM * CG));
    p.tok_cap = tok_cap;
    const int64_t block = kRowBlockBytes / (tok_cap * K * 2), most = (rows + tok_cap - 1) / tok_cap;
    p.row_block = (int)(block < 1 ? 1 : block > most ? most : block);
    p.slot_bytes = W_BYTES + tok_cap / CG * BK * 2;
    const int slots = (RING_BYTES - (SPLIT ? PARTIAL_BYTES : 0)) / p.slot_bytes;
    p.stages = slots < MAX_STAGES ? slots : MAX_STAGES;
    p.split = split;
    p.out = static_cast<uint8_t *>(out);
    p.out_row_bytes = ldo * (out_f32 ? 4 : 2);
    p.vec = p.out_row_bytes % 16 == 0;
    p.status = status;
    p.part_kb = out_f32 ? kPartStages : kLongPartStages<DT>;
    // a wait may last one unit's whole reduction, a producer's as many short units
    // as the ring has stages
    p.wait_ns = wait_limit_ns() + work_ns((uint64_t)((K + BK - 1) / BK + p.stages), (uint64_t)p.stages);
    // an upper bound: every expert adds at most one unit that is not full
    const int64_t units = (rows / tok_cap + (rows < E ? rows : E)) * p.w_tiles;
    if constexpr (!SPLIT) {
        if (out_f32 && (K + BK - 1) / BK > kPartStages)
            return kn ? launch_kernel<DT, CG, true, true, false, true>(units, mw, ma, p, s)
                      : launch_kernel<DT, CG, false, true, false, true>(units, mw, ma, p, s);
    }
    if (out_f32)
        return kn ? launch_kernel<DT, CG, true, true, SPLIT, false>(units, mw, ma, p, s)
                  : launch_kernel<DT, CG, false, true, SPLIT, false>(units, mw, ma, p, s);
    return kn ? launch_kernel<DT, CG, true, false, SPLIT, false>(units, mw, ma, p, s)
              : launch_kernel<DT, CG, false, false, SPLIT, false>(units, mw, ma, p, s);
}

template <int DT>
cudaError_t launch_dt(const void *a, int64_t lda, const int32_t *offsets, int64_t rows, const void *w,
                      int E, int64_t N, int64_t K, bool kn, void *out, int64_t ldo, bool out_f32,
                      unsigned *status, cudaStream_t s)
{
    // Few units (of the single form's 64 rows by 128 columns): split k over as
    // many CTAs, 2 to 8, as the GPU has room for and as leave each four k-blocks.
    const int64_t units = (rows / SPLIT_CAP + (rows < E ? rows : E)) * ((N + BM - 1) / BM);
    const int64_t num_kb = (K + BK - 1) / BK, sms = device_sm_count();
    int split = 1;
    while (split < 8 && units * split * 2 <= sms && num_kb >= split * 2 * 4) split *= 2;
    if (split > 1)
        return launch_cg<DT, 1, true>(a, lda, offsets, rows, w, E, N, K, kn, out, ldo, out_f32, SPLIT_CAP,
                                      split, status, s);
    // Pairs or single CTAs, by the average rows of an expert. 64 experts, N = K =
    // 2048 (16 experts, N = K = 4096), us at 4, 32, 48, 64, 96 rows on average:
    // singles 82.7 87.0 89.4 93.7 113 (87.1 89.9 91.5 101 106),
    // pairs   87.9 92.9 93.5 95.2 98.1 (91.9 95.2 95.1 97.0 98.6) in 16 bits;
    // FP32 outputs, there and at 192: singles 82.8 87.3 90.0 91.6 114 156 (86.5
    // 89.2 92.0 92.0 108 151), pairs 87.4 93.2 95.4 97.2 101 135 (92.2 94.8 97.0
    // 97.7 101 126).
    if (rows >= 64 * (int64_t)E)
        return launch_cg<DT, 2, false>(a, lda, offsets, rows, w, E, N, K, kn, out, ldo, out_f32,
                                       out_f32 && num_kb > kPartStages ? PARTS_CAP : 256, 1, status, s);
    return launch_cg<DT, 1, false>(a, lda, offsets, rows, w, E, N, K, kn, out, ldo, out_f32, 64, 1, status, s);
}

}  // namespace

cudaError_t launch_grouped_gemm_tc(int dt, const void *a, int64_t lda, const int32_t *offsets,
                                   int64_t rows, const void *w, int E, int64_t N, int64_t K,
                                   bool transposed, void *out, int64_t ldo, bool out_f32,
                                   unsigned *status, cudaStream_t s)
{
    if (dt == DT_BF16)
        return launch_dt<DT_BF16>(a, lda, offsets, rows, w, E, N, K, transposed, out, ldo, out_f32, status, s);
    return launch_dt<DT_F16>(a, lda, offsets, rows, w, E, N, K, transposed, out, ldo, out_f32, status, s);
}

}  // namespace moe
