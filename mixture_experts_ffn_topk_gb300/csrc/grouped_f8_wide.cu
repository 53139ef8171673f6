// grouped_f8_wide.cu -- grouped products of e4m3 rows and matrices with FP32 scales
// per block of 128, for experts of many rows (see grouped_f8.cu for the product).
//
// Here the rows take the MMA's M side: M = 256 over a CTA pair, 128 rows per CTA, by
// N = 256 weight columns. A TMEM lane is a row and a column of the accumulator a
// weight column, so the two scales of a block are one number for all 128 columns
// that a thread of the epilogue reads: it adds a block to its sums with one
// multiply-add per value and nothing else. (With rows as columns each column has a
// scale of its own, and fetching those from shared memory, 512 bytes per warp for
// every 16-byte broadcast, took 1000 cycles of a block whose MMAs take 512.) An
// expert's last unit may leave half a tile idle: with up to 64 rows in each expert the
// other form is faster, with 64 on average and rows as a router spreads them this one
// (launch_grouped_gemm_f8).
//
// What bounds it is the epilogue's latency per block of k: a barrier, 128 columns out
// of TMEM, 128 multiply-adds (256 issue cycles of an SM partition's two warps), a
// barrier; some 800 cycles and 100 of a unit's stores, where the MMAs take 512. 16384
// rows on 8 experts of 4096 x 4096 take 218 us in a graph of ten calls (214 without
// scales_apart: one flag to read and one branch per four blocks). In an older form,
// of 247 us by single calls, 191 were left without TMEM reads and multiply-adds, 216
// with the reads alone, 243 with the multiply-adds alone. Tried: paired
// multiply-adds (320 against 273 us), four groups of epilogue warps with 64 columns
// each (302), accumulators of 128 columns, four in turn (284).
//
// Per CTA (one per SM, 384 threads, persistent over the units):
//   warp 0   TMA producer of the weights: half of 256 n x 128 k (16 KiB) per stage;
//   warp 2   TMA producer of its 128 rows x 128 k (16 KiB), into the same stages;
//   warp 1   of the even CTA: tcgen05.mma issuer, K = 32 per instruction, one
//            accumulator of 256 columns per block, two in turn;
//   warp 3   scales of its rows, four blocks at a time, and the unit they belong to;
//   warps 4-7, 8-11  one group per 128 columns: sums stay in registers until the last
//            block, and rows leave in 32-byte stores.
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

constexpr int ROWS = 128;                // of a CTA
constexpr int COLS = 256;                // of a pair
constexpr int SLOT_BYTES = W_BYTES + ROWS * BK;
constexpr int STAGES = 6;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int ACCS = 2;
constexpr int TMEM_COLS = ACCS * COLS;
constexpr int SCALE_STAGES = 3, SCALE_KB = 4;        // scales are staged for four blocks at a time
// Units that the scales' warp announces. It begins a unit when every warp of the
// epilogue has taken scales of the third unit before it, at the least, and so has read
// and stored the fourth.
constexpr int UNITS = 4;
static_assert(UNITS > SCALE_STAGES && (UNITS & (UNITS - 1)) == 0, "");

struct __align__(1024) Smem {
    uint8_t ring[STAGES * SLOT_BYTES];
    float scale[SCALE_STAGES][ROWS][SCALE_KB];
    float w_scale[SCALE_STAGES][2][SCALE_KB];
    int plain[SCALE_STAGES];             // the products of these scales need no shift (scales_apart)
    int4 unit[UNITS];                    // first row, rows, first column
    uint64_t scale_full[SCALE_STAGES];
    uint64_t scale_empty[SCALE_STAGES];
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t acc_full[ACCS];
    uint64_t acc_empty[ACCS];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int warp_sum[THREADS / 32];
    Segments seg;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;       // + alignment slack
static_assert(kSmemBytes <= 232448, "one CTA's shared memory");

struct WideParams {
    const int32_t *offsets;
    const float *a_scales;   // [rows, KB]
    const float *w_scales;   // [E, NB, KB] or [E, KB, NB]
    int E, rows, N, K;
    int w_tiles;             // weight tiles of 256 columns
    int tok_cap;             // rows per unit at most: 256
    int row_block;           // row units per block
    int out_bf16;            // 16-bit outputs: BF16 or F16
    uint8_t *out;
    int64_t out_row_bytes;
    int align;               // rows of out start on this many bytes (32, 16 or less)
    unsigned *status;
    uint64_t wait_ns;
};

__device__ __forceinline__ void store32(uint8_t *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The four MMAs of a block and the commits of its stage and accumulator, under one
// predicate. alo, blo: the low words of the operands' descriptors, whose high word is
// the same; a step of 32 k is 32 bytes further, or 32 rows of 128 in an MN-major B.
template <bool KN>
__device__ __forceinline__ void block_mmas(uint32_t on, uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi,
                                           uint32_t idesc, uint32_t empty, uint32_t full)
{
    constexpr uint32_t SB = KN ? UK * 128 / 16 : UK / 16;
    static_assert(BK / UK == 4 && UK / 16 == 2, "four steps, two units of 16 bytes each");
    asm volatile(
        "{\n\t.reg .pred q, p0, p1;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t.reg .b16 m;\n\t"
        "setp.ne.u32 q, %0, 0;\n\tsetp.ne.u32 p0, 0, 0;\n\tsetp.eq.u32 p1, 0, 0;\n\t"
        "mov.b64 a, {%2, %4};\n\tmov.b64 b, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%1], a, b, %5, p0;\n\t"
        "add.u32 x, %2, 2;\n\tadd.u32 y, %3, %8;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%1], a, b, %5, p1;\n\t"
        "add.u32 x, %2, 4;\n\tadd.u32 y, %3, %9;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%1], a, b, %5, p1;\n\t"
        "add.u32 x, %2, 6;\n\tadd.u32 y, %3, %10;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%1], a, b, %5, p1;\n\t"
        "mov.b16 m, 3;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6], m;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%7], m;\n\t}"
        ::"r"(on), "r"(d), "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(empty), "r"(full), "n"(SB), "n"(2 * SB),
          "n"(3 * SB)
        : "memory");
}

template <bool KN, bool OUT_F32>
__global__ void __launch_bounds__(THREADS, 1)
grouped_f8_wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                       const WideParams p)
{
    extern __shared__ uint8_t smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int unit0 = (int)blockIdx.x / 2, unit_step = (int)gridDim.x / 2;
    const int num_kb = (p.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&S.full[s], 1); mbar_init(&S.empty[s], 1); }
        for (int a = 0; a < ACCS; ++a) { mbar_init(&S.acc_full[a], 1); mbar_init(&S.acc_empty[a], 2 * EPI_WARPS); }
        for (int s = 0; s < SCALE_STAGES; ++s) { mbar_init(&S.scale_full[s], 1); mbar_init(&S.scale_empty[s], EPI_WARPS); }
        mbar_init(&S.drain, 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc<2>(&S.tmem_base, TMEM_COLS);
        tmem_relinquish<2>();
    }
    pdl_wait();
    pdl_launch_dependents();
    load_segments<THREADS>(S.seg, S.warp_sum, p.offsets, p.E, p.rows, p.status,
                           [&](int cnt) { return (cnt + p.tok_cap - 1) / p.tok_cap * p.w_tiles; });
    tc_fence_before();
    // makes each CTA's barrier initialisation visible to the other before any
    // copy or arrival targets it
    cluster_sync();
    tc_fence_after();

    const uint32_t tmem_base = S.tmem_base;
    const int total = S.seg.unit[p.E];
    volatile int *abort_flag = &S.abort;
    UnitWalk<2, WideParams> walk(S.seg, p, 0);
    // columns of a unit's tile; [E, N, K] weights cut the last one short, in halves
    // of whole 16
    auto cols_of = [&](int n0) { return KN || p.N - n0 >= COLS ? COLS : (p.N - n0 + 31) / 32 * 32; };

    // 384 threads start with 168 registers each: 128 * (72 + 2 * 216) is the same
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
            // ------------------------------------------- TMA producer: weights
            const uint32_t on = elect_lane(), arm = leader ? on : 0u;
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const int n0 = u.w0 + rank * (cols_of(u.w0) / 2);
                for (int kb = 0; kb < num_kb; ++kb) {
                    ok = warp_wait<1>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    // all copies of both CTAs complete on the leader's barrier
                    const uint32_t bar = mapa_shared(smem_u32(&S.full[stage]), 0);
                    expect_tx_on(arm, &S.full[stage], 2 * SLOT_BYTES);
                    if constexpr (KN) load_3d_on<2>(on, ring + stage * SLOT_BYTES, &map_w, bar, n0, kb * BK, u.e);
                    else load_3d_on<2>(on, ring + stage * SLOT_BYTES, &map_w, bar, kb * BK, n0, u.e);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
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
                for (int kb = 0; kb < num_kb; ++kb) {
                    ok = warp_wait<1>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    load_2d_on<2>(on, ring + stage * SLOT_BYTES + W_BYTES, &map_a,
                                  mapa_shared(smem_u32(&S.full[stage]), 0), kb * BK, u.row0 + rank * ROWS);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        } else if (warp == 1 && leader) {
            // ------------------------------------------------------ MMA issuer
            const uint32_t on = elect_lane();
            const uint32_t ring = smem_u32(S.ring);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            const uint64_t da = sdesc_k_sw128(ring + W_BYTES);
            const uint64_t db = KN ? sdesc_mn_sw128(ring, W_BYTES) : sdesc_k_sw128(ring);
            uint32_t alo = (uint32_t)da, blo = (uint32_t)db;
            const uint32_t hi = (uint32_t)(da >> 32);
            const uint32_t empty0 = smem_u32(&S.empty[0]), full0 = smem_u32(&S.acc_full[0]);
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const uint32_t idesc = idesc_e4m3(2 * ROWS, cols_of(u.w0), false, KN);
                for (int kb = 0; kb < num_kb; ++kb) {
                    ok = warp_wait_both(&S.acc_empty[acc], acc_phase ^ 1u, &S.full[stage], phase, abort_flag,
                                        p.status, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    block_mmas<KN>(on, tmem_base + (uint32_t)(acc * COLS), alo, blo, hi, idesc, empty0 + stage * 8,
                                   full0 + acc * 8);
                    alo += SLOT_BYTES / 16;
                    blo += SLOT_BYTES / 16;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                        alo -= STAGES * (SLOT_BYTES / 16);
                        blo -= STAGES * (SLOT_BYTES / 16);
                    }
                    if (++acc == ACCS) { acc = 0; acc_phase ^= 1u; }
                }
            }
            // every MMA issued must finish before TMEM is released, also where
            // another role has given up
            if (on) {
                umma_commit<2>(&S.drain);
                mbar_wait(&S.drain, 0, nullptr, p.status, kDrainLimitNs);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ------------------------------------------------------ scales
            // of this CTA's rows, four blocks at a time: four lanes to a row. A stage is
            // handed over when the next one's copies are under way; whether its products
            // stay within FP32's range is found here, where there is time for it (in the
            // epilogue the same took 6 to 8 % of the whole)
            const int n_blocks = (p.N + BM - 1) / BM, k = lane & 3;
            int stage = 0, slot = 0, last = -1, last_rows = 0, last_n = 0;
            uint32_t phase = 0;
            bool ok = true;
            auto hand_over = [&]() {
                __syncwarp();
                bool plain = lane >= 8 || k >= last_n || plain_scale(S.w_scale[last][lane >> 2 & 1][k]);
#pragma unroll
                for (int i = 0; i < ROWS / 32; ++i) {
                    const float4 s = *reinterpret_cast<const float4 *>(S.scale[last][lane + 32 * i]);
                    plain = plain && (lane + 32 * i >= last_rows ||
                                      (plain_scale(s.x) && (last_n < 2 || plain_scale(s.y)) &&
                                       (last_n < 3 || plain_scale(s.z)) && (last_n < 4 || plain_scale(s.w))));
                }
                plain = __all_sync(0xffffffffu, plain);
                if (!plain) {                    // rare: the products themselves
                    plain = true;
#pragma unroll 1
                    for (int r = lane; r < last_rows; r += 32)
#pragma unroll 1
                        for (int b = 0; b < SCALE_KB && b < last_n; ++b)
                            for (int g = 0; g < 2; ++g) {
                                float s;
                                plain = plain && scales_apart(S.scale[last][r][b], S.w_scale[last][g][b], s) == 0;
                            }
                    plain = __all_sync(0xffffffffu, plain);
                }
                if (lane == 0) S.plain[last] = plain;
                arrive_on(lane == 0, &S.scale_full[last]);
            };
            for (int unit = unit0; unit < total && ok; unit += unit_step) {
                const Unit u = walk.at(unit);
                const int rows = min(u.rows - rank * ROWS, ROWS), nb = min(u.w0 / BM + (lane >> 2 & 1), n_blocks - 1);
                for (int kb = 0; kb < num_kb; kb += SCALE_KB) {
                    ok = warp_wait<1>(&S.scale_empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    if (kb + k < num_kb) {
                        const float *src = p.a_scales + (int64_t)(u.row0 + rank * ROWS + lane / 4) * num_kb + kb + k;
                        float *dst = &S.scale[stage][lane / 4][k];
                        for (int r = lane / 4; r < rows; r += 8, dst += 8 * SCALE_KB, src += 8 * num_kb) copy4_async(dst, src);
                        if (lane < 8)
                            copy4_async(&S.w_scale[stage][lane >> 2][k],
                                        p.w_scales + (KN ? ((int64_t)u.e * num_kb + kb + k) * n_blocks + nb
                                                         : ((int64_t)u.e * n_blocks + nb) * num_kb + kb + k));
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (lane == 0 && kb == 0) S.unit[slot] = make_int4(u.row0, u.rows, u.w0, 0);
                    if (last >= 0) {
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        hand_over();
                    }
                    last = stage;
                    last_rows = rows;
                    last_n = num_kb - kb;
                    if (++stage == SCALE_STAGES) { stage = 0; phase ^= 1u; }
                }
                slot = (slot + 1) % UNITS;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (ok && last >= 0) hand_over();
        }
    } else {
        // ------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int q = warp & 3;                          // TMEM lane quadrant of this warp
        const int group = warp >= 8 ? 1 : 0;             // columns [128 group, + 128)
        const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16) + group * BM;
        const uint32_t acc_free = mapa_shared(smem_u32(&S.acc_empty[0]), 0);
        int stage = 0;
        uint32_t phase = 0, block = 0, slot = 0;     // blocks so far: accumulators and phases go by them
        for (int unit = unit0; unit < S.seg.unit[p.E]; unit += unit_step) {
            // the unit comes with its first scales: to search for it took the epilogue
            // some 1000 cycles (384 rows x 64 experts, 2048 -> 1408: 112 against 106 us)
            if (!warp_wait<1>(&S.scale_full[stage], phase, abort_flag, p.status, p.wait_ns)) break;
            // and is read again for its stores, so that it takes no registers beside the
            // sums (no spills; 1 %)
            const volatile int4 &u = S.unit[slot];
            slot = (slot + 1) % UNITS;
            float sums[4][32];                           // [chunk of 32 columns][column]
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 32; ++i) sums[j][i] = 0.0f;
            // NJ chunks of 32 columns: all, or none where the tile ends before this group
            // (columns past a narrow tile are added up and not stored). Four blocks per
            // round of scales, two of them unrolled: what a block costs beside its
            // multiply-adds is a chain of short instructions (1070 -> 950 cycles per block)
            auto add_blocks = [&](auto chunks) {
                constexpr int NJ = decltype(chunks)::value;
                // a block's columns, on their way out of TMEM 16 at a time while the 16
                // before are added up; SHIFT: times k first
                auto add_block = [&](auto shift, float s, float k) {
                    const uint32_t acc = block & 1u;
                    if (!__all_sync(0xffffffffu, mbar_try_wait(&S.acc_full[acc], block >> 1 & 1u)) &&
                        !warp_wait<1>(&S.acc_full[acc], block >> 1 & 1u, abort_flag, p.status, p.wait_ns))
                        return false;
                    tc_fence_after();
                    const uint32_t tbase = tlane + acc * COLS;
                    uint32_t v[2][16];
                    if constexpr (NJ > 0) tmem_ld16(tbase, v[0]);
#pragma unroll
                    for (int j = 0; j < 2 * NJ; ++j) {
                        tmem_ld_wait16(v[j & 1]);
                        if (j + 1 < 2 * NJ) tmem_ld16(tbase + (j + 1) * 16, v[(j + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float f = __uint_as_float(v[j & 1][i]);
                            if constexpr (decltype(shift)::value) f *= k;
                            sums[j / 2][j % 2 * 16 + i] = fmaf(f, s, sums[j / 2][j % 2 * 16 + i]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    arrive_relaxed_on(lane == 0, acc_free + acc * 8);
                    ++block;
                    return true;
                };
                auto release = [&]() {
                    __syncwarp();
                    arrive_on(lane == 0, &S.scale_empty[stage]);
                    if (++stage == SCALE_STAGES) { stage = 0; phase ^= 1u; }
                };
                int kb = 0;
                for (; kb < num_kb; kb += SCALE_KB) {
                    if (!warp_wait<1>(&S.scale_full[stage], phase, abort_flag, p.status, p.wait_ns)) return false;
                    const float4 sa = *reinterpret_cast<const float4 *>(S.scale[stage][q * 32 + lane]);
                    const float4 sw = *reinterpret_cast<const float4 *>(S.w_scale[stage][group]);
                    if (!S.plain[stage]) break;
                    float s4[SCALE_KB] = {sa.x * sw.x, sa.y * sw.y, sa.z * sw.z, sa.w * sw.w};
                    release();
                    const int n = num_kb - kb;
#pragma unroll 2
                    for (int b = 0; b < SCALE_KB; ++b) {
                        if (b >= n) break;
                        const float s = s4[0];
#pragma unroll
                        for (int i = 0; i + 1 < SCALE_KB; ++i) s4[i] = s4[i + 1];
                        if (!add_block(std::false_type(), s, 1.0f)) return false;
                    }
                }
                // the rest of a unit in which a product of scales leaves FP32's range
#pragma unroll 1
                for (; kb < num_kb; kb += SCALE_KB) {
                    if (!warp_wait<1>(&S.scale_full[stage], phase, abort_flag, p.status, p.wait_ns)) return false;
#pragma unroll 1
                    for (int b = 0; b < SCALE_KB && kb + b < num_kb; ++b) {
                        float s;
                        const float k = shift_of(scales_apart(S.scale[stage][q * 32 + lane][b], S.w_scale[stage][group][b], s));
                        if (!add_block(std::true_type(), s, k)) return false;
                    }
                    release();
                }
                return true;
            };
            const bool ok = cols_of(u.z) > group * BM ? add_blocks(std::integral_constant<int, 4>())
                                                      : add_blocks(std::integral_constant<int, 0>());
            if (!ok) break;
            const int mine = rank * ROWS + q * 32 + lane;            // this thread's row of the unit
            if (mine >= u.y) continue;
            constexpr int ESZ = OUT_F32 ? 4 : 2, PER = 32 / ESZ;         // columns in 32 bytes
            const int col0 = u.z + group * BM;
            uint8_t *out = p.out + (int64_t)(u.x + mine) * p.out_row_bytes + (int64_t)col0 * ESZ;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int b = 0; b < 32 / PER; ++b) {
                    const int col = j * 32 + b * PER;
                    if (col0 + col >= p.N) continue;
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float *f = &sums[j][b * PER + i * PER / 8];
                        if constexpr (OUT_F32) v[i] = __float_as_uint(f[0]);
                        else v[i] = p.out_bf16 ? float2_to_bf16x2(f[0], f[1]) : float2_to_f16x2(f[0], f[1]);
                    }
                    uint8_t *to = out + col * ESZ;
                    if (p.align >= 16 && col0 + col + PER <= p.N) {
                        if (p.align == 32) {
                            store32(to, v);
                        } else {
                            reinterpret_cast<uint4 *>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
                            reinterpret_cast<uint4 *>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            if (col0 + col + i >= p.N) continue;
                            if constexpr (OUT_F32) reinterpret_cast<uint32_t *>(to)[i] = v[i];
                            else reinterpret_cast<uint16_t *>(to)[i] = (uint16_t)(v[i / 2] >> (i & 1) * 16);
                        }
                    }
                }
            }
        }
    }

    // ------------------------------------------------------------ teardown
    __syncthreads();
    if (*abort_flag) let_copies_land();
    // both CTAs stay (their shared memory is read by the leader's MMAs and
    // signalled by its commits) until both are done
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<2>(tmem_base, TMEM_COLS);
    }
}

// ---- host side ---------------------------------------------------------------

template <bool KN, bool OUT_F32>
cudaError_t launch_kernel(int64_t units, const CUtensorMap &mw, const CUtensorMap &ma, const WideParams &p,
                          cudaStream_t s)
{
    static std::atomic<int> cache[kCachedDevices];
    auto kernel = grouped_f8_wide_kernel<KN, OUT_F32>;
    int ctas = 0;
    cudaError_t err = prepare_kernel(kernel, 2, THREADS, kSmemBytes, cache, &ctas);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * units < ctas ? 2 * units : ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, mw, ma, p);
}

}  // namespace

cudaError_t launch_grouped_gemm_f8_wide(const GroupedF8 &g, unsigned *status, cudaStream_t s)
{
    const uint64_t N = (uint64_t)g.N, K = (uint64_t)g.K, E = (uint64_t)g.E;
    CUtensorMap mw, ma;
    const bool ok = (g.transposed ? encode_bytes(&mw, g.w, 3, {N, K, E}, {N, N * K}, BK)
                                  : encode_bytes(&mw, g.w, 3, {K, N, E}, {K, N * K}, BM)) &&
                    encode_bytes(&ma, g.a, 2, {K, (uint64_t)g.rows, 1}, {(uint64_t)g.lda, 0}, ROWS);
    if (!ok) return cudaErrorInvalidValue;
    WideParams p{};
    p.offsets = g.offsets;
    p.a_scales = g.a_scales;
    p.w_scales = g.w_scales;
    p.E = g.E;
    p.rows = (int)g.rows;
    p.N = (int)g.N;
    p.K = (int)g.K;
    p.w_tiles = (int)((g.N + COLS - 1) / COLS);
    p.tok_cap = 2 * ROWS;
    const int64_t block = kRowBlockBytes / (p.tok_cap * g.K), most = (g.rows + p.tok_cap - 1) / p.tok_cap;
    p.row_block = (int)(block < 1 ? 1 : block > most ? most : block);
    p.out_bf16 = g.out_dt == DT_BF16;
    p.out = static_cast<uint8_t *>(g.out);
    p.out_row_bytes = g.ldo * (g.out_dt == DT_F32 ? 4 : 2);
    const uint64_t at = reinterpret_cast<uintptr_t>(g.out) | (uint64_t)p.out_row_bytes;
    p.align = at % 32 == 0 ? 32 : at % 16 == 0 ? 16 : 1;
    p.status = status;
    // a wait may last one unit's whole reduction, a producer's as many short units
    // as the ring has stages
    p.wait_ns = wait_limit_ns() + work_ns(2 * (uint64_t)((g.K + BK - 1) / BK + STAGES), (uint64_t)STAGES);
    // an upper bound: every expert adds at most one unit that is not full
    const int64_t units = (g.rows / p.tok_cap + (g.rows < g.E ? g.rows : g.E)) * p.w_tiles;
    if (g.out_dt == DT_F32)
        return g.transposed ? launch_kernel<true, true>(units, mw, ma, p, s) : launch_kernel<false, true>(units, mw, ma, p, s);
    return g.transposed ? launch_kernel<true, false>(units, mw, ma, p, s) : launch_kernel<false, false>(units, mw, ma, p, s);
}

}  // namespace moe
