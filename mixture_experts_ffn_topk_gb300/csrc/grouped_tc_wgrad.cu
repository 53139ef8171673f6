// grouped_tc_wgrad.cu -- weight gradient of a grouped product on tcgen05.
//
//   grad_w[e][n, k] (+)= sum over the rows r of expert e of grad[r, n] a[r, k]
//
// BF16 / F16 operands, FP32 accumulation in tensor memory, FP32 or 16-bit
// output. Both operands are read across their rows: TMA boxes of 64 columns
// (128 bytes) by 64 rows, 128-byte swizzle, described to the MMA as MN-major.
// An expert's rows start and end anywhere, so its last box of 64 rows runs
// into the next expert's. The MMA reduces 16 rows at a time: steps past the
// segment are left out, and the at most 15 foreign rows of the last step are
// set to zero in shared memory, in both operands (a NaN there would survive
// a zero in one), by a warp that stands between that stage's copies and its
// MMAs. No tensor map depends on the offsets, no workspace is needed.
//
// Per CTA (one per SM, 256 threads, persistent over the units):
//   warps 0, 7 TMA producers: 128 columns of grad (16 KiB), 256 / CG of a;
//   warp 1     tcgen05.mma issuer, M = 128 * CG by N up to 256;
//   warps 2-5  epilogue: 32 rows x 64 bytes at a time into a swizzled staging
//              buffer that a TMA store carries off, two buffers per warp, so
//              that the warp only reads tensor memory and fills buffers; the
//              store clips the tile at the matrix's edges;
//   warp 6     zeroes foreign rows of a segment's last stage.
// CTA pairs (CG = 2): M = 256, each CTA holds 128 columns of grad and half of
// a's; the even CTA issues the MMAs.
// Few units (narrow matrices) and long segments: a cluster of 2, 4 or 8 single
// CTAs shares each unit's rows (SPLIT; FP32 gradients in units of 128 columns);
// the FP32 partial sums meet through distributed shared memory, each CTA adding its share of
// the columns in rank order.
// Gradients are summed in parts, of kPartStages stages (FP32) or kLongPartStages
// (16 bits), each in an accumulator of its own. The total stays in the first
// part's accumulator (TOTAL), and the later parts, all in the other one, wait
// until the part before is added; the parts of FP32 gradients that a cluster
// shares are added in shared memory. (Sums in the epilogue's registers, which let
// the next part run meanwhile but hold units of 128 columns at most, took 1.10 ms
// on 8 experts of 4096 rows, N = K = 4096, where this takes 0.76.)
// Units run over (expert, tile of the wider matrix, tile of the narrower one),
// the last fastest: the narrower operand's segment stays in L2 while the wider
// one passes once.
//
// Every wait is bounded, as in grouped_tc.cu.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "grouped.cuh"
#include "grouped_issue.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int BM = 128;                  // rows of grad_w per CTA
constexpr int BK = 64;                   // rows reduced per stage
constexpr int UK = 16;                   // rows reduced per tcgen05.mma
constexpr int BOX_BYTES = 64 * BK * 2;   // 64 columns x 64 rows
constexpr int G_BYTES = 2 * BOX_BYTES;
// Columns of grad_w per unit; half as many for FP32 sums of parts that are
// added in shared memory (SPLIT).
template <bool HALF>
constexpr int BN = HALF ? 128 : 256;
template <int CG, bool HALF>
constexpr int SLOT_BYTES = G_BYTES + BN<HALF> / 64 / CG * BOX_BYTES;
constexpr int RING_BYTES = 192 << 10;
template <int CG, bool HALF>
constexpr int STAGES = CG == 2 ? 6 : 4;
template <bool HALF>
constexpr int PARTIAL_AT = HALF ? STAGES<1, true> * SLOT_BYTES<1, true> : 0;  // SPLIT: the sums, [column][row]
static_assert(STAGES<1, false> * SLOT_BYTES<1, false> <= RING_BYTES &&
              STAGES<2, false> * SLOT_BYTES<2, false> <= RING_BYTES &&
              PARTIAL_AT<true> + BN<true> * BM * 4 <= RING_BYTES && BN<false> * BM * 4 <= RING_BYTES, "the ring");
constexpr int MAX_STAGES = 6;
constexpr int ACC_COLS = 256;
constexpr int TMEM_COLS = 2 * ACC_COLS;
constexpr int THREADS = 256;
constexpr int STG_ROW_BYTES = 64;        // staged bytes per row of grad_w
constexpr int STG_BYTES = 32 * STG_ROW_BYTES;
constexpr uint64_t kDrainLimitNs = 100000000ull;

struct __align__(1024) Smem {
    uint8_t ring[RING_BYTES];
    uint8_t stg[4][2][STG_BYTES];
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t tail_in[MAX_STAGES];        // this CTA's copies of a stage with foreign rows
    uint64_t tail_out[MAX_STAGES];       // (leader) the rows of both CTAs are zeroed
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

struct WgradParams {
    const int32_t *offsets;
    int E, rows, N, K;
    int n_tiles, k_tiles;
    int n_fast;              // the n tile runs fastest (grad is the narrower operand)
    int split;               // SPLIT: CTAs that share a unit's rows
    int part_kb;             // blocks of rows summed in one accumulator: kPartStages or kLongPartStages
    uint8_t *out;            // read where the gradient is added to, written where split
    int64_t out_row_bytes;
    int accumulate;
    unsigned *status;
    uint64_t wait_ns;
};

struct Unit {
    int e, row0, cnt;        // expert, first row and number of rows (of this CTA's slice)
    bool idle;               // the expert has no rows
    int nkb;                 // stages: blocks of 64 rows
    int tail;                // rows of the last block that are the expert's
    int n0;                  // this CTA's first row of grad_w
    int k0, mma_n;           // the unit's columns of grad_w, and how wide the MMA is
};

// Walks a CTA's units, first and then every step-th, as (expert, outer tile,
// inner tile) without dividing between units.
template <int CG, bool SPLIT, bool HALF>
struct UnitWalk {
    const Segments &S;
    const WgradParams &p;
    int rank, outer_n, inner_n;          // how many outer and inner tiles
    int e, outer, inner, de, douter, dinner;

    __device__ __forceinline__ void split(int unit, int &x, int &y, int &z) const
    {
        x = unit / (outer_n * inner_n);
        const int rem = unit - x * (outer_n * inner_n);
        y = rem / inner_n;
        z = rem - y * inner_n;
    }
    __device__ __forceinline__ UnitWalk(const Segments &seg, const WgradParams &params, int r, int first, int step)
        : S(seg), p(params), rank(r)
    {
        outer_n = p.n_fast ? p.k_tiles : p.n_tiles;
        inner_n = p.n_fast ? p.n_tiles : p.k_tiles;
        split(first, e, outer, inner);
        split(step, de, douter, dinner);
    }
    // the current unit; moves on to the next
    __device__ __forceinline__ Unit next()
    {
        Unit u;
        const int nt = p.n_fast ? inner : outer, kt = p.n_fast ? outer : inner;
        u.e = e;
        u.row0 = S.first[e];
        u.cnt = S.count[e];
        u.idle = u.cnt == 0;
        if constexpr (SPLIT) {
            const int all = (u.cnt + BK - 1) / BK, slice = (int)cluster_ctarank();
            const int from = (int)((int64_t)all * slice / p.split) * BK;
            const int64_t to = (int64_t)all * (slice + 1) / p.split * BK;
            u.row0 += from;
            u.cnt = (to < u.cnt ? (int)to : u.cnt) - from;
        }
        u.nkb = (u.cnt + BK - 1) / BK;
        u.tail = u.cnt - (u.nkb - 1) * BK;
        u.n0 = (nt * CG + rank) * BM;
        u.k0 = kt * BN<HALF>;
        // whole 64-column boxes for each CTA: an MN-major operand's 128-byte rows
        const int left = p.K - u.k0;
        u.mma_n = left >= BN<HALF> ? BN<HALF> : (left + 64 * CG - 1) / (64 * CG) * (64 * CG);
        e += de;
        outer += douter;
        inner += dinner;
        if (inner >= inner_n) { inner -= inner_n; ++outer; }
        if (outer >= outer_n) { outer -= outer_n; ++e; }
        return u;
    }
};

template <int DT, int CG, bool OUT_F32, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
grouped_wgrad_kernel(const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_out, const WgradParams p)
{
    constexpr bool HALF = OUT_F32 && SPLIT, TOTAL = !HALF;
    constexpr int NS = STAGES<CG, HALF>;
    extern __shared__ uint8_t smem_raw[];
    Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)cluster_ctarank() : 0;
    const bool leader = rank == 0;
    static_assert(!SPLIT || CG == 1, "a split unit runs on single CTAs");
    const int ways = SPLIT ? p.split : CG;           // CTAs per unit
    const int unit0 = (int)blockIdx.x / ways, unit_step = (int)gridDim.x / ways;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
            mbar_init(&S.tail_in[s], 1);
            mbar_init(&S.tail_out[s], CG);
        }
        for (int a = 0; a < 2; ++a) { mbar_init(&S.acc_full[a], 1); mbar_init(&S.acc_empty[a], 4 * CG); }
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
                           [&](int) { return p.n_tiles * p.k_tiles; });
    tc_fence_before();
    // a pair also makes each CTA's barrier initialisation visible to the
    // other before any copy or arrival targets it
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = S.tmem_base;
    const int total = p.E * p.n_tiles * p.k_tiles;
    volatile int *abort_flag = &S.abort;
    UnitWalk<CG, SPLIT, HALF> walk(S.seg, p, rank, unit0, unit_step);

    // A producer's loop: loads(dst, bar, u, row) issues its copies of one
    // stage; with ARM it also expects both producers' bytes.
    auto produce = [&](uint32_t on, auto arm, auto loads) {
        constexpr bool ARM = decltype(arm)::value;
        const uint32_t ring = smem_u32(S.ring);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int unit = unit0; unit < total && ok; unit += unit_step) {
            const Unit u = walk.next();
            const uint32_t bytes = G_BYTES + u.mma_n / CG / 64 * BOX_BYTES;
            for (int kb = 0; kb < u.nkb; ++kb) {
                ok = warp_wait<CG>(&S.empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_ns);
                if (!ok) break;
                // a stage with foreign rows completes in its own CTA, where
                // warp 6 zeroes them; any other on the leader's barrier, which
                // expects both CTAs' bytes (copies may land before it is armed:
                // the phase cannot complete while its arrival is pending)
                const bool tail = kb == u.nkb - 1 && u.tail % UK != 0;
                uint32_t bar;
                if (tail) {
                    const uint32_t here = smem_u32(&S.tail_in[stage]);
                    bar = CG == 2 ? mapa_shared(here, (uint32_t)rank) : here;
                    if (ARM) {
                        expect_tx_on(on, &S.tail_in[stage], bytes);
                        if (leader) arrive_on(on, &S.full[stage]);
                    }
                } else {
                    const uint32_t here = smem_u32(&S.full[stage]);
                    bar = CG == 2 ? mapa_shared(here, 0) : here;
                    if (ARM && leader) expect_tx_on(on, &S.full[stage], CG * bytes);
                }
                loads(ring + stage * SLOT_BYTES<CG, HALF>, bar, u, u.row0 + kb * BK);
                if (++stage == NS) { stage = 0; phase ^= 1u; }
            }
        }
    };
    if (warp == 0) {
        // ------------------------------------------- TMA producer: grad
        const uint32_t on = elect_lane();
        produce(on, std::true_type{}, [&](uint32_t dst, uint32_t bar, const Unit &u, int row) {
            load_2d_on<CG>(on, dst, &map_g, bar, u.n0, row);
            load_2d_on<CG>(on, dst + BOX_BYTES, &map_g, bar, u.n0 + 64, row);
        });
    } else if (warp == 7) {
        // ------------------------------------------- TMA producer: a
        const uint32_t on = elect_lane();
        produce(on, std::false_type{}, [&](uint32_t dst, uint32_t bar, const Unit &u, int row) {
            const int mine = u.mma_n / CG, col0 = u.k0 + rank * mine;     // columns this CTA loads
#pragma unroll
            for (int j = 0; j < BN<HALF> / 64 / CG; ++j)
                load_2d_on<CG>(j * 64 < mine ? on : 0u, dst + G_BYTES + j * BOX_BYTES, &map_a, bar, col0 + j * 64, row);
        });
    } else if (warp == 1 && leader) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc0 = idesc_f16_major<DT>(BM * CG, 0, true, true);
        const uint32_t on = elect_lane();
        const uint32_t ring = smem_u32(S.ring);
        int stage = 0;
        uint32_t phase = 0, tails = 0;
        int acc = 0;
        uint32_t used = 0;                         // parity of each accumulator's uses so far
        bool ok = true;
        for (int unit = unit0; unit < total && ok; unit += unit_step) {
            const Unit u = walk.next();
            const uint32_t idesc = idesc0 | ((uint32_t)(u.mma_n >> 3) << 17);
            // (an expert without rows commits one part with no MMA: its epilogue writes zeros)
            int kb0 = 0;
            do {
                const int kb1 = u.nkb - kb0 < p.part_kb ? u.nkb : kb0 + p.part_kb;
                ok = warp_wait<CG>(&S.acc_empty[acc], (used >> acc & 1u) ^ 1u, abort_flag, p.status, p.wait_ns);
                if (!ok) break;
                used ^= 1u << acc;
                const uint32_t d = tmem_base + (uint32_t)(acc * ACC_COLS);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = warp_wait<CG>(&S.full[stage], phase, abort_flag, p.status, p.wait_ns);
                    if (!ok) break;
                    const int valid = kb == u.nkb - 1 ? u.tail : BK;
                    if (valid % UK != 0) {
                        ok = warp_wait<CG>(&S.tail_out[stage], tails >> stage & 1u, abort_flag, p.status, p.wait_ns);
                        if (!ok) break;
                        tails ^= 1u << stage;
                    }
                    tc_fence_after();
                    const uint32_t g = ring + stage * SLOT_BYTES<CG, HALF>, a = g + G_BYTES;
                    auto mma = [&](int k) {
                        umma_on<CG>(on, d, sdesc_mn_sw128(g + k * UK * 128, BOX_BYTES),
                                    sdesc_mn_sw128(a + k * UK * 128, BOX_BYTES), idesc, (kb - kb0) | k ? 1u : 0u);
                    };
                    if (valid == BK) {
#pragma unroll
                        for (int k = 0; k < BK / UK; ++k) mma(k);
                    } else {
                        for (int k = 0; k * UK < valid; ++k) mma(k);
                    }
                    commit_on<CG>(on, &S.empty[stage]);
                    if (++stage == NS) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                commit_on<CG>(on, &S.acc_full[acc]);
                acc = next_acc<TOTAL>(acc, kb0 != 0, kb1 == u.nkb);
                kb0 = kb1;
            } while (kb0 < u.nkb);
        }
        // every MMA issued must finish before TMEM is released, also where
        // another role has given up
        if (on) {
            umma_commit<CG>(&S.drain);
            mbar_wait(&S.drain, 0, nullptr, p.status, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------ foreign rows
        int stage = 0;
        uint32_t tails = 0;
        for (int unit = unit0; unit < total; unit += unit_step) {
            const Unit u = walk.next();
            if (u.nkb == 0) continue;
            stage = (stage + u.nkb - 1) % NS;                 // the unit's last stage
            if (u.tail % UK != 0) {
                const bool ready = mbar_wait<CG>(&S.tail_in[stage], tails >> stage & 1u, abort_flag, p.status, p.wait_ns);
                if (!__all_sync(0xffffffffu, ready)) break;
                tails ^= 1u << stage;
                // whole 128-byte rows of every box: the swizzle stays inside a row
                const int nrows = UK - u.tail % UK;
                const int boxes = 2 + u.mma_n / CG / 64;
                for (int i = lane; i < boxes * nrows * 8; i += 32) {
                    const int box = i / (nrows * 8), c = i - box * (nrows * 8);
                    *reinterpret_cast<uint4 *>(S.ring + stage * SLOT_BYTES<CG, HALF> + box * BOX_BYTES + u.tail * 128 + c * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                // the MMA reads shared memory through the async proxy
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2 && !leader) mbar_arrive_cluster(mapa_shared(smem_u32(&S.tail_out[stage]), 0));
                    else mbar_arrive(&S.tail_out[stage]);
                }
            }
            if (++stage == NS) stage = 0;
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3;                    // TMEM lane quadrant of this warp
        constexpr int ESZ = OUT_F32 ? 4 : 2;
        constexpr int COLS = STG_ROW_BYTES / ESZ;  // columns per staging buffer: 16 / 32
        const uint32_t on = elect_lane();
        int next = 0, buf = 0, unit = unit0, kb0 = 0;
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
        // unit by unit, part by part (kb0: the part's first block of rows)
        for (; unit < total; kb0 += p.part_kb) {
            if (kb0 != 0 && kb0 >= u.nkb) {
                kb0 = 0;
                unit += unit_step;
                if (unit >= total) break;
            }
            if (kb0 == 0) u = walk.next();
            const bool more = kb0 != 0, last = u.nkb - kb0 <= p.part_kb;      // adds to the earlier parts; ends the sum
            const int acc = next;
            const uint32_t acc_phase = used >> acc & 1u;
            used ^= 1u << acc;
            next = next_acc<TOTAL>(acc, more, last);
            const bool ready = mbar_wait<CG>(&S.acc_full[acc], acc_phase, abort_flag, p.status, p.wait_ns);
            if (!__all_sync(0xffffffffu, ready)) break;
            tc_fence_after();
            const int row0 = u.n0 + q * 32;            // this warp's first row of grad_w[e]
            const bool empty = u.cnt == 0;
            int width = p.K - u.k0 < BN<HALF> ? p.K - u.k0 : BN<HALF>;
            auto tmem_of = [&](int a) { return tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * ACC_COLS); };
            int held = acc;                            // the accumulator that holds the sum
            if constexpr (TOTAL) {
                // a later part is added to the first one, which stays where it is
                if (more) {
                    held = acc ^ 1;
                    for (int c0 = 0; c0 < width; c0 += 32) {
                        uint32_t v[32], sum[32];
                        tmem_ld32(tmem_of(acc) + c0, v);
                        tmem_ld32(tmem_of(held) + c0, sum);
                        tmem_ld_wait(v);
                        tmem_ld_wait(sum);
                        add_to(sum, v);
                        tmem_st32(tmem_of(held) + c0, sum);
                    }
                    tmem_st_wait();
                    release(acc);
                }
                if (!last) continue;
            }
            const uint32_t tbase = tmem_of(held);
            if constexpr (SPLIT) {
                // the partial sums stay here, [column][row] in FP32 (16-bit
                // gradients: over the ring, whose last MMA is done)
                float *mine = reinterpret_cast<float *>(S.ring + PARTIAL_AT<HALF>) + q * 32 + lane;
                for (int c0 = 0; c0 < width; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld32(tbase + c0, v);
                    tmem_ld_wait(v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float x = empty ? 0.0f : __uint_as_float(v[i]);
                        mine[(c0 + i) * BM] = HALF && more ? mine[(c0 + i) * BM] + x : x;
                    }
                }
                width = 0;
            }
            if (row0 >= p.N || (empty && p.accumulate)) width = 0;
            // stores 32 columns from c0 on, accumulating what grad_w holds
            auto emit = [&](uint32_t (&v)[32], int c0) {
                if (p.accumulate && row0 + lane < p.N) {
                    const int64_t col_byte = (int64_t)(u.k0 + c0) * ESZ;
                    const uint8_t *old = p.out + ((int64_t)u.e * p.N + row0 + lane) * p.out_row_bytes + col_byte;
#pragma unroll
                    for (int c = 0; c < 32 * ESZ / 16; ++c) {
                        if (col_byte + c * 16 >= p.out_row_bytes) continue;
                        Vec16 o;
                        // past L1: read once
                        asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(o.w[0]), "=r"(o.w[1]), "=r"(o.w[2]), "=r"(o.w[3])
                                     : "l"(old + c * 16)
                                     : "memory");
                        if constexpr (OUT_F32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[c * 4 + i] = __float_as_uint(__uint_as_float(v[c * 4 + i]) + o.f[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 f = DT == DT_BF16 ? bf16x2_to_float2(o.w[i]) : f16x2_to_float2(o.w[i]);
                                v[c * 8 + 2 * i] = __float_as_uint(__uint_as_float(v[c * 8 + 2 * i]) + f.x);
                                v[c * 8 + 2 * i + 1] = __float_as_uint(__uint_as_float(v[c * 8 + 2 * i + 1]) + f.y);
                            }
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 32 / COLS; ++h, buf ^= 1) {
                    uint8_t *stg = S.stg[warp - 2][buf];
                    // the store before last has read this buffer
                    if (on) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    __syncwarp();
                    // this lane's 64 bytes, in the 64-byte swizzle: 16-byte
                    // piece c of row r at c ^ (r / 2 % 4), free of bank conflicts
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = OUT_F32 ? v[(h * COLS + c * 4 + i) % 32]
                                           : pack2<DT>(__uint_as_float(v[(c * 8 + 2 * i) % 32]),
                                                       __uint_as_float(v[(c * 8 + 2 * i + 1) % 32]));
                        *reinterpret_cast<uint4 *>(stg + lane * STG_ROW_BYTES + ((c ^ (lane >> 1 & 3)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (on) {
                        if (c0 + h * COLS < width)
                            asm volatile(
                                "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group"
                                " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(&map_out)),
                                "r"(smem_u32(stg)), "r"(u.k0 + c0 + h * COLS), "r"(row0), "r"(u.e)
                                : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            };
            for (int c0 = 0; c0 < width; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tbase + c0, v);
                tmem_ld_wait(v);
                if (empty) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                }
                emit(v, c0);
            }
            release(held);
        }
        // the stores have read their buffers and written what they carried
        if (on) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    if constexpr (SPLIT) {
        // every CTA's partial sums are written; each adds its columns, eight
        // of a row at a time
        __syncwarp();
        cluster_sync();
        if (unit0 < total) {
            const int slice = (int)cluster_ctarank();
            const Unit u = UnitWalk<CG, SPLIT, HALF>(S.seg, p, rank, unit0, unit_step).next();
            const int width = p.K - u.k0 < BN<HALF> ? p.K - u.k0 : BN<HALF>;
            const uint32_t partial = smem_u32(S.ring + PARTIAL_AT<HALF>);
            for (int i = threadIdx.x; !(u.idle && p.accumulate); i += THREADS) {
                const int c = (i / BM * ways + slice) * 8, n = i % BM;
                if (c >= width) break;
                if (u.n0 + n >= p.N) continue;
                float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                for (int r = 0; r < ways; ++r) {
                    const uint32_t from = mapa_shared(partial + (c * BM + n) * 4, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + j * BM * 4) : "memory");
                        sum[j] += v;
                    }
                }
                uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((int64_t)u.e * p.N + u.n0 + n) * p.out_row_bytes +
                                                       (int64_t)(u.k0 + c) * (OUT_F32 ? 4 : 2));
#pragma unroll
                for (int h = 0; h < (OUT_F32 ? 2 : 1); ++h) {
                    Vec16 o;
                    o.u = p.accumulate ? dst[h] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (OUT_F32) {
                            o.f[j] = p.accumulate ? sum[h * 4 + j] + o.f[j] : sum[h * 4 + j];
                        } else {
                            float2 f = make_float2(sum[2 * j], sum[2 * j + 1]);
                            if (p.accumulate) {
                                const float2 old = DT == DT_BF16 ? bf16x2_to_float2(o.w[j]) : f16x2_to_float2(o.w[j]);
                                f.x += old.x;
                                f.y += old.y;
                            }
                            o.w[j] = pack2<DT>(f.x, f.y);
                        }
                    }
                    dst[h] = o.u;
                }
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

// grad_w [E, N, K] in boxes of 64 bytes x 32 rows, 64-byte swizzle.
bool encode_out(CUtensorMap *m, CUtensorMapDataType dt, void *base, uint64_t K, uint64_t N, uint64_t E,
                uint32_t esz)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {K, N, E};
    cuuint64_t strides[2] = {K * esz, K * N * esz};
    cuuint32_t box[3] = {STG_ROW_BYTES / esz, 32, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, dt, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, int CG, bool OUT_F32, bool SPLIT>
cudaError_t launch_kernel(const CUtensorMap &mg, const CUtensorMap &ma, const CUtensorMap &mo, WgradParams p,
                          cudaStream_t s)
{
    // CTAs the GPU holds at once, per device; 0: the kernel is not yet opted
    // in to its shared memory there
    static std::atomic<int> cache[kCachedDevices];
    auto kernel = grouped_wgrad_kernel<DT, CG, OUT_F32, SPLIT>;
    const int ways = SPLIT ? p.split : CG;
    p.n_tiles = (p.N + BM * CG - 1) / (BM * CG);
    constexpr int COLS = BN<(OUT_F32 && SPLIT)>;
    p.k_tiles = (p.K + COLS - 1) / COLS;
    p.n_fast = p.N <= p.K;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ways;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kCachedDevices;
    int ctas = cached ? cache[dev].load() : 0;
    if (ctas == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (err != cudaSuccess) return err;
        ctas = device_sm_count();
        if (CG == 2) {
            int pairs = 0;
            cfg.gridDim = dim3((unsigned)(ctas & ~1));
            cfg.numAttrs = 1;
            err = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
            if (err != cudaSuccess) return err;
            if (pairs < 1) return cudaErrorInvalidConfiguration;
            ctas = 2 * pairs;
        }
        if (cached) cache[dev].store(ctas);
    }
    const int64_t units = (int64_t)p.E * p.n_tiles * p.k_tiles;
    cfg.gridDim = dim3((unsigned)(SPLIT || ways * units < ctas ? ways * units : ctas));
    cfg.numAttrs = 2;
    // The warp that zeroes foreign rows passes over units without any, and the
    // producers over experts without rows, so their waits may last most of what a
    // CTA does: per expert, its share of the expert's tiles.
    const uint64_t groups = cfg.gridDim.x / (unsigned)ways;
    const uint64_t tiles = ((uint64_t)p.n_tiles * p.k_tiles + groups - 1) / groups;
    p.wait_ns = wait_limit_ns() + work_ns(tiles * (uint64_t)(p.rows / BK + p.E), tiles * (uint64_t)p.E);
    return cudaLaunchKernelEx(&cfg, kernel, mg, ma, mo, p);
}

template <int DT>
cudaError_t launch_dt(const void *grad, int64_t ldg, const void *a, int64_t lda, const int32_t *offsets,
                      int64_t rows, int E, int64_t N, int64_t K, void *grad_w, bool out_f32,
                      bool accumulate, unsigned *status, cudaStream_t s)
{
    const CUtensorMapDataType tdt =
        DT == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap mg, ma, mo;
    if (!encode_2d_strided(&mg, tdt, grad, (uint64_t)N, (uint64_t)rows, (uint64_t)ldg * 2, 64, BK) ||
        !encode_2d_strided(&ma, tdt, a, (uint64_t)K, (uint64_t)rows, (uint64_t)lda * 2, 64, BK) ||
        !encode_out(&mo, out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : tdt, grad_w, (uint64_t)K, (uint64_t)N,
                    (uint64_t)E, out_f32 ? 4 : 2))
        return cudaErrorInvalidValue;
    WgradParams p{};
    p.offsets = offsets;
    p.E = E;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.out = static_cast<uint8_t *>(grad_w);
    p.out_row_bytes = K * (out_f32 ? 4 : 2);
    p.accumulate = accumulate;
    p.status = status;
    p.part_kb = out_f32 ? kPartStages : kLongPartStages<DT>;
    // Few units: split an expert's rows over as many CTAs, 2 to 8, as the GPU has
    // room for and as leave each four blocks of rows on average.
    const int cols = out_f32 ? BN<true> : BN<false>;
    const int64_t units = (int64_t)E * ((N + BM - 1) / BM) * ((K + cols - 1) / cols);
    const int64_t blocks = rows / E / BK, sms = device_sm_count();
    p.split = 1;
    while (p.split < 8 && units * p.split * 2 <= sms && blocks >= p.split * 2 * 4) p.split *= 2;
    if (p.split > 1)
        return out_f32 ? launch_kernel<DT, 1, true, true>(mg, ma, mo, p, s)
                       : launch_kernel<DT, 1, false, true>(mg, ma, mo, p, s);
    // Pairs or single CTAs, by the average rows of an expert: us at 256, 384, 512,
    // 768, 1024, 4096 rows, 64 experts of 2048 x 1408 (16 of 4096 x 4096):
    // 16 bits, singles 111 125 152 214 278 1028 (143 178 221 301 386 1303),
    //          pairs   128 140 153 192 239 937 (166 192 208 260 315 1230);
    // FP32,    singles 155 173 195 245 354 1172 (200 230 275 357 483 1552),
    //          pairs   171 188 200 229 386 1160 (225 250 279 320 491 1538).
    if (rows >= 512 * (int64_t)E)
        return out_f32 ? launch_kernel<DT, 2, true, false>(mg, ma, mo, p, s)
                       : launch_kernel<DT, 2, false, false>(mg, ma, mo, p, s);
    return out_f32 ? launch_kernel<DT, 1, true, false>(mg, ma, mo, p, s)
                   : launch_kernel<DT, 1, false, false>(mg, ma, mo, p, s);
}

}  // namespace

cudaError_t launch_grouped_weight_grad_tc(int dt, const void *grad, int64_t ldg, const void *a,
                                          int64_t lda, const int32_t *offsets, int64_t rows, int E,
                                          int64_t N, int64_t K, void *grad_w, bool out_f32,
                                          bool accumulate, unsigned *status, cudaStream_t s)
{
    if (dt == DT_BF16)
        return launch_dt<DT_BF16>(grad, ldg, a, lda, offsets, rows, E, N, K, grad_w, out_f32, accumulate, status, s);
    return launch_dt<DT_F16>(grad, ldg, a, lda, offsets, rows, E, N, K, grad_w, out_f32, accumulate, status, s);
}

}  // namespace moe
