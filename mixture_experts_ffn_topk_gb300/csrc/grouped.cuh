// grouped.cuh -- what the grouped-product kernels share: a CTA's table of the
// experts' row segments, built from the device-side offsets with no host
// synchronisation.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int kGroupedMaxE = 1024;

// The tensor cores add into their FP32 accumulator by truncation, so a long
// reduction drifts towards zero. Normal operands of either sign: relative errors
// against 64 bits of 3.5e-7 over 384 terms, 1.0e-6 over 1048, 3.2e-6 over 3000 and
// 7.8e-6 over 7032, where FP32 sums in torch stay at 1e-7 to 8e-7. Positive terms,
// the worst: 6.4e-9 of the sum per term, 3.3e-3 over 2^19. Sums are therefore formed in parts of so many stages of 64, each in
// an accumulator of its own, added up by ordinary FP32 additions: FP32 outputs in
// parts of 768 terms (positive ones 4.3e-6 low); 16-bit ones, rounded by half a
// step (2^-12 to 2^-11 of an F16 value, 2^-9 to 2^-8 of a BF16 one), in parts of
// 16384 and 32768, over which positive terms drift by 2^-13.2 and 2^-12.2. Parts of
// 4096 cost F16 5 to 7 % over K = 7168 and 14336 (8 experts of 4096 rows, N = 4096:
// 2.30 against 2.18 ms), where these are one part.
constexpr int kPartStages = 12;
template <int DT>
constexpr int kLongPartStages = DT == DT_F16 ? 256 : 512;

// What a wait may last for the launch's own work, on top of the wait limit: a
// microsecond per stage and 20 per stored tile it may have to wait for, three
// times what either takes on all SMs at once.
inline uint64_t work_ns(uint64_t stages, uint64_t tiles) { return 1000ull * stages + 20000ull * tiles; }

// sum[i] += v[i] of FP32 values held as their bits.
template <int N>
__device__ __forceinline__ void add_to(uint32_t (&sum)[N], const uint32_t (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = __float_as_uint(__uint_as_float(sum[i]) + __uint_as_float(v[i]));
}

// Accumulators take turns; where a sum's total stays in its first part's
// accumulator (TOTAL), the later parts of that sum all have the other one.
// more: the part adds to earlier ones; last: no other part follows.
template <bool TOTAL>
__device__ __forceinline__ int next_acc(int acc, bool more, bool last)
{
    return TOTAL && more && !last ? acc : acc ^ 1;
}

// Expert e has rows [first[e], first[e] + count[e]) and the work units
// [unit[e], unit[e + 1]).
struct Segments {
    int first[kGroupedMaxE];
    int count[kGroupedMaxE];
    int unit[kGroupedMaxE + 1];
};

// Fills the table: the first THREADS threads of the CTA take part, all of
// them call; a __syncthreads() by the caller publishes it. units_of(rows)
// gives an expert's number of units. An expert whose offsets fall, are
// negative or pass `rows`, or whose rows an earlier one has, gets no rows, and
// the status word records ST_BAD_INDEX: whatever the offsets hold, every row
// that a unit names lies in [0, rows), and no row belongs to two experts.
template <int THREADS, typename UnitsOf>
__device__ __forceinline__ void load_segments(Segments &S, int *warp_sum,
                                              const int32_t *__restrict__ offsets, int E,
                                              int rows, unsigned *status, UnitsOf units_of)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    for (int e = threadIdx.x; e < E; e += THREADS) {
        const int a = offsets[e], b = offsets[e + 1];
        const bool ok = a >= 0 && b >= a && b <= rows;
        bad |= !ok;
        S.first[e] = ok ? a : 0;
        S.count[e] = ok ? b - a : 0;
    }
    if (__syncthreads_or(bad)) {
        // offsets that fall somewhere may also name rows twice: the later
        // expert yields, so that there are never more units than the launch
        // was sized for and no two experts write one row
        if (threadIdx.x == 0) {
            if (blockIdx.x == 0) atomicOr(status, ST_BAD_INDEX);
            int end = 0;
            for (int e = 0; e < E; ++e) {
                if (S.first[e] < end) S.count[e] = 0;
                if (S.count[e] > 0) end = S.first[e] + S.count[e];
            }
        }
        __syncthreads();
    }
    // exclusive prefix over the experts' units: a run of experts per thread,
    // then the warps' totals
    const int per = (E + THREADS - 1) / THREADS, e0 = threadIdx.x * per;
    int local = 0;
    for (int e = e0; e < e0 + per && e < E; ++e) local += units_of(S.count[e]);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int run = incl - local;
    for (int i = 0; i < warp; ++i) run += warp_sum[i];
    for (int e = e0; e < e0 + per && e < E; ++e) {
        S.unit[e] = run;
        run += units_of(S.count[e]);
    }
    if (threadIdx.x == THREADS - 1) S.unit[E] = run;
}

// The expert whose units hold `unit` (an expert without units is passed over).
__device__ __forceinline__ int expert_of(const Segments &S, int E, int unit)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (S.unit[mid] <= unit) lo = mid; else hi = mid - 1;
    }
    return lo;
}

}  // namespace
}  // namespace moe
