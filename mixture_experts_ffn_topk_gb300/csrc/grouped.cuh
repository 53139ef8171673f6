// grouped.cuh -- what the grouped-product kernels share: a CTA's table of the
// experts' row segments, built from the device-side offsets with no host
// synchronisation.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int kGroupedMaxE = 1024;

// The tensor cores add into their FP32 accumulator by truncation, so a long
// reduction drifts towards zero: relative errors measured against 64 bits were
// 3.5e-7 over 384 terms, 1.0e-6 over 1048, 3.2e-6 over 3000 and 7.8e-6 over
// 7032, where FP32 sums in torch stay at 1e-7 to 8e-7. FP32 outputs are
// therefore summed in parts of this many stages of 64, each in an accumulator
// of its own, added up by ordinary FP32 additions. 16-bit outputs, whose
// rounding is 2^-9 or 2^-12 of a value, take one accumulator.
constexpr int kPartStages = 12;

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
