// grouped_units.cuh -- the work units of the grouped products, which compute
// out^T = w a^T: an expert's rows are cut into units of equal width, at most
// tok_cap; units run over (expert, block of row units, weight tile, row unit),
// the row unit fastest.
#pragma once

#include <atomic>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int BM = 128;                  // weight columns per CTA

// Bytes of rows a block of row units may cover, well inside the 129 MB L2
// that also carries the streamed weights and the output.
constexpr int64_t kRowBlockBytes = 48ll << 20;

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
// Params: E, tok_cap, row_block and w_tiles.
template <int CG, typename Params>
struct UnitWalk {
    const Segments &S;
    const Params &p;
    int rank, e, cnt, n_units, each;

    __device__ __forceinline__ UnitWalk(const Segments &seg, const Params &params, int r)
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

// ---- host side ---------------------------------------------------------------

// Opts this kernel instance in to its shared memory, and (pairs) asks how many
// clusters the GPU holds at once, once per device.
template <typename Kernel>
cudaError_t prepare_kernel(Kernel kernel, int cg, int threads, size_t smem, std::atomic<int> *cache, int *ctas)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool cached = dev >= 0 && dev < kCachedDevices;
    int n = cached ? cache[dev].load() : 0;
    if (n == 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
        n = device_sm_count();
        if (cg == 2) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(n & ~1));
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
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

}  // namespace
}  // namespace moe
