// grouped_simt.cu -- grouped products of FP32 rows on CUDA cores (true FP32:
// tensor cores would round the operands to TF32).
//
// For the rows r of expert e (offsets[e] <= r < offsets[e + 1]):
//   product       out[r, n] = sum_k a[r, k] w[e][n, k]   (or w[e][k, n])
//   weight grad   grad_w[e][n, k] = sum_r grad[r, n] a[r, k]
// One tiled kernel: C [M, N] = sum_k X(m, k) Y(n, k), where each operand is
// stored either with k contiguous (X[m][k]) or with m contiguous (X[k][m]), and
// is kept so in shared memory: a ring of steps filled by 16-byte asynchronous
// copies, several steps ahead, zero-filled at the edges. A thread computes
// TM x TN outputs, four k at a time. Its rows and columns lie one thread apart
// where k is contiguous (padded rows: no bank conflicts), in fours otherwise.
// Bound: FP32 multiply-adds with many rows per expert, the weights' bytes with
// few, so the tile's height follows the average number of rows.
#include <atomic>

#include "common.cuh"
#include "grouped.cuh"
#include "kernels.h"

namespace moe {

namespace {

struct SimtOperand {
    const float *p;         // element (0, 0) of the whole operand
    int64_t ld;             // elements between rows
    int64_t per_expert;     // elements between experts' matrices (0: rows of a dispatched matrix)
};

// 16 bytes, or zeros where !ok (then src is any readable address).
__device__ __forceinline__ void copy16(float *dst, const float *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}

template <int B, int BK, bool MAJOR>
constexpr int kTileFloats = MAJOR ? BK * (B + 4) : B * (BK + 4);

// Tile of an operand: `extent` of B indices from i0, k from k0 to k_end.
template <int B, int BK, bool MAJOR, int THREADS>
__device__ __forceinline__ void fetch_tile(float *dst, const float *p, int64_t ld, int i0, int i_end,
                                           int k0, int k_end)
{
    constexpr int VECS = B * BK / 4;
#pragma unroll
    for (int q = 0; q < (VECS + THREADS - 1) / THREADS; ++q) {
        const int v = threadIdx.x + q * THREADS;
        if (VECS % THREADS != 0 && v >= VECS) break;
        const int i = MAJOR ? v % (B / 4) * 4 : v / (BK / 4);
        const int k = MAJOR ? v / (B / 4) : v % (BK / 4) * 4;
        const bool ok = i0 + i < i_end && k0 + k < k_end;
        const int64_t at = MAJOR ? (int64_t)(k0 + k) * ld + i0 + i : (int64_t)(i0 + i) * ld + k0 + k;
        copy16(dst + (MAJOR ? k * (B + 4) + i : i * (BK + 4) + k), ok ? p + at : p, ok);
    }
}

// Index of a thread's j-th row or column: T of them, `groups` threads side by side.
template <int T, int GROUPS, bool MAJOR>
__device__ __forceinline__ int index_of(int j, int t)
{
    return MAJOR ? j / 4 * (GROUPS * 4) + t * 4 + j % 4 : j * GROUPS + t;
}

// A thread's values of an operand at k, ..., k + 3.
template <int B, int BK, int T, int GROUPS, bool MAJOR>
__device__ __forceinline__ void frag(const float *tile, int k, int t, float (&f)[T][4])
{
    if constexpr (MAJOR) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < T; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    tile + (k + kk) * (B + 4) + index_of<T, GROUPS, true>(j, t));
                f[j][kk] = v.x; f[j + 1][kk] = v.y; f[j + 2][kk] = v.z; f[j + 3][kk] = v.w;
            }
    } else {
#pragma unroll
        for (int j = 0; j < T; ++j)
            *reinterpret_cast<float4 *>(f[j]) = *reinterpret_cast<const float4 *>(
                tile + index_of<T, GROUPS, false>(j, t) * (BK + 4) + k);
    }
}

// Two FP32 multiply-adds in one instruction: each half of d += that of a * b.
__device__ __forceinline__ void fma2(float2 &d, float2 a, float2 b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<unsigned long long &>(d))
        : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)));
}

// WG: the reduction runs over the expert's rows (X = grad, Y = a, both stored
// with the output index contiguous). Otherwise X = a (k contiguous), Y = w,
// k contiguous unless Y_MAJOR.
template <bool WG, bool Y_MAJOR, int BM, int BN, int TM, int TN, int BK, int STAGES>
struct SimtShape {
    static constexpr int THREADS = BM / TM * (BN / TN);
    static constexpr int X_FLOATS = kTileFloats<BM, BK, WG>, Y_FLOATS = kTileFloats<BN, BK, Y_MAJOR>;
    static constexpr size_t SMEM = sizeof(float) * STAGES * (X_FLOATS + Y_FLOATS);
};

template <bool WG, bool Y_MAJOR, int BM, int BN, int TM, int TN, int BK, int STAGES>
__global__ void __launch_bounds__(BM / TM * (BN / TN), 2)
grouped_simt_kernel(SimtOperand x, SimtOperand y, const int32_t *__restrict__ offsets, int E,
                    int rows, int M, int N, int K, float *__restrict__ out, int64_t ldo,
                    int accumulate, unsigned *status)
{
    using Shape = SimtShape<WG, Y_MAJOR, BM, BN, TM, TN, BK, STAGES>;
    constexpr int THREADS = Shape::THREADS, GM = BM / TM, GN = BN / TN;
    __shared__ Segments S;
    __shared__ int warp_sum[THREADS / 32];
    extern __shared__ __align__(16) float ring[];
    float *xs = ring, *ys = ring + STAGES * Shape::X_FLOATS;
    pdl_wait();
    pdl_launch_dependents();
    const int nt = (N + BN - 1) / BN;
    load_segments<THREADS>(S, warp_sum, offsets, E, rows, status, [&](int cnt) {
        return WG ? (M + BM - 1) / BM * nt : (cnt + BM - 1) / BM * nt;
    });
    __syncthreads();
    const int total = S.unit[E];
    const int tm = threadIdx.x / GN, tn = threadIdx.x % GN;
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
        const int e = expert_of(S, E, unit), loc = unit - S.unit[e];
        const int first = S.first[e], cnt = S.count[e];
        const int m0 = loc / nt * BM, n0 = loc % nt * BN;
        const int m_end = WG ? M : cnt, k_end = WG ? cnt : K;
        // element (0, 0) of this unit's operands
        const float *xp = x.p + (int64_t)first * x.ld;
        const float *yp = y.p + (WG ? (int64_t)first * y.ld : (int64_t)e * y.per_expert);
        const int steps = (k_end + BK - 1) / BK;
        auto fetch = [&](int t) {
            if (t < steps) {
                fetch_tile<BM, BK, WG, THREADS>(xs + t % STAGES * Shape::X_FLOATS, xp, x.ld, m0, m_end, t * BK, k_end);
                fetch_tile<BN, BK, Y_MAJOR, THREADS>(ys + t % STAGES * Shape::Y_FLOATS, yp, y.ld, n0, N, t * BK, k_end);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // where a thread's columns are neighbours, two of them share an
        // instruction (6 % faster there; sums over even and odd k of one
        // output, the pairing that k-contiguous operands offer, cost registers
        // and were 11 % slower than single multiply-adds)
        constexpr bool PAIRED = WG || Y_MAJOR;
        float2 acc[TM][TN / 2];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) acc[i][j] = make_float2(0.0f, 0.0f);
        for (int t = 0; t < STAGES - 1; ++t) fetch(t);
        for (int t = 0; t < steps; ++t) {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncthreads();            // step t is here, and all are done with step t - 1
            fetch(t + STAGES - 1);
            const float *xt = xs + t % STAGES * Shape::X_FLOATS, *yt = ys + t % STAGES * Shape::Y_FLOATS;
#pragma unroll
            for (int k = 0; k < BK; k += 4) {
                float a[TM][4], b[TN][4];
                frag<BM, BK, TM, GM, WG>(xt, k, tm, a);
                frag<BN, BK, TN, GN, Y_MAJOR>(yt, k, tn, b);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN / 2; ++j) {
                            const float2 y2 = make_float2(b[2 * j][kk], b[2 * j + 1][kk]);
                            if constexpr (PAIRED) {
                                fma2(acc[i][j], make_float2(a[i][kk], a[i][kk]), y2);
                            } else {
                                acc[i][j].x = fmaf(a[i][kk], y2.x, acc[i][j].x);
                                acc[i][j].y = fmaf(a[i][kk], y2.y, acc[i][j].y);
                            }
                        }
            }
        }
        __syncthreads();                // the ring is free for the next unit
        const int64_t out0 = WG ? (int64_t)e * M * ldo : (int64_t)first * ldo;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = m0 + index_of<TM, GM, WG>(i, tm);
            if (m >= m_end) continue;
            float *row = out + out0 + (int64_t)m * ldo;
            if constexpr (WG) {
                // rows of grad_w are whole vectors
#pragma unroll
                for (int j = 0; j < TN; j += 4) {
                    const int n = n0 + index_of<TN, GN, true>(j, tn);
                    if (n >= N) continue;
                    float4 v = make_float4(acc[i][j / 2].x, acc[i][j / 2].y, acc[i][j / 2 + 1].x, acc[i][j / 2 + 1].y);
                    if (accumulate) {
                        const float4 old = *reinterpret_cast<const float4 *>(row + n);
                        v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
                    }
                    *reinterpret_cast<float4 *>(row + n) = v;
                }
            } else {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int n = n0 + index_of<TN, GN, Y_MAJOR>(j, tn);
                    if (n < N) row[n] = j & 1 ? acc[i][j / 2].y : acc[i][j / 2].x;
                }
            }
        }
    }
}

template <bool WG, bool Y_MAJOR, int BM, int BN, int TM, int TN, int BK, int STAGES>
cudaError_t launch_tile(const SimtOperand &x, const SimtOperand &y, const int32_t *offsets, int E,
                        int64_t rows, int M, int N, int K, float *out, int64_t ldo,
                        int accumulate, unsigned *status, cudaStream_t s)
{
    using Shape = SimtShape<WG, Y_MAJOR, BM, BN, TM, TN, BK, STAGES>;
    auto kernel = grouped_simt_kernel<WG, Y_MAJOR, BM, BN, TM, TN, BK, STAGES>;
    static std::atomic<uint64_t> opted{0};          // devices whose shared-memory limit is raised
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev >= 0 && dev < kCachedDevices ? 1ull << dev : 0ull;
    if (bit == 0 || !(opted.load() & bit)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::SMEM);
        if (err != cudaSuccess) return err;
        opted.fetch_or(bit);
    }
    const int64_t nt = (N + BN - 1) / BN;
    const int64_t mt = WG ? (int64_t)E * ((M + BM - 1) / BM) : rows / BM + (rows < E ? rows : E);
    const int64_t units = mt * nt, most = (int64_t)device_sm_count() * 8;
    return launch_pdl(kernel, dim3((unsigned)(units < most ? units : most)), dim3(Shape::THREADS),
                      Shape::SMEM, s, x, y, offsets, E, (int)rows, M, N, K, out, ldo, accumulate, status);
}

// Tile by the extent of C's rows: the average number of an expert's rows, or
// grad_w's N. Measured on 64 experts, N = K = 1024 (us at 8, 32, 48, 96, 256,
// 1024 rows on average; 2.98 ms are 46 TFLOP/s, [E, K, N] weights take 2.80):
//   16 x 128   76.2   181   248   450   1133   4396
//   64 x 128   -      -     216   387    854   2975
//   64 x 64    227   225    214   414    903   3243
// (128 x 64 and 128 x 128: 381 to 412 at 96 rows, 2952 to 3156 at 1024). Weight
// gradient, N = 16, 32, 64: 17.7 22.2 33.1 us flat, 22.8 22.8 23.7 square.
// Fewer 64-row tiles than SMs also take the flat one, which gives four times as
// many: us flat and tall, 8 experts of 100 rows, N = 512, K = 2048: 73 and 127
// ([E, K, N] weights 72 and 112); of 64 rows, N = 256: 47 and 126; gradients of
// 128 x 256 over 1000 rows 22 and 54, of 512 x 128 over 200 rows 10 and 14. Just
// below the SMs' number it loses: 3 experts of 579 rows, N = 520, K = 1024, 150
// tiles: 76 and 65.
constexpr int64_t kFlatTile = 40;

template <bool WG, bool Y_MAJOR>
cudaError_t launch_sizes(const SimtOperand &x, const SimtOperand &y, const int32_t *offsets, int E,
                         int64_t rows, int M, int N, int K, float *out, int64_t ldo,
                         int accumulate, unsigned *status, cudaStream_t s)
{
    const int64_t height = WG ? M : rows / E;
    const int64_t tiles = (WG ? (int64_t)E * ((M + 63) / 64) : rows / 64 + (rows < E ? rows : E)) * ((N + 127) / 128);
    if (height < kFlatTile || tiles < device_sm_count())
        return launch_tile<WG, Y_MAJOR, 16, 128, 4, 4, 32, 4>(x, y, offsets, E, rows, M, N, K, out, ldo,
                                                              accumulate, status, s);
    if (N > 64)
        return launch_tile<WG, Y_MAJOR, 64, 128, 4, 8, 16, 3>(x, y, offsets, E, rows, M, N, K, out, ldo,
                                                              accumulate, status, s);
    return launch_tile<WG, Y_MAJOR, 64, 64, 4, 4, 32, 3>(x, y, offsets, E, rows, M, N, K, out, ldo,
                                                         accumulate, status, s);
}

}  // namespace

cudaError_t launch_grouped_gemm_simt(const float *a, int64_t lda, const int32_t *offsets,
                                     int64_t rows, const float *w, int E, int64_t N, int64_t K,
                                     bool transposed, float *out, int64_t ldo, unsigned *status,
                                     cudaStream_t s)
{
    const SimtOperand x{a, lda, 0}, y{w, transposed ? N : K, N * K};
    if (transposed)
        return launch_sizes<false, true>(x, y, offsets, E, rows, 0, (int)N, (int)K, out, ldo, 0, status, s);
    return launch_sizes<false, false>(x, y, offsets, E, rows, 0, (int)N, (int)K, out, ldo, 0, status, s);
}

cudaError_t launch_grouped_weight_grad_simt(const float *grad, int64_t ldg, const float *a,
                                            int64_t lda, const int32_t *offsets, int64_t rows,
                                            int E, int64_t N, int64_t K, float *grad_w,
                                            bool accumulate, unsigned *status, cudaStream_t s)
{
    const SimtOperand x{grad, ldg, 0}, y{a, lda, 0};
    return launch_sizes<true, true>(x, y, offsets, E, rows, (int)N, (int)K, 0, grad_w, K, accumulate, status, s);
}

}  // namespace moe
