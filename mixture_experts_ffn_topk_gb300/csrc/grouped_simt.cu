// grouped_simt.cu -- grouped products of FP32 rows on CUDA cores (true FP32:
// tensor cores would round the operands to TF32).
//
// For the rows r of expert e (offsets[e] <= r < offsets[e + 1]):
//   product       out[r, n] = sum_k a[r, k] w[e][n, k]   (or w[e][k, n])
//   weight grad   grad_w[e][n, k] = sum_r grad[r, n] a[r, k]
// One tiled kernel: C [M, N] = sum_k X(m, k) Y(n, k), where each operand is
// stored either with k contiguous (X[m][k]) or with m contiguous (X[k][m]).
// Tiles of BM x BN outputs, TM x TN of them per thread, k in steps of BK kept
// twice in shared memory (k-major, so that a thread's TM and TN values are
// vector loads); the next step's global loads are in flight during the
// current one's products.
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

// WG: the reduction runs over the expert's rows (X = grad, Y = a, both stored
// with the output index contiguous). Otherwise X = a (k contiguous), Y = w,
// k contiguous unless Y_MAJOR.
template <bool WG, bool Y_MAJOR, int BM, int BN, int TM, int TN>
__global__ void __launch_bounds__(BM / TM * (BN / TN))
grouped_simt_kernel(SimtOperand x, SimtOperand y, const int32_t *__restrict__ offsets, int E,
                    int rows, int M, int N, int K, float *__restrict__ out, int64_t ldo,
                    int accumulate, unsigned *status)
{
    constexpr int BK = 16, THREADS = BM / TM * (BN / TN);
    constexpr int XV = BM * BK / 4 / THREADS, YV = BN * BK / 4 / THREADS;
    static_assert(XV >= 1 && YV >= 1, "each thread loads at least one vector of each operand");
    constexpr bool X_MAJOR = WG;
    __shared__ Segments S;
    __shared__ int warp_sum[THREADS / 32];
    __shared__ __align__(16) float Xs[2][BK][BM + 4];
    __shared__ __align__(16) float Ys[2][BK][BN + 4];
    pdl_wait();
    pdl_launch_dependents();
    const int nt = (N + BN - 1) / BN;
    load_segments<THREADS>(S, warp_sum, offsets, E, rows, status, [&](int cnt) {
        return WG ? (M + BM - 1) / BM * nt : (cnt + BM - 1) / BM * nt;
    });
    __syncthreads();
    const int total = S.unit[E];
    const int tm = threadIdx.x / (BN / TN), tn = threadIdx.x % (BN / TN);
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
        const int e = expert_of(S, E, unit), loc = unit - S.unit[e];
        const int first = S.first[e], cnt = S.count[e];
        const int m0 = loc / nt * BM, n0 = loc % nt * BN;
        const int m_end = WG ? M : cnt, k_end = WG ? cnt : K;
        // element (0, 0) of this unit's operands
        const float *xp = x.p + (int64_t)first * x.ld;
        const float *yp = y.p + (WG ? (int64_t)first * y.ld : (int64_t)e * y.per_expert);

        float4 xr[XV], yr[YV];
        // one vector of four: along k (k contiguous) or along the output index
        auto fetch = [&](const float *p, int64_t ld, bool major, int i0, int i_end, int k0, int v, int B) {
            int i, k;
            if (major) { k = v / (B / 4); i = v % (B / 4) * 4; }
            else { i = v / (BK / 4); k = v % (BK / 4) * 4; }
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + i < i_end && k0 + k < k_end)
                r = *reinterpret_cast<const float4 *>(
                    p + (major ? (int64_t)(k0 + k) * ld + i0 + i : (int64_t)(i0 + i) * ld + k0 + k));
            return r;
        };
        auto fetch_all = [&](int k0) {
#pragma unroll
            for (int q = 0; q < XV; ++q)
                xr[q] = fetch(xp, x.ld, X_MAJOR, m0, m_end, k0, threadIdx.x + q * THREADS, BM);
#pragma unroll
            for (int q = 0; q < YV; ++q)
                yr[q] = fetch(yp, y.ld, Y_MAJOR, n0, N, k0, threadIdx.x + q * THREADS, BN);
        };
        auto put = [&](int buf) {
#pragma unroll
            for (int q = 0; q < XV; ++q) {
                const int v = threadIdx.x + q * THREADS;
                if (X_MAJOR) {
                    *reinterpret_cast<float4 *>(&Xs[buf][v / (BM / 4)][v % (BM / 4) * 4]) = xr[q];
                } else {
                    const int i = v / (BK / 4), k = v % (BK / 4) * 4;
                    Xs[buf][k][i] = xr[q].x; Xs[buf][k + 1][i] = xr[q].y;
                    Xs[buf][k + 2][i] = xr[q].z; Xs[buf][k + 3][i] = xr[q].w;
                }
            }
#pragma unroll
            for (int q = 0; q < YV; ++q) {
                const int v = threadIdx.x + q * THREADS;
                if (Y_MAJOR) {
                    *reinterpret_cast<float4 *>(&Ys[buf][v / (BN / 4)][v % (BN / 4) * 4]) = yr[q];
                } else {
                    const int i = v / (BK / 4), k = v % (BK / 4) * 4;
                    Ys[buf][k][i] = yr[q].x; Ys[buf][k + 1][i] = yr[q].y;
                    Ys[buf][k + 2][i] = yr[q].z; Ys[buf][k + 3][i] = yr[q].w;
                }
            }
        };

        float acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = 0.0f;
        const int steps = (k_end + BK - 1) / BK;
        if (steps > 0) {
            fetch_all(0);
            put(0);
        }
        __syncthreads();
        for (int t = 0; t < steps; ++t) {
            const int buf = t & 1;
            if (t + 1 < steps) fetch_all((t + 1) * BK);
#pragma unroll
            for (int k = 0; k < BK; ++k) {
                float a[TM], b[TN];
#pragma unroll
                for (int i = 0; i < TM; i += 2)
                    *reinterpret_cast<float2 *>(&a[i]) = *reinterpret_cast<const float2 *>(&Xs[buf][k][tm * TM + i]);
#pragma unroll
                for (int j = 0; j < TN; j += 2)
                    *reinterpret_cast<float2 *>(&b[j]) = *reinterpret_cast<const float2 *>(&Ys[buf][k][tn * TN + j]);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            }
            if (t + 1 < steps) put(buf ^ 1);
            __syncthreads();
        }
        const int64_t out0 = WG ? (int64_t)e * M * ldo : (int64_t)first * ldo;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = m0 + tm * TM + i;
            if (m >= m_end) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = n0 + tn * TN + j;
                if (n >= N) continue;
                const int64_t at = out0 + (int64_t)m * ldo + n;
                out[at] = accumulate ? out[at] + acc[i][j] : acc[i][j];
            }
        }
    }
}

template <bool WG, bool Y_MAJOR, int BM, int BN, int TM, int TN>
cudaError_t launch_tile(const SimtOperand &x, const SimtOperand &y, const int32_t *offsets, int E,
                        int64_t rows, int M, int N, int K, float *out, int64_t ldo,
                        int accumulate, unsigned *status, cudaStream_t s)
{
    const int64_t nt = (N + BN - 1) / BN;
    const int64_t mt = WG ? (int64_t)E * ((M + BM - 1) / BM) : rows / BM + (rows < E ? rows : E);
    const int64_t units = mt * nt, most = (int64_t)device_sm_count() * 4;
    return launch_pdl(grouped_simt_kernel<WG, Y_MAJOR, BM, BN, TM, TN>,
                      dim3((unsigned)(units < most ? units : most)), dim3(BM / TM * (BN / TN)), 0, s,
                      x, y, offsets, E, (int)rows, M, N, K, out, ldo, accumulate, status);
}

template <bool WG, bool Y_MAJOR>
cudaError_t launch_sizes(const SimtOperand &x, const SimtOperand &y, const int32_t *offsets, int E,
                         int64_t rows, int M, int N, int K, float *out, int64_t ldo,
                         int accumulate, unsigned *status, cudaStream_t s)
{
    return launch_tile<WG, Y_MAJOR, 64, 64, 4, 4>(x, y, offsets, E, rows, M, N, K, out, ldo,
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
