// k_linear.cu -- matrix products with bias, activation and residual on the
// CUDA cores (fp32 accumulation), the activation's derivative, column sums.
//
//   C[m][n] = sum_k A(m, k) B(n, k);  z = C + bias;  y = act(z) + residual
// The three products of a linear layer are this one with other layouts:
// forward A = x, B = W; dx: A = dz, B = W read along its rows; dW: both read
// along their rows.
#include "la_dit.cuh"

namespace la {
namespace {

constexpr int kBM = 64, kBN = 64, kBK = 16, kThreads = 256;

// 64x64 tile, 4x4 outputs a thread.  AMN / BMN: the operand's m (n) index is contiguous.
template <typename T, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads)
gemm_ffma(const GemmPlan g) {
    __shared__ float sa[kBK][kBM + 4], sb[kBK][kBN + 4];
    const T *A = (const T *)g.a, *B = (const T *)g.b;
    const long long nt = (g.N + kBN - 1) / kBN;
    const long long m0 = (long long)blockIdx.x / nt * kBM, n0 = (long long)blockIdx.x % nt * kBN;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (long long k0 = 0; k0 < g.K; k0 += kBK) {
#pragma unroll
        for (int i = 0; i < kBM * kBK / kThreads; ++i) {
            const int e = threadIdx.x + i * kThreads;
            {
                const int m = AMN ? e % kBM : e / kBK, k = AMN ? e / kBM : e % kBK;
                const bool ok = m0 + m < g.M && k0 + k < g.K;
                sa[k][m] = ok ? to_f(AMN ? A[(k0 + k) * g.lda + m0 + m] : A[(m0 + m) * g.lda + k0 + k]) : 0.f;
            }
            {
                const int n = BMN ? e % kBN : e / kBK, k = BMN ? e / kBN : e % kBK;
                const bool ok = n0 + n < g.N && k0 + k < g.K;
                sb[k][n] = ok ? to_f(BMN ? B[(k0 + k) * g.ldb + n0 + n] : B[(n0 + n) * g.ldb + k0 + k]) : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sa[k][ty * 4 + i], b[i] = sb[k][tx * 4 + i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += a[i] * b[j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= g.M || n >= g.N) continue;
            const long long o = m * g.N + n;
            float z = acc[i][j];
            if (g.bias) z += to_f(((const T *)g.bias)[n]);
            if (g.pre) ((T *)g.pre)[o] = from_f<T>(z);
            z = act_f(z, g.act);
            if (g.res) z += to_f(((const T *)g.res)[o]);
            ((T *)g.y)[o] = from_f<T>(z);
        }
}

template <typename T>
int gemm_t(const GemmPlan &g, cudaStream_t s) {
    const long long grid = ((g.M + kBM - 1) / kBM) * ((g.N + kBN - 1) / kBN);
    if (grid > 0x7fffffffLL) return -1;
    auto f = g.a_mn ? (g.b_mn ? gemm_ffma<T, true, true> : gemm_ffma<T, true, false>)
                    : (g.b_mn ? gemm_ffma<T, false, true> : gemm_ffma<T, false, false>);
    f<<<(unsigned)grid, kThreads, 0, s>>>(g);
    return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
act_bwd_kernel(const T *__restrict__ dy, const T *__restrict__ pre, T *__restrict__ dz, long long n, int act) {
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads)
        dz[i] = from_f<T>(to_f(dy[i]) * act_slope(to_f(pre[i]), act));
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
col_part(const T *__restrict__ x, float *__restrict__ part, long long R, long long C) {
    const long long c = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long sp = blockIdx.y, splits = gridDim.y;
    if (c >= C) return;
    float a = 0.f;
    for (long long r = R * sp / splits; r < R * (sp + 1) / splits; ++r) a += to_f(x[r * C + c]);
    part[sp * C + c] = a;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
col_sum(const float *__restrict__ part, T *__restrict__ out, long long C, int splits) {
    const long long c = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float a = 0.f;
    for (int s = 0; s < splits; ++s) a += part[(long long)s * C + c];
    out[c] = from_f<T>(a);
}

int col_splits(long long R, long long C) {
    const long long cb = (C + kThreads - 1) / kThreads;
    long long s = (4 * kTargetCtas + cb - 1) / cb;
    if (s > (R + 15) / 16) s = (R + 15) / 16;
    return (int)(s < 1 ? 1 : s);
}

}  // namespace

int launch_gemm_ffma(int is_bf16, const GemmPlan &g, cudaStream_t s) {
    return is_bf16 ? gemm_t<__nv_bfloat16>(g, s) : gemm_t<float>(g, s);
}

int launch_act_bwd(int is_bf16, const void *dy, const void *pre, void *dz, long long n, int act, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const long long want = (n + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(want < 16 * kTargetCtas ? want : 16 * kTargetCtas);
    if (is_bf16) act_bwd_kernel<bf><<<grid, kThreads, 0, s>>>((const bf *)dy, (const bf *)pre, (bf *)dz, n, act);
    else act_bwd_kernel<float><<<grid, kThreads, 0, s>>>((const float *)dy, (const float *)pre, (float *)dz, n, act);
    return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

size_t col_sum_ws(long long R, long long C) { return align256(size_t(col_splits(R, C)) * C * sizeof(float)); }

int launch_col_sum(int is_bf16, const void *x, void *out, long long R, long long C, void *ws, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const int sp = col_splits(R, C);
    const unsigned cb = (unsigned)((C + kThreads - 1) / kThreads);
    if (is_bf16) col_part<bf><<<dim3(cb, sp), kThreads, 0, s>>>((const bf *)x, (float *)ws, R, C);
    else col_part<float><<<dim3(cb, sp), kThreads, 0, s>>>((const float *)x, (float *)ws, R, C);
    if (cudaGetLastError() != cudaSuccess) return -1;
    if (is_bf16) col_sum<bf><<<cb, kThreads, 0, s>>>((const float *)ws, (bf *)out, C, sp);
    else col_sum<float><<<cb, kThreads, 0, s>>>((const float *)ws, (float *)out, C, sp);
    return cudaGetLastError() == cudaSuccess ? 2 : -1;
}

}  // namespace la
