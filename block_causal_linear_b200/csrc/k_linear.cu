// k_linear.cu -- the parts of the linear layer that run on the CUDA cores:
// products with few rows, the activation's derivative and column sums.
//
//   C[m][n] = sum_k A(m, k) B(n, k);  z = C + bias;  pre = z;  y = act(z) + residual
#include "la_sm100_dit.cuh"

namespace la {

using namespace sm100;

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void epilogue(const GemmPlan &g, long long m, long long n, float z) {
    const long long o = m * g.N + n;
    if (g.bias) z += to_f(((const T *)g.bias)[n]);
    using P = typename PreOf<T>::type;
    if (g.pre) ((P *)g.pre)[o] = to_pre<P>(z, g.act);
    z = act_f(z, g.act);
    if (g.res) z += to_f(((const T *)g.res)[o]);
    ((T *)g.y)[o] = from_f<T>(z);
}

// Products with at most 8 rows, both operands k-contiguous: the weight's bytes
// are the time, so each is read once, by whole warps, up to 16 bytes a lane
// (VEC), NC columns at a time for all R rows.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T, int VEC, int R, int NC>
__global__ void __launch_bounds__(kThreads)
gemm_rows(const GemmPlan g) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n0 = ((long long)blockIdx.x * (kThreads / 32) + warp) * NC;
    const T *A = (const T *)g.a, *B = (const T *)g.b;
    if (n0 >= g.N) return;
    float acc[R][NC] = {};
    constexpr int kAhead = VEC * sizeof(T) >= 8 ? 2 : 4;
#pragma unroll kAhead
    for (long long k = lane * VEC; k < g.K; k += 32 * VEC) {
        Pack<T, VEC> b[NC], a[R];
#pragma unroll
        for (int j = 0; j < NC; ++j)
            b[j] = *reinterpret_cast<const Pack<T, VEC> *>(B + (n0 + j < g.N ? n0 + j : g.N - 1) * g.ldb + k);
#pragma unroll
        for (int i = 0; i < R; ++i)
            a[i] = *reinterpret_cast<const Pack<T, VEC> *>(A + (i < g.M ? i : g.M - 1) * g.lda + k);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const float f = to_f(b[j].v[e]);
#pragma unroll
                for (int i = 0; i < R; ++i) acc[i][j] += to_f(a[i].v[e]) * f;
            }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const float z = warp_sum(acc[i][j]);
            if (lane == i * NC + j && i < g.M && n0 + j < g.N) epilogue<T>(g, i, n0 + j, z);
        }
}

template <typename T, int VEC, int R>
int rows_nc(const GemmPlan &g, cudaStream_t s) {
    // 4 columns a warp where that still leaves 4 warps a scheduler of the GPU, else 1
    const bool ok = g.N >= 4 * 16 * kSmCount ? launch_dep(gemm_rows<T, VEC, R, 4>, dim3((unsigned)((g.N + 31) / 32)), kThreads, 0, s, g)
                                             : launch_dep(gemm_rows<T, VEC, R, 1>, dim3((unsigned)((g.N + 7) / 8)), kThreads, 0, s, g);
    return ok ? 1 : -1;
}

template <typename T, int VEC>
int rows_r(const GemmPlan &g, cudaStream_t s) {
    if (g.M <= 1) return rows_nc<T, VEC, 1>(g, s);
    if (g.M <= 2) return rows_nc<T, VEC, 2>(g, s);
    if (g.M <= 4) return rows_nc<T, VEC, 4>(g, s);
    return rows_nc<T, VEC, 8>(g, s);
}

// dz = dy act'(pre) and the column sums of dz (of dy without an activation),
// in one pass: a warp walks rows of 32 x VEC columns, a CTA's 8 warps every
// 8th row of its range; the warps' sums are added in warp order and leave as
// part[split][C].  dz or part may be null.
constexpr int kColCtas = 5;      // CTAs a SM
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, kColCtas)
act_col(const T *__restrict__ dy, const typename PreOf<T>::type *__restrict__ pre, T *__restrict__ dz,
        float *__restrict__ part, long long R, long long C) {
    pdl_wait_for(dy, pre);
    pdl_trigger();
    using P = typename PreOf<T>::type;
    __shared__ float red[8][32 * VEC];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long c = ((long long)blockIdx.x * 32 + lane) * VEC;
    const long long sp = blockIdx.y, splits = gridDim.y;
    const long long r1 = R * (sp + 1) / splits;
    float a[VEC] = {};
    // (more CTAs carry a slope's arithmetic better than more rows a warp: 8190 x 5120 SiLU 51 us, 73 with four rows in flight)
    constexpr int kAhead = ACT ? 1 : 4;
    if (c < C) {
#pragma unroll kAhead
        for (long long r = R * sp / splits + warp; r < r1; r += 8) {
            Pack<T, VEC> d = *reinterpret_cast<const Pack<T, VEC> *>(dy + r * C + c);
            if constexpr (ACT != 0) {
                const Pack<P, VEC> z = *reinterpret_cast<const Pack<P, VEC> *>(pre + r * C + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float f = to_f(d.v[j]) * act_slope(from_pre(z.v[j]), ACT);
                    a[j] += f;
                    d.v[j] = from_f<T>(f);
                }
                if (dz) *reinterpret_cast<Pack<T, VEC> *>(dz + r * C + c) = d;
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) a[j] += to_f(d.v[j]);
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[warp][j * 32 + lane] = a[j];
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * VEC; e += kThreads) {
        const long long col = ((long long)blockIdx.x * 32 + e % 32) * VEC + e / 32;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += red[w][e];
        if (col < C) part[sp * C + col] = s;
    }
}

int col_splits(long long R, long long C) {
    const long long cb = (C + 255) / 256;
    long long s = kColCtas * kSmCount / cb;
    if (s > (R + 31) / 32) s = (R + 31) / 32;
    if (s > 65535) s = 65535;
    return (int)(s < 1 ? 1 : s);
}

template <typename T, int VEC>
int act_col_t(const void *dy, const void *pre, void *dz, float *part, long long R, long long C, int act, cudaStream_t s) {
    const dim3 grid((unsigned)((C + 32 * VEC - 1) / (32 * VEC)), (unsigned)col_splits(R, C));
    auto f = act == 1 ? act_col<T, VEC, 1> : (act == 2 ? act_col<T, VEC, 2> : (act == 3 ? act_col<T, VEC, 3> : act_col<T, VEC, 0>));
    return launch_dep(f, grid, kThreads, 0, s, (const T *)dy, (const typename PreOf<T>::type *)pre, (T *)dz, part, R, C) ? 1 : -1;
}

}  // namespace

int launch_gemm_rows(int is_bf16, const GemmPlan &g, cudaStream_t s) {
    if (is_bf16)
        return g.K % 8 == 0   ? rows_r<__nv_bfloat16, 8>(g, s)
               : g.K % 4 == 0 ? rows_r<__nv_bfloat16, 4>(g, s)
               : g.K % 2 == 0 ? rows_r<__nv_bfloat16, 2>(g, s)
                              : rows_r<__nv_bfloat16, 1>(g, s);
    return g.K % 4 == 0 ? rows_r<float, 4>(g, s) : (g.K % 2 == 0 ? rows_r<float, 2>(g, s) : rows_r<float, 1>(g, s));
}

size_t act_col_ws(long long R, long long C) { return align256(size_t(col_splits(R, C)) * C * sizeof(float)); }

int launch_act_col(int is_bf16, const void *dy, const void *pre, void *dz, void *colsum, long long R, long long C,
                   int act, void *ws, cudaStream_t s) {
    float *part = colsum ? (float *)ws : nullptr;
    int r;
    if (is_bf16)
        r = C % 8 == 0 ? act_col_t<__nv_bfloat16, 8>(dy, pre, dz, part, R, C, act, s)
                       : act_col_t<__nv_bfloat16, 1>(dy, pre, dz, part, R, C, act, s);
    else
        r = C % 4 == 0 ? act_col_t<float, 4>(dy, pre, dz, part, R, C, act, s)
                       : act_col_t<float, 1>(dy, pre, dz, part, R, C, act, s);
    if (r < 0 || !colsum) return r;
    return launch_split_sum(is_bf16, part, colsum, C, col_splits(R, C), s) < 0 ? -1 : 2;
}

}  // namespace la
