// k_norm.cu -- layer norm over the channels of [B][N][C], forward and backward.
//
//   xh = (x - mean) rstd, mean and variance over C, rstd = 1 / sqrt(var + eps);  y = w xh + b
//   g = w dy;  dx = rstd (g - mean(g) - xh mean(g xh));  dw = sum dy xh, db = sum dy over the rows
#include "la_dit.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float x, float *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_sum(x);
    __syncthreads();
    if (lane == 0) red[warp] = x;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) t += red[i];
    return t;
}

// One CTA a row, any C: the row is read three times (the second and third time from L1 or L2).
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_fwd_any(const T *__restrict__ x, const T *__restrict__ w, const T *__restrict__ b, T *__restrict__ y,
             float *__restrict__ mean_out, float *__restrict__ rstd_out, const NormPlan p) {
    __shared__ float red[kThreads / 32];
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *xr = x + r * p.C;
        const long long vo = p.per_batch ? r / p.N * p.C : 0;
        float s = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) s += to_f(xr[c]);
        const float mean = block_sum(s, red) / (float)p.C;
        s = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float t = to_f(xr[c]) - mean;
            s += t * t;
        }
        const float rstd = rsqrtf(block_sum(s, red) / (float)p.C + p.eps);
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            float t = (to_f(xr[c]) - mean) * rstd;
            if (w) t *= to_f(w[vo + c]);
            if (b) t += to_f(b[vo + c]);
            y[r * p.C + c] = from_f<T>(t);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_dx_any(const T *__restrict__ dy, const T *__restrict__ x, const T *__restrict__ w,
            const float *__restrict__ mean, const float *__restrict__ rstd, T *__restrict__ dx, const NormPlan p) {
    __shared__ float red[kThreads / 32];
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const long long o = r * p.C, vo = p.per_batch ? r / p.N * p.C : 0;
        const float m = mean[r], rs = rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float g = to_f(dy[o + c]) * (w ? to_f(w[vo + c]) : 1.f);
            s1 += g;
            s2 += g * ((to_f(x[o + c]) - m) * rs);
        }
        s1 = block_sum(s1, red) / (float)p.C;
        s2 = block_sum(s2, red) / (float)p.C;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float g = to_f(dy[o + c]) * (w ? to_f(w[vo + c]) : 1.f);
            const float xh = (to_f(x[o + c]) - m) * rs;
            dx[o + c] = from_f<T>(rs * (g - s1 - xh * s2));
        }
    }
}

// Column sums of dy xh and dy: one thread a column, `splits` row ranges a
// group of rows (a batch element, or all rows); part[group][split][2][C].
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_dw_part(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
             const float *__restrict__ rstd, float *__restrict__ part, const NormPlan p, int splits) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    const int g = blockIdx.z, sp = blockIdx.y;
    const long long rows = p.per_batch ? p.N : p.rows;
    const long long r0 = g * rows + rows * sp / splits, r1 = g * rows + rows * (sp + 1) / splits;
    if (c >= p.C) return;
    float a = 0.f, bsum = 0.f;
    for (long long r = r0; r < r1; ++r) {
        const float d = to_f(dy[r * p.C + c]);
        a += d * ((to_f(x[r * p.C + c]) - mean[r]) * rstd[r]);
        bsum += d;
    }
    float *o = part + ((long long)g * splits + sp) * 2 * p.C;
    o[c] = a;
    o[p.C + c] = bsum;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_dw_sum(const float *__restrict__ part, T *__restrict__ dw, T *__restrict__ db, int C, int splits) {
    const int c = blockIdx.x * kThreads + threadIdx.x, g = blockIdx.y;
    if (c >= C) return;
    float a = 0.f, b = 0.f;
    for (int s = 0; s < splits; ++s) {
        const float *o = part + ((long long)g * splits + s) * 2 * C;
        a += o[c];
        b += o[C + c];
    }
    if (dw) dw[(long long)g * C + c] = from_f<T>(a);
    if (db) db[(long long)g * C + c] = from_f<T>(b);
}

// Row ranges per group of the partial sums.
int norm_splits(const NormPlan &p) {
    const long long rows = p.per_batch ? p.N : p.rows, groups = p.per_batch ? p.B : 1;
    long long s = (2 * kTargetCtas + groups - 1) / groups;
    if (s > (rows + 15) / 16) s = (rows + 15) / 16;
    return (int)(s < 1 ? 1 : s);
}

template <typename T>
int norm_fwd_t(const T *x, const T *w, const T *b, T *y, float *mean, float *rstd, const NormPlan &p, cudaStream_t s) {
    const long long grid = p.rows < (1 << 30) ? p.rows : (1 << 30);
    norm_fwd_any<T><<<(unsigned)grid, kThreads, 0, s>>>(x, w, b, y, mean, rstd, p);
    return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

template <typename T>
int norm_bwd_t(const T *dy, const T *x, const T *w, const float *mean, const float *rstd, T *dx, T *dw, T *db,
               float *part, const NormPlan &p, cudaStream_t s) {
    const long long grid = p.rows < (1 << 30) ? p.rows : (1 << 30);
    norm_dx_any<T><<<(unsigned)grid, kThreads, 0, s>>>(dy, x, w, mean, rstd, dx, p);
    if (cudaGetLastError() != cudaSuccess) return -1;
    if (!dw && !db) return 1;
    const int sp = norm_splits(p), groups = p.per_batch ? p.B : 1;
    const unsigned cb = (unsigned)((p.C + kThreads - 1) / kThreads);
    norm_dw_part<T><<<dim3(cb, sp, groups), kThreads, 0, s>>>(dy, x, mean, rstd, part, p, sp);
    if (cudaGetLastError() != cudaSuccess) return -1;
    norm_dw_sum<T><<<dim3(cb, groups), kThreads, 0, s>>>(part, dw, db, p.C, sp);
    return cudaGetLastError() == cudaSuccess ? 3 : -1;
}

}  // namespace

size_t norm_bwd_ws(const NormPlan &p) {
    return align256(size_t(p.per_batch ? p.B : 1) * norm_splits(p) * 2 * p.C * sizeof(float));
}

int launch_norm_fwd(int is_bf16, const void *x, const void *w, const void *b, void *y, float *mean, float *rstd,
                    const NormPlan &p, cudaStream_t s) {
    using bf = __nv_bfloat16;
    return is_bf16 ? norm_fwd_t<bf>((const bf *)x, (const bf *)w, (const bf *)b, (bf *)y, mean, rstd, p, s)
                   : norm_fwd_t<float>((const float *)x, (const float *)w, (const float *)b, (float *)y, mean, rstd, p, s);
}

int launch_norm_bwd(int is_bf16, const void *dy, const void *x, const void *w, const float *mean, const float *rstd,
                    void *dx, void *dw, void *db, void *ws, const NormPlan &p, cudaStream_t s) {
    using bf = __nv_bfloat16;
    return is_bf16 ? norm_bwd_t<bf>((const bf *)dy, (const bf *)x, (const bf *)w, mean, rstd, (bf *)dx, (bf *)dw,
                                    (bf *)db, (float *)ws, p, s)
                   : norm_bwd_t<float>((const float *)dy, (const float *)x, (const float *)w, mean, rstd, (float *)dx,
                                       (float *)dw, (float *)db, (float *)ws, p, s);
}

}  // namespace la
