// k_cross.cu -- cross attention to an encoder's states on the CUDA cores.
//
//   s_j = scale q . k_j over the valid states j < len;  p = softmax(s);  o = sum p_j v_j
// One pass over the states with the running maximum and sum; a sample without
// valid states has o = 0 and lse = -inf.  Backward, with D = dout . o:
//   dv_j = sum_i p_ij dout_i;  ds_ij = p_ij (dout_i . v_j - D_i);
//   dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_i ds_ij q_i
#include "la_dit.cuh"

namespace la {
namespace {

constexpr int kQ = 128;      // queries (threads) a CTA, one each
constexpr int kKeys = 32;    // states a shared-memory tile
constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int D>
__device__ __forceinline__ void load_row(float (&r)[D], const T *p, bool ok) {
#pragma unroll
    for (int i = 0; i < D; ++i) r[i] = ok ? to_f(p[i]) : 0.f;
}

// rows [j0, j0 + n) of a [..][ld] tensor's head, as fp32, n <= kKeys
template <typename T, int D>
__device__ __forceinline__ void load_tile(float (&t)[kKeys][D], const T *base, long long ld, int j0, int n) {
    for (int e = threadIdx.x; e < n * D; e += blockDim.x) t[e / D][e % D] = to_f(base[(long long)(j0 + e / D) * ld + e % D]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ)
cross_fwd_ffma(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, T *__restrict__ out,
               float *__restrict__ lse, const CrossPlan p) {
    __shared__ float ks[kKeys][D], vs[kKeys][D];
    const int b = blockIdx.y / p.H, h = blockIdx.y % p.H;
    const long long i = (long long)blockIdx.x * kQ + threadIdx.x;
    const bool ok = i < p.N;
    const long long qo = (((long long)b * p.N + (ok ? i : 0)) * p.H + h) * D;
    const T *kb = k + (long long)b * p.M * p.ldk + (long long)h * D;
    const T *vb = v + (long long)b * p.M * p.ldv + (long long)h * D;
    const int len = cross_len(p, b);
    const float c = p.scale * kLog2e;
    float qr[D], acc[D] = {};
    load_row<T, D>(qr, q + qo, ok);
    float m = -INFINITY, l = 0.f;
    for (int j0 = 0; j0 < len; j0 += kKeys) {
        const int n = len - j0 < kKeys ? len - j0 : kKeys;
        __syncthreads();
        load_tile<T, D>(ks, kb, p.ldk, j0, n);
        load_tile<T, D>(vs, vb, p.ldv, j0, n);
        __syncthreads();
        for (int j = 0; j < n; ++j) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < D; ++e) s += qr[e] * ks[j][e];
            s *= c;
            const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
            l = l * f + w;
            m = mn;
#pragma unroll
            for (int e = 0; e < D; ++e) acc[e] = acc[e] * f + w * vs[j][e];
        }
    }
    if (!ok) return;
    const float inv = len > 0 ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < D; ++e) out[qo + e] = from_f<T>(acc[e] * inv);
    if (lse) lse[((long long)b * p.H + h) * p.N + i] = len > 0 ? (m + log2f(l)) / kLog2e : -INFINITY;
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ)
cross_dq_ffma(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ out,
              const T *__restrict__ dout, const float *__restrict__ lse, T *__restrict__ dq, float *__restrict__ delta,
              const CrossPlan p) {
    __shared__ float ks[kKeys][D], vs[kKeys][D];
    const int b = blockIdx.y / p.H, h = blockIdx.y % p.H;
    const long long i = (long long)blockIdx.x * kQ + threadIdx.x;
    const bool ok = i < p.N;
    const long long qo = (((long long)b * p.N + (ok ? i : 0)) * p.H + h) * D;
    const long long ro = ((long long)b * p.H + h) * p.N + i;
    const T *kb = k + (long long)b * p.M * p.ldk + (long long)h * D;
    const T *vb = v + (long long)b * p.M * p.ldv + (long long)h * D;
    const int len = cross_len(p, b);
    float qr[D], dr[D], acc[D] = {}, dl = 0.f;
    load_row<T, D>(qr, q + qo, ok);
    load_row<T, D>(dr, dout + qo, ok);
#pragma unroll
    for (int e = 0; e < D; ++e) dl += ok ? dr[e] * to_f(out[qo + e]) : 0.f;
    const float ls = ok && len > 0 ? lse[ro] * kLog2e : 0.f, c = p.scale * kLog2e;
    for (int j0 = 0; j0 < len; j0 += kKeys) {
        const int n = len - j0 < kKeys ? len - j0 : kKeys;
        __syncthreads();
        load_tile<T, D>(ks, kb, p.ldk, j0, n);
        load_tile<T, D>(vs, vb, p.ldv, j0, n);
        __syncthreads();
        for (int j = 0; j < n; ++j) {
            float s = 0.f, dp = 0.f;
#pragma unroll
            for (int e = 0; e < D; ++e) s += qr[e] * ks[j][e], dp += dr[e] * vs[j][e];
            const float ds = exp2f(s * c - ls) * (dp - dl) * p.scale;
#pragma unroll
            for (int e = 0; e < D; ++e) acc[e] += ds * ks[j][e];
        }
    }
    if (!ok) return;
    delta[ro] = dl;
#pragma unroll
    for (int e = 0; e < D; ++e) dq[qo + e] = from_f<T>(acc[e]);
}

constexpr int kStates = 64;   // encoder states (threads) a CTA of the key side

// dk, dv of 64 states over one range of queries: part[split][b][h][M][2][D]
template <typename T, int D>
__global__ void __launch_bounds__(kStates)
cross_dkv_ffma(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ dout,
               const float *__restrict__ lse, const float *__restrict__ delta, float *__restrict__ part,
               const CrossPlan p) {
    __shared__ float qs[kKeys][D], gs[kKeys][D], ls[kKeys], dl[kKeys];
    const int b = blockIdx.y / p.H, h = blockIdx.y % p.H, sp = blockIdx.z, splits = gridDim.z;
    const int j = blockIdx.x * kStates + threadIdx.x;
    const int len = cross_len(p, b);
    if (blockIdx.x * kStates >= len) return;   // these states' sums are not read
    const bool ok = j < len;
    const int i0 = (int)((long long)p.N * sp / splits), i1 = (int)((long long)p.N * (sp + 1) / splits);
    float kr[D], vr[D], dk[D] = {}, dv[D] = {};
    load_row<T, D>(kr, k + ((long long)b * p.M + (ok ? j : 0)) * p.ldk + (long long)h * D, ok);
    load_row<T, D>(vr, v + ((long long)b * p.M + (ok ? j : 0)) * p.ldv + (long long)h * D, ok);
    const long long base = ((long long)b * p.N * p.H + h) * D, ld = (long long)p.H * D;
    const long long ro = ((long long)b * p.H + h) * p.N;
    const float c = p.scale * kLog2e;
    for (int t = i0; t < i1; t += kKeys) {
        const int n = i1 - t < kKeys ? i1 - t : kKeys;
        __syncthreads();
        load_tile<T, D>(qs, q + base, ld, t, n);
        load_tile<T, D>(gs, dout + base, ld, t, n);
        for (int e = threadIdx.x; e < n; e += kStates) ls[e] = lse[ro + t + e] * kLog2e, dl[e] = delta[ro + t + e];
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            float s = 0.f, dp = 0.f;
#pragma unroll
            for (int e = 0; e < D; ++e) s += kr[e] * qs[i][e], dp += vr[e] * gs[i][e];
            const float w = exp2f(s * c - ls[i]), ds = w * (dp - dl[i]) * p.scale;
#pragma unroll
            for (int e = 0; e < D; ++e) dv[e] += w * gs[i][e], dk[e] += ds * qs[i][e];
        }
    }
    if (!ok) return;
    float *o = part + ((((long long)sp * p.B + b) * p.H + h) * p.M + j) * 2 * D;
#pragma unroll
    for (int e = 0; e < D; ++e) o[e] = dk[e], o[D + e] = dv[e];
}

// dk, dv = the splits' sums in split order; zero behind a sample's last valid state
template <typename T, int D>
__global__ void __launch_bounds__(256)
cross_dkv_sum(const float *__restrict__ part, T *__restrict__ dk, T *__restrict__ dv, const CrossPlan p, int splits) {
    const long long per = (long long)p.B * p.H * p.M * 2 * D;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < per; e += (long long)gridDim.x * 256) {
        const int f = (int)(e % (2 * D));
        long long r = e / (2 * D);
        const int j = (int)(r % p.M);
        r /= p.M;
        const int h = (int)(r % p.H), b = (int)(r / p.H);
        float a = 0.f;
        if (j < cross_len(p, b))
            for (int s = 0; s < splits; ++s) a += part[s * per + e];
        T *o = f < D ? dk + ((long long)b * p.M + j) * p.lddk : dv + ((long long)b * p.M + j) * p.lddv;
        o[(long long)h * D + f % D] = from_f<T>(a);
    }
}

int dkv_splits(const CrossPlan &p) {
    const long long ctas = (long long)p.B * p.H * ((p.M + kStates - 1) / kStates);
    long long s = (2 * kTargetCtas + ctas - 1) / ctas;
    if (s > (p.N + 63) / 64) s = (p.N + 63) / 64;
    return (int)(s < 1 ? 1 : s);
}

size_t dkv_part_bytes(const CrossPlan &p, int splits) {
    return align256(size_t(splits) * p.B * p.H * p.M * 2 * p.d * sizeof(float));
}

template <typename T, int D>
int fwd_t(const void *q, const void *k, const void *v, void *out, float *lse, const CrossPlan &p, cudaStream_t s) {
    const dim3 grid((unsigned)((p.N + kQ - 1) / kQ), (unsigned)(p.B * p.H));
    cross_fwd_ffma<T, D><<<grid, kQ, 0, s>>>((const T *)q, (const T *)k, (const T *)v, (T *)out, lse, p);
    return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

template <typename T, int D>
int bwd_t(const void *q, const void *k, const void *v, const void *out, const void *dout, const float *lse, void *dq,
          void *dk, void *dv, const CrossPlan &p, void *ws, cudaStream_t s) {
    const int sp = dkv_splits(p);
    float *part = (float *)ws, *delta = (float *)((char *)ws + dkv_part_bytes(p, sp));
    const dim3 gq((unsigned)((p.N + kQ - 1) / kQ), (unsigned)(p.B * p.H));
    cross_dq_ffma<T, D><<<gq, kQ, 0, s>>>((const T *)q, (const T *)k, (const T *)v, (const T *)out, (const T *)dout,
                                          lse, (T *)dq, delta, p);
    if (cudaGetLastError() != cudaSuccess) return -1;
    const dim3 gk((unsigned)((p.M + kStates - 1) / kStates), (unsigned)(p.B * p.H), (unsigned)sp);
    cross_dkv_ffma<T, D><<<gk, kStates, 0, s>>>((const T *)q, (const T *)k, (const T *)v, (const T *)dout, lse, delta,
                                                part, p);
    if (cudaGetLastError() != cudaSuccess) return -1;
    const long long n = (long long)p.B * p.H * p.M * 2 * D;
    const long long want = (n + 255) / 256;
    cross_dkv_sum<T, D><<<(unsigned)(want < 16 * kTargetCtas ? want : 16 * kTargetCtas), 256, 0, s>>>(
        part, (T *)dk, (T *)dv, p, sp);
    return cudaGetLastError() == cudaSuccess ? 3 : -1;
}

}  // namespace

size_t cross_fwd_ws(int is_bf16, const CrossPlan &p) {
    const size_t n = is_bf16 ? cross_fwd_tc_ws(p) : 0;
    return n ? n : 256;
}

size_t cross_bwd_ws(int is_bf16, const CrossPlan &p) {
    if (is_bf16) return cross_bwd_tc_ws(p);
    return dkv_part_bytes(p, dkv_splits(p)) + align256(size_t(p.B) * p.H * p.N * sizeof(float));
}

int launch_cross_fwd(int is_bf16, const void *q, const void *k, const void *v, void *out, float *lse,
                     const CrossPlan &p, void *ws, cudaStream_t s) {
    if (is_bf16) return launch_cross_fwd_tc(q, k, v, out, lse, p, ws, s);
    return p.d == 32 ? fwd_t<float, 32>(q, k, v, out, lse, p, s) : fwd_t<float, 64>(q, k, v, out, lse, p, s);
}

int launch_cross_bwd(int is_bf16, const void *q, const void *k, const void *v, const void *out, const void *dout,
                     const float *lse, void *dq, void *dk, void *dv, const CrossPlan &p, void *ws, cudaStream_t s) {
    if (is_bf16) return launch_cross_bwd_tc(q, k, v, out, dout, lse, dq, dk, dv, p, ws, s);
    return p.d == 32 ? bwd_t<float, 32>(q, k, v, out, dout, lse, dq, dk, dv, p, ws, s)
                     : bwd_t<float, 64>(q, k, v, out, dout, lse, dq, dk, dv, p, ws, s);
}

}  // namespace la
