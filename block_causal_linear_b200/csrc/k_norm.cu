// k_norm.cu -- layer norm over the channels of [B][N][C], forward and backward.
//
//   xh = (x - mean) rstd, mean and variance over C, rstd = 1 / sqrt(var + eps);  y = w xh + b
//   g = w dy;  dx = rstd (g - mean(g) - xh mean(g xh));  dw = sum dy xh, db = sum dy over the rows
//
// Bound by HBM: each element is read once (x; x and dy) and written once (75600
// rows of 2048 bf16: 117 us, 5.3 TB/s; 4 x 8190 rows forward and backward 138
// us, 4.9 TB/s).  Many
// rows of whole 16 bytes run a warp a row (forward, up to 2048 channels) or a
// few (backward, up to 8192), the rows arriving by bulk copies in rings of
// those warps' own, so that what is in flight does not depend on registers or
// on other warps; few rows, wider ones and ones at odd addresses have forms of
// their own below.
#include "la_sm100_dit.cuh"

namespace la {

using namespace sm100;

namespace {

// Raised by a bounded wait that gave up; read by la_device_status.
__device__ unsigned int g_norm_flag = 0;

constexpr int kThreads = 256;
constexpr int kRing = 8;       // most stages of the backward pass's ring

// VEC elements moved by one load or store.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// Elements j and j + 1 (j even) as floats, and back: a bf16 pair is one word, so
// that reading it is two instructions and writing it one (element by element
// it was six).
template <typename T, int VEC>
__device__ __forceinline__ float2 get2(const Pack<T, VEC> &p, int j) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(&p)[j / 2];
        return make_float2(bf_lo(w), bf_hi(w));
    } else {
        return make_float2(p.v[j], p.v[j + 1]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void set2(Pack<T, VEC> &p, int j, float2 f) {
    if constexpr (sizeof(T) == 2) {
        reinterpret_cast<uint32_t *>(&p)[j / 2] = pack_bf2(f.x, f.y);
    } else {
        p.v[j] = f.x;
        p.v[j + 1] = f.y;
    }
}

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) { return *reinterpret_cast<const Pack<T, VEC> *>(p); }

// A warp's rows r0, r0 + step, ... in a ring of slots of `pieces` rows (x, or x
// and dy) each.
template <typename T, int PIECES>
struct RowRing {
    uint8_t *slots;
    uint64_t *full;
    const T *src[PIECES];
    long long r0, step, rows;
    uint32_t rowb;
    int C, S;

    // lane 0: the copies of the i-th row
    __device__ __forceinline__ void issue(int i) const {
        const long long r = r0 + i * step;
        if (r >= rows) return;
        const int s = i % S;
        mbar_arrive_expect_tx(&full[s], PIECES * rowb);
#pragma unroll
        for (int p = 0; p < PIECES; ++p) bulk_load(slots + (size_t)(s * PIECES + p) * rowb, src[p] + r * C, rowb, &full[s]);
    }
    __device__ __forceinline__ const T *row(int i, int p) const {
        return reinterpret_cast<const T *>(slots + (size_t)(i % S * PIECES + p) * rowb);
    }
    // after an abort: copies in flight land before the shared memory goes
    __device__ __forceinline__ void drain(int i) const {
        for (int k = i; k < i + S; ++k)
            if (r0 + k * step < rows) final_wait(&full[k % S], (uint32_t)(k / S) & 1u);
    }
};

// The batch element of a row, for rows that advance by a fixed step.
struct RowGroup {
    int b;
    unsigned n;
    __device__ __forceinline__ RowGroup(long long r, int N) : b((int)(r / N)), n((unsigned)(r % N)) {}
    __device__ __forceinline__ void advance(unsigned step, unsigned N) {
        n += step;
        if (n >= N) b += n / N, n %= N;
    }
};

// Forward, a warp a row of up to 32 EPT channels, one CTA a SM.  The row is held
// in fp32 from its one conversion on (reading it three times from its slot
// took 1336 instructions a row of 2048, which bound the kernel at 4.4 TB/s);
// the vectors stay in registers in bf16, fp32 ones would not fit and come from L1.
constexpr int kFwdThreads = 384;
template <typename T, int EPT>
__global__ void __launch_bounds__(kFwdThreads, 1)
norm_fwd_ring(const T *__restrict__ x, const T *__restrict__ w, const T *__restrict__ b, T *__restrict__ y,
              float *__restrict__ mean_out, float *__restrict__ rstd_out, const NormPlan p, int slots) {
    constexpr int VEC = 16 / sizeof(T), NV = EPT / VEC;
    constexpr bool kHold = sizeof(T) == 2;
    using P = Pack<T, VEC>;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kFwdThreads / 32][kRing];
    __shared__ int abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * (kFwdThreads / 32);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kFwdThreads / 32; ++i)
            for (int s = 0; s < slots; ++s) mbar_init(&full[i][s], 1);
        abort_word = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait_for(x, w, b);
    pdl_trigger();
    RowRing<T, 1> rr;
    rr.rowb = (uint32_t)p.C * sizeof(T);
    rr.slots = ring + (size_t)warp * slots * rr.rowb;
    rr.full = full[warp];
    rr.src[0] = x;
    rr.r0 = (long long)blockIdx.x * (kFwdThreads / 32) + warp;
    rr.step = step, rr.rows = p.rows, rr.C = p.C, rr.S = slots;
    if (lane == 0)
        for (int i = 0; i < slots; ++i) rr.issue(i);
    const float inv = 1.f / (float)p.C;
    RowGroup gr(rr.r0, p.N);
    int held = -1;
    P wk[kHold ? NV : 1], bk[kHold ? NV : 1];
    int i = 0;
    for (long long r = rr.r0; r < p.rows; r += step, ++i) {
        const long long vo = p.per_batch ? (long long)gr.b * p.C : 0;
        if (kHold && held != (p.per_batch ? gr.b : 0)) {
            held = p.per_batch ? gr.b : 0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * 32 + lane) * VEC;
                if (c < p.C) {
                    if (w) wk[k] = load_pack<T, VEC>(w + vo + c);
                    if (b) bk[k] = load_pack<T, VEC>(b + vo + c);
                }
            }
        }
        if (!mbar_poll(&rr.full[i % slots], (uint32_t)(i / slots) & 1u, &abort_word, &g_norm_flag, 2)) {
            if (lane == 0) rr.drain(i);
            return;
        }
        const T *xs = rr.row(i, 0);
        float2 v[EPT / 2], s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * 32 + lane) * VEC;
            if (c < p.C) {
                const P u = load_pack<T, VEC>(xs + c);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    v[(k * VEC + j) / 2] = get2(u, j);
                    s2 = fadd2(s2, v[(k * VEC + j) / 2]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) rr.issue(i + slots);
        const float mean = warp_sum(s2.x + s2.y) * inv;
        s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if ((k * 32 + lane) * VEC < p.C) {
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    float2 &d = v[(k * VEC + j) / 2];
                    d = fadd2(d, make_float2(-mean, -mean));
                    s2 = ffma2(d, d, s2);
                }
            }
        const float rstd = rsqrtf(warp_sum(s2.x + s2.y) * inv + p.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * 32 + lane) * VEC;
            if (c < p.C) {
                P wv, bv, o;
                if (w) wv = kHold ? wk[k] : load_pack<T, VEC>(w + vo + c);
                if (b) bv = kHold ? bk[k] : load_pack<T, VEC>(b + vo + c);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    float2 f = fmul2(v[(k * VEC + j) / 2], make_float2(rstd, rstd));
                    if (w) f = fmul2(f, get2(wv, j));
                    if (b) f = fadd2(f, get2(bv, j));
                    set2(o, j, f);
                }
                *reinterpret_cast<P *>(y + r * p.C + c) = o;
            }
        }
        if (lane == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        gr.advance((unsigned)step, (unsigned)p.N);
    }
}

// Backward, a team of WPR warps a row, 32 channels a lane, one CTA of 16 warps a
// SM.  A lane keeps its channels' sums of dy xh and dy; the row is read from
// its slot twice (for the row's sums, then for dx), which costs less than the
// registers to hold it.  CTA c of a group (a batch element with per_batch,
// else all rows) takes the rows c * teams + team, + splits * teams, ...; its
// teams' sums are added in team order into part[group][split][2][C].
constexpr int kBwdThreads = 512, kLane = 32;
template <typename T, int WPR>
__global__ void __launch_bounds__(kBwdThreads, 1)
norm_bwd_team(const T *__restrict__ dy, const T *__restrict__ x, const T *__restrict__ w,
              const float *__restrict__ mean, const float *__restrict__ rstd, T *__restrict__ dx,
              float *__restrict__ part, const NormPlan p, int splits, int slots) {
    constexpr int VEC = 16 / sizeof(T), NV = kLane / VEC, kTeams = kBwdThreads / 32 / WPR;
    using P = Pack<T, VEC>;
    extern __shared__ __align__(128) uint8_t ring[];     // the rings; at the end [2][C] floats
    __shared__ uint64_t full[kTeams][kRing];
    __shared__ float2 red[2][kBwdThreads / 32];
    __shared__ int abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / WPR, t = threadIdx.x % (32 * WPR);
    const int g = blockIdx.x / splits, sp = blockIdx.x % splits;
    const long long n = p.per_batch ? p.N : p.rows, first = g * n;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kTeams; ++i)
            for (int s = 0; s < slots; ++s) mbar_init(&full[i][s], 1);
        abort_word = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait_for(dy, x, w, mean, rstd);
    pdl_trigger();
    RowRing<T, 2> rr;
    rr.rowb = (uint32_t)p.C * sizeof(T);
    rr.slots = ring + (size_t)team * slots * 2 * rr.rowb;
    rr.full = full[team];
    rr.src[0] = x, rr.src[1] = dy;
    rr.r0 = first + (long long)sp * kTeams + team;
    rr.step = (long long)splits * kTeams, rr.rows = first + n, rr.C = p.C, rr.S = slots;
    if (t == 0)
        for (int i = 0; i < slots; ++i) rr.issue(i);
    const float inv = 1.f / (float)p.C;
    P wk[NV];
    float2 aw[kLane / 2], ab[kLane / 2];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * 32 * WPR + t) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) wk[k].v[j] = from_f<T>(1.f);
        if (w && c < p.C) wk[k] = load_pack<T, VEC>(w + (p.per_batch ? (long long)g * p.C : 0) + c);
    }
#pragma unroll
    for (int e = 0; e < kLane / 2; ++e) aw[e] = ab[e] = make_float2(0.f, 0.f);
    float m1 = rr.r0 < rr.rows ? mean[rr.r0] : 0.f, rs1 = rr.r0 < rr.rows ? rstd[rr.r0] : 0.f;
    int i = 0;
    // (after a wait that gave up the rows go on, without meaning: the team's barriers stay in step)
    for (long long r = rr.r0; r < rr.rows; r += rr.step, ++i) {
        const float rs = rs1, nm = -m1 * rs1;
        if (r + rr.step < rr.rows) m1 = mean[r + rr.step], rs1 = rstd[r + rr.step];
        mbar_poll(&rr.full[i % slots], (uint32_t)(i / slots) & 1u, &abort_word, &g_norm_flag, 3);
        const T *xs = rr.row(i, 0), *ds = rr.row(i, 1);
        float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * 32 * WPR + t) * VEC;
            if (c < p.C) {
                const P xp = load_pack<T, VEC>(xs + c), dp = load_pack<T, VEC>(ds + c);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    const int e = (k * VEC + j) / 2;
                    const float2 xh = ffma2(get2(xp, j), make_float2(rs, rs), make_float2(nm, nm));
                    const float2 d = get2(dp, j);
                    const float2 gi = fmul2(d, get2(wk[k], j));
                    s1 = fadd2(s1, gi);
                    s2 = ffma2(gi, xh, s2);
                    aw[e] = ffma2(d, xh, aw[e]);
                    ab[e] = fadd2(ab[e], d);
                }
            }
        }
        float t1 = warp_sum(s1.x + s1.y), t2 = warp_sum(s2.x + s2.y);
        if constexpr (WPR > 1) {
            if (lane == 0) red[i & 1][warp] = make_float2(t1, t2);
            named_bar_sync(1 + team, 32 * WPR);
            t1 = t2 = 0.f;
#pragma unroll
            for (int q = 0; q < WPR; ++q) {
                const float2 f = red[i & 1][team * WPR + q];
                t1 += f.x, t2 += f.y;
            }
        } else {
            __syncwarp();
        }
        // every warp of the team is past the last row: its slot takes a new one
        if (t == 0 && i > 0 && !abort_word) rr.issue(i - 1 + slots);
        t1 *= inv;
        t2 *= inv;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * 32 * WPR + t) * VEC;
            if (c < p.C) {
                const P xp = load_pack<T, VEC>(xs + c), dp = load_pack<T, VEC>(ds + c);
                P o;
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    const float2 xh = ffma2(get2(xp, j), make_float2(rs, rs), make_float2(nm, nm));
                    const float2 gi = ffma2(get2(dp, j), get2(wk[k], j), make_float2(-t1, -t1));
                    const float2 f = fmul2(ffma2(xh, make_float2(-t2, -t2), gi), make_float2(rs, rs));
                    set2(o, j, f);
                }
                *reinterpret_cast<P *>(dx + r * p.C + c) = o;
            }
        }
    }
    if (abort_word && t == 0)
        for (int k = 0; k < slots; ++k) final_wait(&rr.full[k], 0), final_wait(&rr.full[k], 1);
    __syncthreads();
    if (abort_word || !part) return;
    float *sum = reinterpret_cast<float *>(ring);
    for (int q = 0; q < kTeams; ++q) {
        if (team == q) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * 32 * WPR + t) * VEC;
                if (c < p.C) {
#pragma unroll
                    for (int j = 0; j < VEC; j += 4) {
                        const int e = (k * VEC + j) / 2;
                        float4 *sw = reinterpret_cast<float4 *>(sum + c + j), *sb = reinterpret_cast<float4 *>(sum + p.C + c + j);
                        float4 u = make_float4(aw[e].x, aw[e].y, aw[e + 1].x, aw[e + 1].y), v = make_float4(ab[e].x, ab[e].y, ab[e + 1].x, ab[e + 1].y);
                        if (q) {
                            const float4 a = *sw, b = *sb;
                            u.x += a.x, u.y += a.y, u.z += a.z, u.w += a.w;
                            v.x += b.x, v.y += b.y, v.z += b.z, v.w += b.w;
                        }
                        *sw = u;
                        *sb = v;
                    }
                }
            }
        }
        __syncthreads();
    }
    float *o = part + ((long long)g * splits + sp) * 2 * p.C;
    for (int e = threadIdx.x; e < 2 * p.C; e += kBwdThreads) o[e] = sum[e];
}

// Forward, one row on WPR warps, EPT elements a thread.  The variance is the
// mean square of the deviations (a second pass over the registers).
template <typename T, int VEC, int EPT, int WPR>
__global__ void __launch_bounds__(kThreads)
norm_fwd(const T *__restrict__ x, const T *__restrict__ w, const T *__restrict__ b, T *__restrict__ y,
         float *__restrict__ mean_out, float *__restrict__ rstd_out, const NormPlan p) {
    pdl_wait_for(x, w, b);
    pdl_trigger();
    constexpr int TPR = 32 * WPR, RPC = kThreads / TPR, NV = EPT / VEC;
    __shared__ float red[2][kThreads / 32];
    const int t = threadIdx.x % TPR, warp = threadIdx.x >> 5;
    const long long r = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
    const bool ok = r < p.rows;
    const T *xr = x + (ok ? r : 0) * p.C;
    Pack<T, VEC> v[NV];   // as loaded: a bf16 row takes half the registers, so twice the rows are in flight
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC;
        v[i] = load_pack<T, VEC>(xr + (c < p.C ? c : 0));      // (loads under no branch: all in flight at once)
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * TPR + t) * VEC >= p.C) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i].v[j] = from_f<T>(0.f);
        }
    auto row_sum = [&](float s, int which) {
        s = warp_sum(s);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 31) == 0) red[which][warp] = s;
            __syncthreads();
            s = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) s += red[which][warp / WPR * WPR + i];
        }
        return s;
    };
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) s += to_f(v[i / VEC].v[i % VEC]);
    const float mean = row_sum(s, 0) / (float)p.C;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = to_f(v[i].v[j]) - mean;
            s += (i * TPR + t) * VEC < p.C ? d * d : 0.f;
        }
    const float rstd = rsqrtf(row_sum(s, 1) / (float)p.C + p.eps);
    const long long vo = p.per_batch ? (ok ? r : 0) / p.N * p.C : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC, cc = c < p.C ? c : 0;
        Pack<T, VEC> wk, bk, o;
        if (w) wk = load_pack<T, VEC>(w + vo + cc);
        if (b) bk = load_pack<T, VEC>(b + vo + cc);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float f = (to_f(v[i].v[j]) - mean) * rstd;
            if (w) f *= to_f(wk.v[j]);
            if (b) f += to_f(bk.v[j]);
            o.v[j] = from_f<T>(f);
        }
        if (ok && c < p.C) *reinterpret_cast<Pack<T, VEC> *>(y + r * p.C + c) = o;
    }
    if (!ok) return;
    if (t == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
    }
}

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

// Forward of rows too wide for the registers: one CTA a row, read three times
// (the second and third time from L1 or L2).
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_fwd_wide(const T *__restrict__ x, const T *__restrict__ w, const T *__restrict__ b, T *__restrict__ y,
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

// Backward of rows that are not whole 16 bytes, in one pass: a CTA of TPR x TY
// threads walks the rows of its range, TY at a time, kEpt channels a thread,
// the next rows loaded before the current ones are reduced; the channels' sums
// stay in registers and leave as one piece, part[group][split][2][C].
template <typename T, int kEpt, int MAXT>
__global__ void __launch_bounds__(MAXT, kEpt == 4 ? 2 : 1)
norm_bwd(const T *__restrict__ dy, const T *__restrict__ x, const T *__restrict__ w, const float *__restrict__ mean,
         const float *__restrict__ rstd, T *__restrict__ dx, float *__restrict__ part, const NormPlan p, int tpr,
         int splits) {
    pdl_wait_for(dy, x, w, mean, rstd);
    pdl_trigger();
    constexpr int VEC = 1, NV = kEpt;
    extern __shared__ float sh[];          // [2][2][warps], then (at the end) [threads][2 kEpt]
    const int warps = blockDim.x >> 5, wpr = tpr >> 5, ty = blockDim.x / tpr;
    const int t = threadIdx.x % tpr, yy = threadIdx.x / tpr, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x / splits, sp = blockIdx.x % splits;
    const long long rows = p.per_batch ? p.N : p.rows;
    const long long r0 = g * rows + rows * sp / splits, r1 = g * rows + rows * (sp + 1) / splits;
    const float inv = 1.f / (float)p.C;
    float wv[kEpt], aw[kEpt] = {}, ab[kEpt] = {};
    Pack<T, VEC> xp[NV], dp[NV];
    float m = 0.f, rs = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        Pack<T, VEC> k;
        if (w && c < p.C) k = load_pack<T, VEC>(w + (p.per_batch ? (long long)g * p.C : 0) + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) wv[i * VEC + j] = c < p.C ? (w ? to_f(k.v[j]) : 1.f) : 0.f;
    }
    auto fetch = [&](long long r) {
        const bool ok = r < r1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            const long long at = (ok ? r : r0) * p.C + (c < p.C ? c : 0);      // (under no branch: all in flight at once)
            xp[i] = load_pack<T, VEC>(x + at);
            dp[i] = load_pack<T, VEC>(dy + at);
        }
        m = mean[ok ? r : r0];
        rs = rstd[ok ? r : r0];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (!ok || (i * tpr + t) * VEC >= p.C) xp[i].v[0] = dp[i].v[0] = from_f<T>(0.f);
        if (!ok) m = rs = 0.f;
    };
    fetch(r0 + yy);
    int par = 0;
    for (long long r = r0 + yy; r - yy < r1; r += ty, par ^= 1) {
        float xh[kEpt], d[kEpt];
        const float rsc = rs;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < kEpt; ++i) {
            xh[i] = (to_f(xp[i / VEC].v[i % VEC]) - m) * rs;
            d[i] = to_f(dp[i / VEC].v[i % VEC]);
            const float gi = d[i] * wv[i];
            s1 += gi;
            s2 += gi * xh[i];
            aw[i] += d[i] * xh[i];
            ab[i] += d[i];
        }
        fetch(r + ty);
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (wpr > 1) {
            float *red = sh + par * 2 * warps;
            if (lane == 0) red[warp] = s1, red[warps + warp] = s2;
            __syncthreads();
            s1 = s2 = 0.f;
            for (int i = 0; i < wpr; ++i) s1 += red[yy * wpr + i], s2 += red[warps + yy * wpr + i];
        }
        s1 *= inv;
        s2 *= inv;
        if (r < r1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + t) * VEC;
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    o.v[j] = from_f<T>(rsc * (d[e] * wv[e] - s1 - xh[e] * s2));
                }
                if (c < p.C) *reinterpret_cast<Pack<T, VEC> *>(dx + r * p.C + c) = o;
            }
        }
    }
    if (!part) return;
    float *o = part + ((long long)g * splits + sp) * 2 * p.C;
    if (ty == 1) {
#pragma unroll
        for (int i = 0; i < kEpt; ++i) {
            const int c = (i / VEC * tpr + t) * VEC + i % VEC;
            if (c < p.C) o[c] = aw[i], o[p.C + c] = ab[i];
        }
        return;
    }
    // the TY rows' sums, added in row order
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEpt; ++i) sh[i * blockDim.x + threadIdx.x] = aw[i], sh[(kEpt + i) * blockDim.x + threadIdx.x] = ab[i];
    __syncthreads();
    if (yy) return;
#pragma unroll
    for (int i = 0; i < kEpt; ++i) {
        const int c = (i / VEC * tpr + t) * VEC + i % VEC;
        float a = 0.f, bsum = 0.f;
        for (int k = 0; k < ty; ++k) a += sh[i * blockDim.x + k * tpr + t], bsum += sh[(kEpt + i) * blockDim.x + k * tpr + t];
        if (c < p.C) o[c] = a, o[p.C + c] = bsum;
    }
}

// Backward of rows wider than norm_bwd takes: dx a CTA a row, the channels'
// sums in a second pass, one thread a channel.
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_dx_wide(const T *__restrict__ dy, const T *__restrict__ x, const T *__restrict__ w,
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

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_dw_wide(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
             const float *__restrict__ rstd, float *__restrict__ part, const NormPlan p, int splits) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    const int g = blockIdx.y / splits, sp = blockIdx.y % splits;
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

// out[group][e] = sum over splits of part[group][split][e], e < width: 32
// columns a CTA, its 32 warps taking every 32nd split, then the warps' sums in
// warp order.  Columns below `cut` go to out0, the rest to out1.
constexpr int kSumWarps = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kSumWarps)
split_sum(const float *__restrict__ part, T *__restrict__ out0, T *__restrict__ out1, long long width, long long cut,
          int splits) {
    pdl_wait_for(part);
    pdl_trigger();
    __shared__ float red[kSumWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long e = (long long)blockIdx.x * 32 + lane, g = blockIdx.y;
    float a = 0.f;
    if (e < width) {
        const float *src = part + g * splits * width + e;
#pragma unroll 8
        for (int s = warp; s < splits; s += kSumWarps) a += src[s * width];
    }
    red[warp][lane] = a;
    __syncthreads();
    if (warp || e >= width) return;
    a = 0.f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) a += red[i][lane];
    T *o = e < cut ? out0 : out1;
    if (o) o[e < cut ? g * cut + e : g * (width - cut) + e - cut] = from_f<T>(a);
}

// ---------------------------------------------------------------- host

constexpr int kWarpRow = 2048;           // widest row of norm_fwd_ring
constexpr int kRingBytes = 200 << 10;    // the rings of a SM

constexpr int kWideBwd = 512 * 16;       // widest row of norm_bwd
constexpr int kWideFwd = 256 * 64;       // widest row of norm_fwd

// How the backward pass runs, and the row ranges of a group (a batch element
// with per_batch, else all rows): as many CTAs as stay resident.
struct BwdShape {
    int wpr, slots;              // norm_bwd_team: warps a row (0: another form), slots a team
    int ept, tpr, threads;       // norm_bwd
    int splits;
};
BwdShape bwd_shape(const NormPlan &p, int esize) {
    BwdShape b{};
    const long long rows = p.per_batch ? p.N : p.rows, groups = p.per_batch ? p.B : 1;
    if (p.C * (long long)esize % 16 == 0 && p.C <= kWideBwd) {
        // warps for 32 channels a lane, and two slots a team at least
        const int pair = 2 * p.C * esize, warps = kBwdThreads / 32;
        for (b.wpr = 1; 32 * kLane * b.wpr < p.C || warps / b.wpr * 2 * pair > kRingBytes; b.wpr *= 2) {}
        b.slots = kRingBytes / (warps / b.wpr * pair);
        if (b.slots > kRing) b.slots = kRing;
        long long s = kSmCount / groups;
        const int teams = warps / b.wpr;
        if (s > (rows + 2 * teams - 1) / (2 * teams)) s = (rows + 2 * teams - 1) / (2 * teams);
        b.splits = (int)(s < 1 ? 1 : s);
        return b;
    }
    b.ept = p.C <= 2048 ? 4 : (p.C <= 4096 ? 8 : 16);
    b.tpr = ((p.C + b.ept - 1) / b.ept + 31) / 32 * 32;
    if (b.tpr > 512) b.tpr = 256;
    b.threads = b.tpr >= 256 ? b.tpr : 256 / b.tpr * b.tpr;
    const int resident = b.ept == 4 ? 1024 / b.threads : 1;
    long long s = (long long)resident * kSmCount / groups;
    if (s > (rows + 7) / 8) s = (rows + 7) / 8;
    b.splits = (int)(s < 1 ? 1 : s);
    return b;
}

template <typename T> bool g_norm_ready[128] = {};
template <typename T> bool norm_setup() {
    return set_smem((const void *)norm_bwd_team<T, 1>, kRingBytes) && set_smem((const void *)norm_bwd_team<T, 2>, kRingBytes) &&
           set_smem((const void *)norm_bwd_team<T, 4>, kRingBytes) && set_smem((const void *)norm_bwd_team<T, 8>, kRingBytes) &&
           set_smem((const void *)norm_bwd_team<T, 16>, kRingBytes) && set_smem((const void *)norm_fwd_ring<T, 32>, kRingBytes) &&
           set_smem((const void *)norm_fwd_ring<T, 64>, kRingBytes);
}

template <typename T, int VEC, int EPT, int WPR>
int fwd_launch(const T *x, const T *w, const T *b, T *y, float *mean, float *rstd, const NormPlan &p, cudaStream_t s) {
    constexpr int RPC = kThreads / (32 * WPR);
    const long long grid = (p.rows + RPC - 1) / RPC;
    if (grid > 0x7fffffffLL) return -1;
    return launch_dep(norm_fwd<T, VEC, EPT, WPR>, dim3((unsigned)grid), kThreads, 0, s, x, w, b, y, mean, rstd, p) ? 1 : -1;
}

template <typename T, int VEC>
int fwd_pick(const T *x, const T *w, const T *b, T *y, float *mean, float *rstd, const NormPlan &p, cudaStream_t s) {
    if constexpr (VEC == 1) {
        // element loads: few a thread (32 a thread took 155 registers and left one CTA on a SM: 24 us for 3510 rows
        // of 1001 fp32)
        if (p.C <= 256) return fwd_launch<T, 1, 8, 1>(x, w, b, y, mean, rstd, p, s);
        if (p.C <= 512) return fwd_launch<T, 1, 8, 2>(x, w, b, y, mean, rstd, p, s);
        if (p.C <= 1024) return fwd_launch<T, 1, 8, 4>(x, w, b, y, mean, rstd, p, s);
        if (p.C <= 2048) return fwd_launch<T, 1, 8, 8>(x, w, b, y, mean, rstd, p, s);
        if (p.C <= 4096) return fwd_launch<T, 1, 16, 8>(x, w, b, y, mean, rstd, p, s);
        if (p.C <= 8192) return fwd_launch<T, 1, 32, 8>(x, w, b, y, mean, rstd, p, s);
        return fwd_launch<T, 1, 64, 8>(x, w, b, y, mean, rstd, p, s);
    }
    if (p.C <= 256) return fwd_launch<T, VEC, 8, 1>(x, w, b, y, mean, rstd, p, s);
    if (p.C <= 512) return fwd_launch<T, VEC, 16, 1>(x, w, b, y, mean, rstd, p, s);
    if (p.C <= 1024) return fwd_launch<T, VEC, 32, 1>(x, w, b, y, mean, rstd, p, s);
    if (p.C <= 2048) return fwd_launch<T, VEC, 64, 1>(x, w, b, y, mean, rstd, p, s);
    if (p.C <= 4096) return fwd_launch<T, VEC, 64, 2>(x, w, b, y, mean, rstd, p, s);
    if (p.C <= 8192) return fwd_launch<T, VEC, 64, 4>(x, w, b, y, mean, rstd, p, s);
    return fwd_launch<T, VEC, 64, 8>(x, w, b, y, mean, rstd, p, s);
}

template <typename T>
int norm_fwd_t(const T *x, const T *w, const T *b, T *y, float *mean, float *rstd, const NormPlan &p, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    // (from 4 rows a warp on; fewer, or narrower ones, are as fast without a ring)
    constexpr int kWarps = kFwdThreads / 32;
    if (p.C % V == 0 && p.C > 512 && p.C <= kWarpRow && p.rows >= 4LL * kWarps * kSmCount) {
        const int row = p.C * (int)sizeof(T);
        int slots = kRingBytes / (kWarps * row);
        if (slots > kRing) slots = kRing;
        if (!once_per_device(&g_norm_ready<T>, norm_setup<T>)) return -1;
        auto f = p.C <= 1024 ? norm_fwd_ring<T, 32> : norm_fwd_ring<T, 64>;
        return launch_dep(f, dim3(kSmCount), kFwdThreads, kWarps * slots * row, s, x, w, b, y, mean, rstd, p, slots) ? 1 : -1;
    }
    // few rows: all warps of a CTA on each, for the latency of one (2 rows of 2048: 9.3 us with a warp a row)
    if (p.C % V == 0 && p.C > 256 && p.C <= 2048 && p.rows <= 2 * kSmCount) return fwd_launch<T, V, 8, 8>(x, w, b, y, mean, rstd, p, s);
    if (p.C <= kWideFwd)
        return p.C % V == 0 ? fwd_pick<T, V>(x, w, b, y, mean, rstd, p, s) : fwd_pick<T, 1>(x, w, b, y, mean, rstd, p, s);
    const long long grid = p.rows < (1 << 30) ? p.rows : (1 << 30);
    norm_fwd_wide<T><<<(unsigned)grid, kThreads, 0, s>>>(x, w, b, y, mean, rstd, p);
    return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

template <typename T>
int norm_bwd_t(const T *dy, const T *x, const T *w, const float *mean, const float *rstd, T *dx, T *dw, T *db,
               float *part, const NormPlan &p, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const BwdShape b = bwd_shape(p, sizeof(T));
    const int groups = p.per_batch ? p.B : 1;
    if (!dw && !db) part = nullptr;
    const unsigned grid = (unsigned)(groups * b.splits);
    if (b.wpr) {
        const int rings = b.slots * (kBwdThreads / 32 / b.wpr) * 2 * p.C * (int)sizeof(T), sums = 2 * p.C * 4;
        if (!once_per_device(&g_norm_ready<T>, norm_setup<T>)) return -1;
        auto f = b.wpr == 1   ? norm_bwd_team<T, 1>
                 : b.wpr == 2 ? norm_bwd_team<T, 2>
                 : b.wpr == 4 ? norm_bwd_team<T, 4>
                 : b.wpr == 8 ? norm_bwd_team<T, 8>
                              : norm_bwd_team<T, 16>;
        if (!launch_dep(f, dim3(grid), kBwdThreads, rings > sums ? rings : sums, s, dy, x, w, mean, rstd, dx, part, p, b.splits, b.slots))
            return -1;
    } else if (p.C <= kWideBwd) {
        // the CTA's pieces at the end, or two rounds of two sums a warp
        const int smem = b.threads > b.tpr ? b.threads * 2 * b.ept * 4 : b.threads / 32 * 16;
        auto f = b.ept == 16 ? norm_bwd<T, 16, 512> : (b.ept == 8 ? norm_bwd<T, 8, 512> : norm_bwd<T, 4, 512>);
        if (!launch_dep(f, dim3(grid), b.threads, smem, s, dy, x, w, mean, rstd, dx, part, p, b.tpr, b.splits)) return -1;
    } else {
        const long long grid = p.rows < (1 << 30) ? p.rows : (1 << 30);
        norm_dx_wide<T><<<(unsigned)grid, kThreads, 0, s>>>(dy, x, w, mean, rstd, dx, p);
        if (cudaGetLastError() != cudaSuccess) return -1;
        if (part)
            norm_dw_wide<T><<<dim3((unsigned)((p.C + kThreads - 1) / kThreads), (unsigned)(groups * b.splits)), kThreads,
                              0, s>>>(dy, x, mean, rstd, part, p, b.splits);
        if (cudaGetLastError() != cudaSuccess) return -1;
    }
    if (!part) return 1;
    return launch_dep(split_sum<T>, dim3((unsigned)((2 * (long long)p.C + 31) / 32), groups), 32 * kSumWarps, 0, s, part, dw, db,
                      2 * (long long)p.C, (long long)p.C, b.splits) ? 2 : -1;
}

}  // namespace

size_t norm_bwd_ws(const NormPlan &p) {
    const int a = bwd_shape(p, 2).splits, b = bwd_shape(p, 4).splits;      // whichever type the call has
    return align256(size_t(p.per_batch ? p.B : 1) * (a > b ? a : b) * 2 * p.C * sizeof(float));
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

int launch_split_sum(int is_bf16, const float *part, void *out, long long width, int splits, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const dim3 grid((unsigned)((width + 31) / 32));
    const bool ok = is_bf16 ? launch_dep(split_sum<bf>, grid, 32 * kSumWarps, 0, s, part, (bf *)out, (bf *)nullptr, width, width, splits)
                            : launch_dep(split_sum<float>, grid, 32 * kSumWarps, 0, s, part, (float *)out, (float *)nullptr, width, width, splits);
    return ok ? 1 : -1;
}

int read_and_clear_norm_flag(unsigned *flag_out) {
    if (cudaMemcpyFromSymbol(flag_out, g_norm_flag, sizeof(unsigned)) != cudaSuccess) return -1;
    const unsigned zero = 0;
    if (*flag_out && cudaMemcpyToSymbol(g_norm_flag, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return 0;
}

}  // namespace la
