// k_linear_tc.cu -- bf16 matrix products with a fused epilogue on the tensor
// cores (tcgen05, accumulators in TMEM, operands by TMA).
//
//   C[m][n] = sum_k A(m, k) B(n, k);  z = C + bias;  pre = z;  y = act(z) + residual
//
// One CTA a SM, persistent over output tiles: 256 x 256 or 256 x 128 on a pair
// of CTAs (cta_group::2, each holding 128 rows of A and half of B's, so that a
// stage's copies and the MMA's reads stay within a SM's 128 bytes of shared
// memory a clock: a 128 x 256 tile on one CTA needs 192, and ran at 66%), or
// 128 x 128 and 128 x 64 on one CTA for small outputs.  Warp 0 fills a ring of K = 64 stages by TMA, warp 1 issues the MMAs, warps
// 2-5 run the epilogue of one tile while the MMAs of the next fill the other
// half of TMEM.  Either operand may be stored with its k index contiguous
// (K-major boxes of 64 x rows) or with its row index contiguous (MN-major
// boxes of 64 rows x 64 k): the three products of a linear layer need no
// transposed copies.  The residual arrives and the outputs leave by TMA
// through per-warp buffers of 32 x 32.
#include <cudaTypedefs.h>
#include <mutex>

#include "la_sm100_dit.cuh"

namespace la {

using namespace sm100;

namespace {

// Raised by a bounded wait that gave up; read by la_device_status.
__device__ unsigned int g_linear_flag = 0;

constexpr int kBM = 128, kBK = 64;
constexpr int kThreads = 192;
constexpr int kChunk = 32;                        // output columns an epilogue step
constexpr int kBuf = 32 * kChunk * 2;             // one warp's 32 x 32 bf16 buffer

// CG CTAs share a tile of CG * 128 x BN: each holds its 128 rows of A and BN / CG of B's.
template <int BN, int CG>
struct Cfg {
    static constexpr int kBRows = BN / CG;
    static constexpr int kA = kBM * kBK * 2, kB = kBRows * kBK * 2, kStage = kA + kB;
    static constexpr int kStages = kBRows == 256 ? 4 : (kBRows == 128 ? 6 : 8);
    static constexpr int kStg = kStages * kStage;            // 4 warps x (2 y + 2 pre) buffers
    static constexpr int kBar = kStg + 4 * 4 * kBuf;
    static constexpr int kBars = 2 * kStages + 4 + 8;
    static constexpr int kSmem = kBar + kBars * 8 + 16 + 1024;
    static constexpr uint32_t kTmem = 2 * BN;
    static_assert(kSmem <= 232448, "227 KiB of shared memory");
};

struct TcArgs {
    long long M, N;
    int kiters;              // K in stages of 64
    int mt, nt, splits, kper;
    int a_mn, b_mn;
    const __nv_bfloat16 *bias, *res;
    __nv_bfloat16 *pre, *y;
    float *part;             // splits > 1: fp32 [splits][M][ldp]
    long long ldp;
    int act;
    int direct;              // rows of y are not whole 16 bytes: no TMA on y, pre, res
};

// Byte offset of 16-byte chunk j of row r in a 32-row buffer of 64-byte rows, 64-byte swizzle.
__device__ __forceinline__ int sw64(int r, int j) { return r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }

// A warp's 32 x 32 block of a row-major matrix whose rows TMA cannot address, into or out of its buffer.
__device__ __forceinline__ void block_in(uint8_t *buf, const __nv_bfloat16 *src, long long row0, long long col0,
                                         const TcArgs &a, int lane) {
    for (int r = 0; r < 32; ++r)
        if (row0 + r < a.M && col0 + lane < a.N)
            *reinterpret_cast<__nv_bfloat16 *>(buf + sw64(r, lane >> 3) + (lane & 7) * 2) =
                src[(row0 + r) * a.N + col0 + lane];
}
__device__ __forceinline__ void block_out(const uint8_t *buf, __nv_bfloat16 *dst, long long row0, long long col0,
                                          const TcArgs &a, int lane) {
    for (int r = 0; r < 32; ++r)
        if (row0 + r < a.M && col0 + lane < a.N)
            dst[(row0 + r) * a.N + col0 + lane] =
                *reinterpret_cast<const __nv_bfloat16 *>(buf + sw64(r, lane >> 3) + (lane & 7) * 2);
}

template <int BN, int CG>
__global__ void __launch_bounds__(kThreads, 1)
gemm_tc(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
        const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_pre,
        const __grid_constant__ CUtensorMap tm_res, const TcArgs a) {
    using C = Cfg<BN, CG>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBar), *empty = full + C::kStages;
    uint64_t *acc_full = empty + C::kStages, *acc_empty = acc_full + 2, *rbar = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rbar + 8);
    volatile int *abort_word = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long works = (long long)a.mt * a.nt * a.splits;
    const int rank = CG == 2 ? (int)cluster_ctarank() : 0;         // the even CTA of a pair leads
    const int first = blockIdx.x / CG, step = gridDim.x / CG;      // this CTA's (pair's) tiles

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
        for (int s = 0; s < 2; ++s) mbar_init(&acc_full[s], 1), mbar_init(&acc_empty[s], 128 * CG);
        for (int s = 0; s < 8; ++s) mbar_init(&rbar[s], 1);
        *abort_word = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(tmem_slot, C::kTmem);
        } else {
            tmem_alloc(tmem_slot, C::kTmem);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();   // the pair's barriers are set up
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int issued = 0;   // stages filled (warp 0 lane 0) or read (warp 1 lane 0)
    int tiles = 0;    // tiles accumulated (warp 1 lane 0)

    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
        for (long long w = first; w < works; w += step) {
            const int tile = (int)(w % ((long long)a.mt * a.nt)), sp = (int)(w / ((long long)a.mt * a.nt));
            const int m0 = (tile / a.nt * CG + rank) * kBM, n0 = tile % a.nt * BN + rank * C::kBRows;
            const int k1 = (sp + 1) * a.kper < a.kiters ? (sp + 1) * a.kper : a.kiters;
            bool ok = true;
            for (int k = sp * a.kper; k < k1; ++k, ++issued) {
                const int s = issued % C::kStages;
                const uint32_t ph = (uint32_t)(issued / C::kStages) & 1u;
                if (!(ok = mbar_wait(&empty[s], ph ^ 1u, abort_word, &g_linear_flag, 1))) break;
                uint8_t *sa = smem + s * C::kStage, *sb = sa + C::kA;
                // the leader's barrier counts both CTAs' copies
                if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * C::kStage);
                auto load = [&](void *dst, const CUtensorMap *m, int c0, int c1) {
                    if constexpr (CG == 2) tma_load_2d_pair(dst, m, &full[s], c0, c1);
                    else tma_load_2d(dst, m, &full[s], c0, c1);
                };
                if (a.a_mn) {
                    load(sa, &tm_a, m0, k * kBK);
                    load(sa + 8192, &tm_a, m0 + 64, k * kBK);
                } else {
                    load(sa, &tm_a, k * kBK, m0);
                }
                if (a.b_mn) {
#pragma unroll
                    for (int j = 0; j < C::kBRows / 64; ++j) load(sb + j * 8192, &tm_b, n0 + j * 64, k * kBK);
                } else {
                    load(sb, &tm_b, k * kBK, n0);
                }
            }
            if (!ok) break;
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        const uint32_t id = idesc_bf16(CG * kBM, BN, a.a_mn, a.b_mn);
        // one MMA's 16 k: 32 bytes along a K-major row, two 8-k groups of 1024 bytes MN-major
        const uint32_t astep = a.a_mn ? 2048 : 32, bstep = a.b_mn ? 2048 : 32;
        bool ok = true;
        for (long long w = first; ok && w < works; w += step, ++tiles) {
            const int sp = (int)(w / ((long long)a.mt * a.nt));
            const int k0 = sp * a.kper, k1 = k0 + a.kper < a.kiters ? k0 + a.kper : a.kiters;
            const int buf = tiles & 1;
            if (!(ok = mbar_wait(&acc_empty[buf], ((uint32_t)(tiles >> 1) & 1u) ^ 1u, abort_word, &g_linear_flag, 2)))
                break;
            tc_fence_after();
            for (int k = k0; k < k1; ++k, ++issued) {
                const int s = issued % C::kStages;
                if (!(ok = mbar_wait(&full[s], (uint32_t)(issued / C::kStages) & 1u, abort_word, &g_linear_flag, 3)))
                    break;
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * C::kStage), sb = sa + C::kA;
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                {
                    const uint64_t da = smem_desc(sa + kk * astep, a.a_mn ? 8192 : 16, 1024, kLayoutSw128);
                    const uint64_t db = smem_desc(sb + kk * bstep, a.b_mn ? 8192 : 16, 1024, kLayoutSw128);
                    const uint32_t acc = k > k0 || kk > 0 ? 1u : 0u;
                    if constexpr (CG == 2) mma_bf16_pair(tmem + buf * BN, da, db, id, acc);
                    else mma_bf16(tmem + buf * BN, da, db, id, acc);
                }
                if constexpr (CG == 2) mma_commit_pair(&empty[s]);
                else mma_commit(&empty[s]);
            }
            if (ok) {
                if constexpr (CG == 2) mma_commit_pair(&acc_full[buf]);
                else mma_commit(&acc_full[buf]);
            }
        }
    } else if (warp >= 2) {
        const int q = warp & 3;                                 // this warp's quarter of the TMEM lanes
        uint8_t *ybuf = smem + C::kStg + (warp - 2) * 4 * kBuf, *pbuf = ybuf + 2 * kBuf;
        uint64_t *rb = rbar + (warp - 2) * 2;
        uint32_t rphase = 0;                                    // bit i: the next phase of rb[i]
        uint32_t cc = 0;                                        // chunks so far: buffer cc & 1
        const bool staged = a.splits == 1, tma = staged && !a.direct;
        int t = 0;
        for (long long w = first; w < works; w += step, ++t) {
            const int tile = (int)(w % ((long long)a.mt * a.nt)), sp = (int)(w / ((long long)a.mt * a.nt));
            const long long row0 = ((long long)(tile / a.nt) * CG + rank) * kBM + q * 32, n0 = (long long)(tile % a.nt) * BN;
            const long long left = a.N - n0;
            const int chunks = row0 >= a.M ? 0 : (int)(left >= BN ? BN / kChunk : (left + kChunk - 1) / kChunk);
            if (tma && a.res && chunks > 0 && lane == 0) {
                bulk_wait_read<0>();                            // the buffer's last store has been read out
                mbar_arrive_expect_tx(&rb[cc & 1], kBuf);
                tma_load_2d(ybuf + (cc & 1) * kBuf, &tm_res, &rb[cc & 1], (int)n0, (int)row0);
            }
            const int buf = t & 1;
            if (!mbar_wait(&acc_full[buf], (uint32_t)(t >> 1) & 1u, abort_word, &g_linear_flag, 4)) break;
            tc_fence_after();
            __syncwarp();
            bool ok = true;
            for (int c = 0; c < chunks; ++c, ++cc) {
                const int par = cc & 1;
                const long long col = n0 + c * kChunk;
                float v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + buf * BN + c * kChunk, v);
                uint8_t *yb = ybuf + par * kBuf, *pb = pbuf + par * kBuf;
                if (tma && lane == 0) {
                    if (a.res) {
                        bulk_wait_read<0>();
                        if (c + 1 < chunks) {
                            mbar_arrive_expect_tx(&rb[par ^ 1], kBuf);
                            tma_load_2d(ybuf + (par ^ 1) * kBuf, &tm_res, &rb[par ^ 1], (int)(col + kChunk), (int)row0);
                        }
                    } else {
                        bulk_wait_read<1>();
                    }
                }
                tmem_wait_ld();
                __syncwarp();
                if (!staged) {
                    if (row0 + lane < a.M) {
                        float *o = a.part + ((long long)sp * a.M + row0 + lane) * a.ldp + col;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (col + 4 * j < a.ldp)
                                reinterpret_cast<float4 *>(o)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                    continue;
                }
                if (a.bias) {
                    if (!a.direct) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (col + 8 * j >= a.N) break;
                            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(a.bias + col) + j);
                            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[8 * j + 2 * i] += bf_lo(bw[i]), v[8 * j + 2 * i + 1] += bf_hi(bw[i]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < a.N) v[j] += __bfloat162float(a.bias[col + j]);
                    }
                }
                if (a.pre) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(pb + sw64(lane, j)) =
                            make_uint4(pack_bf2(v[8 * j], v[8 * j + 1]), pack_bf2(v[8 * j + 2], v[8 * j + 3]),
                                       pack_bf2(v[8 * j + 4], v[8 * j + 5]), pack_bf2(v[8 * j + 6], v[8 * j + 7]));
                }
                if (a.act) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = act_f(v[j], a.act);
                }
                if (a.res) {
                    if (tma) {
                        if (!(ok = mbar_wait(&rb[par], (rphase >> par) & 1u, abort_word, &g_linear_flag, 5))) break;
                        rphase ^= 1u << par;
                        __syncwarp();
                    } else {
                        block_in(yb, a.res, row0, col, a, lane);
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 r = *reinterpret_cast<const uint4 *>(yb + sw64(lane, j));
                        const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[8 * j + 2 * i] += bf_lo(rw[i]), v[8 * j + 2 * i + 1] += bf_hi(rw[i]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4 *>(yb + sw64(lane, j)) =
                        make_uint4(pack_bf2(v[8 * j], v[8 * j + 1]), pack_bf2(v[8 * j + 2], v[8 * j + 3]),
                                   pack_bf2(v[8 * j + 4], v[8 * j + 5]), pack_bf2(v[8 * j + 6], v[8 * j + 7]));
                if (tma) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tm_y, yb, (int)col, (int)row0);
                        if (a.pre) tma_store_2d(&tm_pre, pb, (int)col, (int)row0);
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    block_out(yb, a.y, row0, col, a, lane);
                    if (a.pre) block_out(pb, a.pre, row0, col, a, lane);
                    __syncwarp();
                }
            }
            if (!ok) break;
            tc_fence_before();
            if constexpr (CG == 2) mbar_arrive_leader(&acc_empty[buf]);
            else mbar_arrive(&acc_empty[buf]);
        }
        if (tma && lane == 0) bulk_wait_all();
    }
    // after an abort: let copies and MMAs in flight finish before shared memory and TMEM go (a pair's
    // copies count on the leader, whose stage is freed on both sides by the MMAs)
    if (*abort_word) {
        if (warp == 0 && lane == 0 && rank == 0)
            for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
                final_wait(&full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u);
        if (warp == 1 && lane == 0 && issued > 0)
            final_wait(&empty[(issued - 1) % C::kStages], (uint32_t)((issued - 1) / C::kStages) & 1u);
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if constexpr (CG == 2) {
        cluster_sync();   // the peer's arrivals and copies that reach this CTA are over
        if (warp == 1) tmem_dealloc_pair(tmem, C::kTmem);
    } else {
        if (warp == 1) tmem_dealloc(tmem, C::kTmem);
    }
}

// y, pre from the splits' sums, in split order
__global__ void __launch_bounds__(256)
gemm_finish(const TcArgs a) {
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < a.M * a.N; e += (long long)gridDim.x * 256) {
        const long long m = e / a.N, n = e - m * a.N;
        float z = 0.f;
        for (int s = 0; s < a.splits; ++s) z += a.part[((long long)s * a.M + m) * a.ldp + n];
        if (a.bias) z += __bfloat162float(a.bias[n]);
        if (a.pre) a.pre[e] = __float2bfloat16_rn(z);
        z = act_f(z, a.act);
        if (a.res) z += __bfloat162float(a.res[e]);
        a.y[e] = __float2bfloat16_rn(z);
    }
}

// Rows of `cols` elements at any pitch, copied to rows of ldo (a multiple of 8) elements.
__global__ void __launch_bounds__(256)
repack(const __nv_bfloat16 *__restrict__ x, __nv_bfloat16 *__restrict__ o, long long rows, long long cols,
       long long ldo) {
    for (long long r = blockIdx.x; r < rows; r += gridDim.x)
        for (long long c = threadIdx.x; c < cols; c += 256) o[r * ldo + c] = x[r * cols + c];
}

// ---------------------------------------------------------------- host

struct TcPlan {
    int cg, bn, mt, nt, kiters, splits, kper;
    size_t part;         // bytes of the splits' sums
};

// The tile, by the time of the waves that it needs on 148 SMs: a tile's cost
// is its time for the same k, measured; 256 x 256 on a pair of CTAs is the
// cheapest an output, smaller ones waste less where there are few.  Few tiles
// over a long k are split along it, at least 4 stages a piece.
TcPlan tc_plan(long long M, long long N, long long K) {
    TcPlan p{};
    p.kiters = (int)((K + kBK - 1) / kBK);
    const int group[4] = {2, 2, 1, 1}, width[4] = {256, 128, 128, 64}, cost[4] = {176, 110, 148, 96};
    long long best = -1;
    for (int i = 0; i < 4; ++i) {
        const long long mt = (M + group[i] * kBM - 1) / (group[i] * kBM), nt = (N + width[i] - 1) / width[i];
        const int slots = kSmCount / group[i];
        const long long c = (mt * nt + slots - 1) / slots * cost[i];
        if (best < 0 || c < best) best = c, p.cg = group[i], p.bn = width[i], p.mt = (int)mt, p.nt = (int)nt;
    }
    const long long tiles = (long long)p.mt * p.nt, slots = kSmCount / p.cg;
    long long s = tiles <= slots / 2 ? slots / tiles : 1;
    if (s > p.kiters / 4) s = p.kiters / 4;
    if (s < 1) s = 1;
    p.kper = (int)((p.kiters + s - 1) / s);
    p.splits = (p.kiters + p.kper - 1) / p.kper;
    p.part = p.splits > 1 ? align256(size_t(p.splits) * M * ((N + 3) / 4 * 4) * sizeof(float)) : 0;
    return p;
}

bool setup() {
    return set_smem((const void *)gemm_tc<256, 2>, Cfg<256, 2>::kSmem) &&
           set_smem((const void *)gemm_tc<128, 2>, Cfg<128, 2>::kSmem) &&
           set_smem((const void *)gemm_tc<128, 1>, Cfg<128, 1>::kSmem) &&
           set_smem((const void *)gemm_tc<64, 1>, Cfg<64, 1>::kSmem);
}
bool g_ready[128] = {};

// An operand's map: rows of `inner` elements at pitch ld, boxes of 64 x box_rows, 128-byte swizzle.
bool operand_map(CUtensorMap *m, const void *base, long long inner, long long rows, long long ld, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return make_dit_map(m, base, 2, dims, strides, box, 128);
}

template <int BN, int CG>
int run_tc(const GemmPlan &g, const TcPlan &p, TcArgs &a, cudaStream_t s) {
    CUtensorMap ma, mb, my, mp, mr;
    // K-major: rows are m (n), boxes 64 k x tile rows; MN-major: rows are k, boxes 64 m (n) x 64 k
    if (!(g.a_mn ? operand_map(&ma, g.a, g.M, g.K, g.lda, kBK) : operand_map(&ma, g.a, g.K, g.M, g.lda, kBM))) return -1;
    if (!(g.b_mn ? operand_map(&mb, g.b, g.N, g.K, g.ldb, kBK) : operand_map(&mb, g.b, g.K, g.N, g.ldb, BN / CG))) return -1;
    my = mp = mr = ma;
    if (p.splits == 1 && !a.direct) {
        const cuuint64_t dims[2] = {(cuuint64_t)g.N, (cuuint64_t)g.M}, strides[1] = {(cuuint64_t)g.N * 2};
        const cuuint32_t box[2] = {kChunk, 32};
        if (!make_dit_map(&my, g.y, 2, dims, strides, box, 64)) return -1;
        if (g.pre && !make_dit_map(&mp, g.pre, 2, dims, strides, box, 64)) return -1;
        if (g.res && !make_dit_map(&mr, g.res, 2, dims, strides, box, 64)) return -1;
    }
    const long long works = (long long)p.mt * p.nt * p.splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(works < kSmCount / CG ? works : kSmCount / CG) * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<BN, CG>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, gemm_tc<BN, CG>, ma, mb, my, mp, mr, a) != cudaSuccess) return -1;
    if (p.splits == 1) return 1;
    const long long want = (g.M * g.N + 255) / 256;
    gemm_finish<<<(unsigned)(want < 16 * kSmCount ? want : 16 * kSmCount), 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? 2 : -1;
}

}  // namespace

bool make_dit_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                  const cuuint32_t *box, int swizzle_bytes) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUtensorMapSwizzle sw = swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE;
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool once_per_device(bool (*done)[128], bool (*f)()) {
    static std::mutex m;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return false;
    std::lock_guard<std::mutex> lock(m);
    if (!(*done)[dev]) (*done)[dev] = f();
    return (*done)[dev];
}

bool gemm_tc_fits(long long M, long long N, long long K) {
    return M < (1LL << 31) - 256 && N < (1LL << 31) - 256 && K < (1LL << 31) - 256 &&
           (M + kBM - 1) / kBM * ((N + 63) / 64) < (1LL << 31);
}

namespace {

// Workspace of a product: the splits' sums, then copies of operands whose rows are not whole 16 bytes.
struct TcWs {
    size_t a, b, total;
};
long long pitch8(long long ld) { return (ld + 7) / 8 * 8; }
TcWs tc_ws(const GemmPlan &g, const TcPlan &p) {
    TcWs w;
    w.a = p.part;
    w.b = w.a + (g.lda % 8 ? align256(size_t(g.a_mn ? g.K : g.M) * pitch8(g.lda) * 2) : 0);
    w.total = w.b + (g.ldb % 8 ? align256(size_t(g.b_mn ? g.K : g.N) * pitch8(g.ldb) * 2) : 0);
    return w;
}

// The operand at a pitch of whole 16 bytes: copied if its rows are not.
bool packed(const void *&x, long long &ld, long long rows, void *to, cudaStream_t s) {
    if (ld % 8 == 0) return true;
    const long long ldo = pitch8(ld);
    repack<<<(unsigned)(rows < 16 * kSmCount ? rows : 16 * kSmCount), 256, 0, s>>>((const __nv_bfloat16 *)x,
                                                                                  (__nv_bfloat16 *)to, rows, ld, ldo);
    x = to;
    ld = ldo;
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace

size_t gemm_tc_ws(const GemmPlan &g) { return tc_ws(g, tc_plan(g.M, g.N, g.K)).total; }

int launch_gemm_tc(const GemmPlan &g0, void *ws, cudaStream_t s) {
    if (!once_per_device(&g_ready, setup)) return -1;
    GemmPlan g = g0;
    const TcPlan p = tc_plan(g.M, g.N, g.K);
    const TcWs w = tc_ws(g, p);
    if (!packed(g.a, g.lda, g.a_mn ? g.K : g.M, (char *)ws + w.a, s)) return -1;
    if (!packed(g.b, g.ldb, g.b_mn ? g.K : g.N, (char *)ws + w.b, s)) return -1;
    TcArgs a{};
    a.M = g.M; a.N = g.N;
    a.kiters = p.kiters; a.mt = p.mt; a.nt = p.nt; a.splits = p.splits; a.kper = p.kper;
    a.a_mn = g.a_mn; a.b_mn = g.b_mn;
    a.bias = (const __nv_bfloat16 *)g.bias; a.res = (const __nv_bfloat16 *)g.res;
    a.pre = (__nv_bfloat16 *)g.pre; a.y = (__nv_bfloat16 *)g.y;
    a.part = (float *)ws; a.ldp = (g.N + 3) / 4 * 4;
    a.act = g.act;
    a.direct = g.N % 8 != 0;
    if (p.cg == 2) return p.bn == 256 ? run_tc<256, 2>(g, p, a, s) : run_tc<128, 2>(g, p, a, s);
    return p.bn == 128 ? run_tc<128, 1>(g, p, a, s) : run_tc<64, 1>(g, p, a, s);
}

int read_and_clear_linear_flag(unsigned *flag_out) {
    if (cudaMemcpyFromSymbol(flag_out, g_linear_flag, sizeof(unsigned)) != cudaSuccess) return -1;
    const unsigned zero = 0;
    if (*flag_out && cudaMemcpyToSymbol(g_linear_flag, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return 0;
}

}  // namespace la
