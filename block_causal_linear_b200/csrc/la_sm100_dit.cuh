// la_sm100_dit.cuh -- the sm_100a pieces that the operators around the linear
// attention need beside la_sm100.cuh: two-dimensional tile copies, tensor maps
// of any matrix, per-device kernel set-up.
#pragma once

#include "la_dit.cuh"
#include "la_sm100.cuh"

namespace la {
namespace sm100 {

constexpr uint32_t kLayoutSw64 = 4;

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}

}  // namespace sm100

// A bf16 tensor map: dims innermost first (elements), byte strides of dims
// 1.., box extents, swizzle of 64 or 128 bytes (or 0), zero fill out of range.
bool make_dit_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                  const cuuint32_t *box, int swizzle_bytes);

// Runs `setup` (function attributes) once on each device that launches; the
// current device's result.
bool once_per_device(bool (*done)[128], bool (*setup)());

}  // namespace la
