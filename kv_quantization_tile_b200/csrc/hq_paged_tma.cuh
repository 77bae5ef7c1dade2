// hq_paged_tma.cuh -- TMA loads of cache pages and their barriers (sm_100a),
// shared by the two attention kernels.
#pragma once

#include <cuda.h>

#include "hq_paged.h"
#include "hq_tcgen05.cuh"

namespace hq {

// A pool as [page][head][slot][d]: one copy takes up to `box` slots of 64
// columns; a page past the pool reads zeros.
cudaError_t page_map(CUtensorMap *m, const PagedArgs &a, const void *pool, int d, int box);

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Up to `box` slots of a page, 64 columns from `col`, to `dst` (128-byte swizzle)
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, uint32_t bar, int col, int slot, int head, int page)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(col), "r"(slot), "r"(head), "r"(page)
        : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// byte offset of 16-byte chunk c of row r in a 128-byte-swizzled operand of
// `rows` rows: blocks of 64 columns, each [rows][128 bytes]
__device__ __forceinline__ uint32_t swizzled_off(int rows, int r, int c)
{
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

}  // namespace hq
