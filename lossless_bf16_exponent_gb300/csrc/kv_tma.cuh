// kv_tma.cuh -- cached rows by the tensor memory accelerator. A pool is a 4-D
// tensor of bytes (row bytes, page tokens, heads, pages) with the pool's own
// strides; one copy brings `box` consecutive tokens of a page, up to 128 bytes
// of each, to shared memory with the swizzle that the matrix loads and the
// tensor core read (kv_attention.cuh's row_chunk). Bytes past a row's end come
// as zeros, and so does a page that does not exist.
//
// A tile of tokens starts on a multiple of its size and a box is the largest
// power of two that divides both tile and page, so a box never leaves a page
// or a tile. It takes 8 rows at least, the swizzle's period; pages of other
// sizes are copied 16 bytes a thread instead. Why: 16-byte asynchronous copies
// keep about 32 KB in flight an SM whatever the ring's size (15 to 20 bytes a
// clock measured); one thread's bulk copies fill the ring.
#pragma once

#include <cuda.h>

#include "kv_attention.cuh"

namespace uzkv {

struct Maps {
    CUtensorMap k, v;
    uint32_t box;  // tokens of a copy
};

// Maps of a cache for tiles of `tile` tokens; false where its pages do not allow them, or copies of at least `least`
// bytes: a copy costs the accelerator about as much time as 1 to 2 KB take, so smaller ones fall behind the threads'
// copies. Measured, bulk / threads: many rows of 128, 2 KB copies 238 / 316 us; E5M2 of 64, 4 KB 39.7 / 48.3, 1 KB 54 / 47;
// mass, rows of 128, 8 KB 90 / 96 us; E5M2 of 64, 4 KB 21.9 / 24.5, 1 KB 27.1 / 24.9 us.
bool maps_of(const AttParams& p, const uzkv_cache_t* c, uint32_t tile, uint32_t least, Maps* m);

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* m, uint32_t x, uint32_t row, uint32_t head, uint32_t page,
                                        uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// One warp's copies of tiles of TILE tokens with RB bytes of a row (64, or blocks of 128). A lane keeps the page and
// row of one box; find() looks them up ahead of the copy.
template <uint32_t TILE, uint32_t RB>
struct TmaFeed {
    static constexpr uint32_t kWide = RB < 128 ? RB : 128, kBlocks = RB / kWide;
    Place at;       // of box `lane`
    uint32_t live;  // boxes of the tile that hold tokens in use

    __device__ __forceinline__ void find(const AttParams& p, const Maps& m, const Unit& u, bool any) {
        const uint32_t lane = threadIdx.x % 32, j0 = u.tile * TILE, end = u.span.old + u.span.fresh;
        live = any ? (min(TILE, end - j0) + m.box - 1) / m.box : 0;
        at = Place{0, 0};
        if (lane < live) at = look_up(p.cache, u.b, j0 + lane * m.box);
    }
    __device__ __forceinline__ uint32_t bytes(const Maps& m) const { return live * m.box * RB; }
    // All lanes, after the barrier expects bytes(): boxes by blocks over the lanes.
    __device__ __forceinline__ void copy(const AttParams& p, const Maps& m, const CUtensorMap* map, uint32_t head, uint32_t dst,
                                         uint32_t bar) const {
        const uint32_t lane = threadIdx.x % 32;
        const Place here = lane < live ? checked(p.cache, at) : Place{-1, 0};
        const uint32_t page = here.page < 0 ? p.cache.pages : (uint32_t)here.page, row = here.row;  // not there: zeros
        for (uint32_t i0 = 0; i0 < live * kBlocks; i0 += 32) {
            const uint32_t i = i0 + lane, block = i % kBlocks, n = i / kBlocks;
            const uint32_t pg = __shfl_sync(0xFFFFFFFFu, page, n % 32), rw = __shfl_sync(0xFFFFFFFFu, row, n % 32);
            if (i < live * kBlocks) tma_box(dst + block * TILE * kWide + n * m.box * kWide, map, block * kWide, rw, head, pg, bar);
        }
    }
};

}  // namespace uzkv
