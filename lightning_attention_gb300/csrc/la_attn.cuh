// la_attn.cuh -- what the two attention kernels share on the device: loads of key and value tiles
// through the page table, MMAs issued from a converged warp, waits, packed arithmetic.
#pragma once

#include "la_attn.h"
#include "la_sm100.cuh"

namespace la {
namespace attn {

using namespace sm100;

constexpr int kTileBytes = kKeyTile * kHeadDim * 2;  // a tile of keys or values: two blocks of 64
constexpr int kHalfBytes = kTileBytes / 2;           // columns, rows of 128 bytes, 128-byte swizzle

// 5D tiled load: coordinates (column, row, block of 64 columns, kv head, page).
__device__ __forceinline__ void tma_load_5d(void *smem_dst, const void *tmap, uint64_t *bar, int c0,
                                            int c1, int c2, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(c4)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *smem_dst, const void *tmap, uint64_t *bar, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Lane l < 128 / page_size: the page that holds positions pos .. of request b, pos = tile * 128 + l *
// page_size; num_pages, whose rows a tiled load fills with zeros, where the request has no such position
// or the table names a page that does not exist (which is reported).
__device__ __forceinline__ int page_of(const CacheParams &c, int b, int kv_len, int tile, int lane,
                                       unsigned int *err) {
    const long long pos = (long long)tile * kKeyTile + (long long)lane * c.page_size;
    if (lane >= kKeyTile / c.page_size || pos >= kv_len) return c.num_pages;
    const int page = c.page_table[(long long)b * c.max_pages + pos / c.page_size];
    if (page >= 0 && page < c.num_pages) return page;
    atomicOr(err, ERR_BIT_PAGE);
    return c.num_pages;
}

// A whole warp brings one tile in; `page` is page_of's.  Every row of the tile is written.
__device__ __forceinline__ void load_tile(const CUtensorMap *map, uint8_t *dst, uint64_t *bar, int page,
                                          int page_size, int head, int lane) {
    if (lane == 0) mbar_arrive_expect_tx(bar, kTileBytes);
    __syncwarp();
    if (lane < kKeyTile / page_size) {
        uint8_t *at = dst + lane * page_size * 128;
        tma_load_5d(at, map, bar, 0, 0, 0, head, page);
        tma_load_5d(at + kHalfBytes, map, bar, 0, 0, 1, head, page);
    }
}

// One lane of a converged warp, always the same.  MMAs are issued by `if (elect()) { ... }` around a batch of
// them and its commits: 38 cycles an issue (N = 16) to 62 (N = 128, as long as the MMA takes); with the instruction
// predicated on lane 0 60 to 80, the operands' uniform registers being loaded for each.
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// A bounded wait; the first to give up reports it.
struct Waiter {
    uint64_t limit_ns;
    unsigned int *err;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_wait(bar, parity, limit_ns)) return true;
        atomicOr(err, ERR_BIT_TIMEOUT);
        return false;
    }
};

// 2^x, what is below the normal range as 0: one instruction, 4 cycles a warp (without .ftz three, 4.6 to 6.5).
__device__ __forceinline__ float ex2z(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace attn

// TMA maps (host): pages of a cache, boxes of 64 columns x page_size rows; rows of q, boxes of 64 columns
// x the query heads of a group x `tokens` tokens.
bool make_pages_map(CUtensorMap *m, const void *pages, const CacheParams &c, int Hkv);
bool make_query_map(CUtensorMap *m, const void *q, long long rows, int H, long long row_stride, int group,
                    int tokens);

}  // namespace la
