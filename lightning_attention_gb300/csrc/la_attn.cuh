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

// log2 of the page size, one of 16 to 128.
__device__ __forceinline__ int page_shift(const CacheParams &c) { return 31 - __clz(c.page_size); }

// Pages of a tile: lane l < 128 / page_size has the one that holds positions tile * 128 + l * page_size and on.
// fetch() asks the table ahead of time (a load that nothing waits for), check() takes its word where the pages are
// needed: num_pages, whose rows a tiled load fills with zeros, where the request has no such position or the
// table names a page that does not exist (which is reported).
struct Pages {
    int raw;
    bool there;
    __device__ __forceinline__ void fetch(const CacheParams &c, int b, int kv_len, int tile, int lane) {
        const int per_tile = kKeyTile >> page_shift(c), at = tile * per_tile + lane;
        there = lane < per_tile && (uint32_t)at << page_shift(c) < (uint32_t)kv_len;
        raw = there ? c.page_table[(long long)b * c.max_pages + at] : 0;
    }
    __device__ __forceinline__ int check(const CacheParams &c, unsigned int *err) const {
        if (!there) return c.num_pages;
        if (raw >= 0 && raw < c.num_pages) return raw;
        atomicOr(err, ERR_BIT_PAGE);
        return c.num_pages;
    }
};

// A whole warp brings one tile in; `page`: Pages::check's.  Every row of the tile is written.
__device__ __forceinline__ void load_tile(const CUtensorMap *map, uint8_t *dst, uint64_t *bar, int page,
                                          int page_size, int head) {
    if (elect()) mbar_arrive_expect_tx(bar, kTileBytes);
#pragma unroll 1
    for (int row = 0, l = 0; row < kKeyTile; row += page_size, ++l) {
        const int at = __shfl_sync(0xffffffffu, page, l);
        if (elect()) {
            tma_load_5d(dst + row * 128, map, bar, 0, 0, 0, head, at);
            tma_load_5d(dst + row * 128 + kHalfBytes, map, bar, 0, 0, 1, head, at);
        }
    }
    __syncwarp();
}

// A bounded wait; the first to give up reports it.  What a role has under way when it ends (copies into shared memory,
// MMAs) is waited for with a limit of its own, however short the one on other waits is set: a CTA that left before
// would have its shared or tensor memory written under the next one.
constexpr uint64_t kDrainLimitNs = 2000000000ull;
struct Waiter {
    uint64_t limit_ns;
    unsigned int *err;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_wait(bar, parity, limit_ns)) return true;
        atomicOr(err, ERR_BIT_TIMEOUT);
        return false;
    }
    __device__ __forceinline__ Waiter to_the_end() const { return {kDrainLimitNs, err}; }
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

// Requests in groups, one for each of kGroups warps.
template <int kGroups>
__device__ __forceinline__ uint32_t group_size(int B) {
    return (((uint32_t)B + kGroups * 32 - 1) / (kGroups * 32)) * 32;
}
__device__ __forceinline__ long long scan_lanes(long long x) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}
// The sum of work(b) over the requests of every group, by warps 0 .. kGroups - 1.
template <int kGroups, class Work>
__device__ __forceinline__ void sum_groups(int B, long long *sums, Work work) {
    const uint32_t size = group_size<kGroups>(B), begin = (threadIdx.x >> 5) * size;
    const uint32_t end = min(begin + size, (uint32_t)B);
    long long x = 0;
#pragma unroll 1
    for (uint32_t b = begin + (threadIdx.x & 31); b < end; b += 32) x += work((int)b);
    x = scan_lanes(x);
    if ((threadIdx.x & 31) == 31) sums[threadIdx.x >> 5] = x;
}
// The work of all requests, and the request within whose work place x = at(all) lies with the place where that begins (none
// behind the last one's).  One warp.
struct Place {
    int b = -1;
    long long first = 0;
    template <int kGroups, class Work, class At>
    __device__ __forceinline__ Place(const long long (&sums)[kGroups], int B, Work work, At at) {
        const uint32_t lane = threadIdx.x & 31, size = group_size<kGroups>(B);
        long long mine = lane < kGroups ? sums[lane] : 0, upto = scan_lanes(mine);
        const long long x = at(__shfl_sync(0xffffffffu, upto, 31));
        unsigned hit = __ballot_sync(0xffffffffu, x >= upto - mine && x < upto);
        if (hit == 0) return;
        int src = __ffs(hit) - 1;
        first = __shfl_sync(0xffffffffu, upto - mine, src);
#pragma unroll 1
        for (uint32_t b0 = (uint32_t)src * size; b0 < (uint32_t)B; b0 += 32) {
            mine = b0 + lane < (uint32_t)B ? work((int)(b0 + lane)) : 0;
            upto = first + scan_lanes(mine);
            hit = __ballot_sync(0xffffffffu, x >= upto - mine && x < upto);
            src = hit ? __ffs(hit) - 1 : 31;
            first = __shfl_sync(0xffffffffu, hit ? upto - mine : upto, src);
            if (hit == 0) continue;
            b = (int)b0 + src;
            return;
        }
    }
};

// The work of a batch in equal runs, one per CTA, the first `more` of them one unit longer.
struct Runs {
    long long each;
    int more, ctas;
    __device__ __forceinline__ Runs(long long all, int ctas_)
        : each(all / ctas_), more((int)(all - each * ctas_)), ctas(ctas_) {}
    __device__ __forceinline__ long long start(int c) const { return each * c + min(c, more); }
};

// The item inside which a CTA's run ends, if it is the first run that does: left for the second launch, which joins the
// results of the CTAs that share it.
struct Tail {
    Runs runs;
    long long at, size;  // the item's work [at, at + size)
    int tiles;           // of the item; 0: nothing to join
    int b, kvh, first;   // request, kv head, first token
    int t0, n;           // the request's first row and its tokens
};

// The partial results of an item: a list, in the CTAs' order, of their numbers (two a CTA: 2 c + 1 from the item's first
// tile on, 2 c from a later one).  One warp, from the CTA whose run ends first inside it; returns their count, 0 if
// one CTA had the whole item (and has written it).  cut(x): the tile at which the item's first x of work end.
template <class Cut>
__device__ __forceinline__ int list_pieces(const Tail &t, int first, int *list, Cut cut) {
    const int lane = threadIdx.x & 31;
    int count = 0;
    for (int c0 = first; c0 < t.runs.ctas; c0 += 32) {
        const int c = min(c0 + lane, t.runs.ctas);
        const long long lo = t.runs.start(c), hi = t.runs.start(min(c + 1, t.runs.ctas));
        const int j0 = cut(lo - t.at), j1 = cut(hi - t.at);
        const bool mine = j0 < j1 && j1 - j0 < t.tiles;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (mine) list[count + __popc(who & ((1u << lane) - 1))] = 2 * c + (j0 == 0);
        count += __popc(who);
        if (__any_sync(0xffffffffu, hi >= t.at + t.size)) break;
    }
    __syncwarp();
    return count;
}

}  // namespace attn

// TMA maps (host): pages of a cache, boxes of 64 columns x page_size rows; rows of q, boxes of 64 columns
// x the query heads of a group x `tokens` tokens.
bool make_pages_map(CUtensorMap *m, const void *pages, const CacheParams &c, int Hkv);
bool make_query_map(CUtensorMap *m, const void *q, long long rows, int H, long long row_stride, int group,
                    int tokens);

}  // namespace la
