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

// Pages of a tile: lane l < 128 / page_size has the one that holds positions tile * 128 + l * page_size and on.
// fetch() asks the table ahead of time (a load that nothing waits for), check() takes its word where the pages are
// needed: num_pages, whose rows a tiled load fills with zeros, where the request has no such position or the
// table names a page that does not exist (which is reported).
struct Pages {
    int raw;
    bool there;
    __device__ __forceinline__ void fetch(const CacheParams &c, int b, int kv_len, int tile, int lane) {
        const long long pos = (long long)tile * kKeyTile + (long long)lane * c.page_size;
        there = lane < kKeyTile / c.page_size && pos < kv_len;
        raw = there ? c.page_table[(long long)b * c.max_pages + pos / c.page_size] : 0;
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
    for (int l = 0; l < kKeyTile / page_size; ++l) {
        const int at = __shfl_sync(0xffffffffu, page, l);
        if (elect()) {
            tma_load_5d(dst + l * page_size * 128, map, bar, 0, 0, 0, head, at);
            tma_load_5d(dst + l * page_size * 128 + kHalfBytes, map, bar, 0, 0, 1, head, at);
        }
    }
    __syncwarp();
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

// A row's partial results joined: o = sum_c 2^{m_c - m} O_c / sum_c 2^{m_c - m} l_c over CTAs c = first .. ctas - 1, a lane
// per CTA and step, four of their rows in flight; lane l gets columns 4 l .. 4 l + 3.  piece(c, at): whether CTA c has
// left a result, and where its O row is (m and l follow `to_ml` floats behind it); `behind(c)`: its run and all later ones
// lie behind the item.  False if no CTA has left any: one had the whole item, and has written it.
template <class Piece, class Behind>
__device__ __forceinline__ bool join_row(int first, int ctas, long long to_ml, int lane, uint2 &out, Piece piece,
                                         Behind behind) {
    bool any = false;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = first; c0 < ctas; c0 += 32) {
        const int c = c0 + lane;
        const bool past = c >= ctas || behind(c);
        const float *at = nullptr;
        float2 ml = make_float2(-INFINITY, 0.f);
        const bool mine = !past && piece(c, at);
        if (mine) ml = *reinterpret_cast<const float2 *>(at + to_ml);
        any |= __any_sync(0xffffffffu, mine);
        float top = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m);
        // a piece whose keys the row does not see, and a lane without one, has m = -inf and counts for nothing
        const float w = ml.x == -INFINITY ? 0.f : ex2z(ml.x - top), f = m == -INFINITY ? 0.f : ex2z(m - top);
        float add = w * ml.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
        m = top;
        l = l * f + add;
        o.x *= f;
        o.y *= f;
        o.z *= f;
        o.w *= f;
        unsigned left = __ballot_sync(0xffffffffu, w > 0.f);
        while (left) {
            float4 x[4];
            float g[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int src = left ? __ffs(left) - 1 : 0;
                g[k] = __shfl_sync(0xffffffffu, w, src);
                const float *row = reinterpret_cast<const float *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), src));
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (left)
                    x[k] = reinterpret_cast<const float4 *>(row)[lane];
                else
                    g[k] = 0.f;
                left &= left - 1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o.x += g[k] * x[k].x;
                o.y += g[k] * x[k].y;
                o.z += g[k] * x[k].z;
                o.w += g[k] * x[k].w;
            }
        }
        if (__any_sync(0xffffffffu, past)) break;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    out = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    return any;
}

}  // namespace attn

// TMA maps (host): pages of a cache, boxes of 64 columns x page_size rows; rows of q, boxes of 64 columns
// x the query heads of a group x `tokens` tokens.
bool make_pages_map(CUtensorMap *m, const void *pages, const CacheParams &c, int Hkv);
bool make_query_map(CUtensorMap *m, const void *q, long long rows, int H, long long row_stride, int group,
                    int tokens);

}  // namespace la
