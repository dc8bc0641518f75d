// la_attn_extend.cu -- softmax attention of packed prompts over a paged key/value cache (causal,
// grouped heads): for query row i of a request, with the keys at and before its position,
//     o_i = sum_j e^{s_ij - m_i} v_j / sum_j e^{s_ij - m_i},   s_ij = scale q_i . k_j
// in one pass over the keys, m_i a running reference.  The same for trees of drafts (and single tokens) whose rows
// -- drafts x query heads of a kv head -- are more than la_attn_verify.cu takes: a row sees the positions before the
// drafts, its ancestors and itself.
//
// An item is two tiles of up to 128 rows -- consecutive tokens x the query heads of one kv head, so
// that the heads of a group share its keys -- and the tiles of 128 keys that they see.  Per key tile and row
// tile, S = Q K^T (tcgen05, fp32 in tensor memory), P = exp2(S scale log2 e - m) by two threads per row
// (bf16, back into S's columns), O += P V (P from tensor memory, V as it lies in its page).  While one
// tile's softmax runs, the tensor cores work on the other tile:
//     S0(j) S1(j) | O0 += P0 V, S0(j+1) | O1 += P1 V, S1(j+1) | ...
// Warps 0-7 and 8-15: softmax of tile 0 and 1, a thread for each half of a row's keys (one thread took 1400 cycles
// a tile, which with the row's MMAs made 2850 of 2048), its weights in two parts, so that O += P V begins with the first;
// warp 16 issues the MMAs; warp 17 works out the items and loads queries and keys, warp 18 the values (TMA, a box per
// page and half of the columns).
//
// Long prompts are bound by the tensor cores: 32 MMAs of 64 cycles per item and key tile, 65 measured (16,384 tokens, 32
// heads on 8: 1300 to 1430 us as the power limit lets the clock go, 1145 with the MMAs alone; floor 1139, or 1279 at the
// rate that large products sustain).  That leaves a row's threads 1024 cycles from S to P, so they do not look for the
// row's largest score first: exponents against the reference they have, which follows only when a weight would pass 2^8
// (S is then read again, and O, which lies in tensor memory, rescaled): sums stay far inside fp32.
// P is rounded to bf16 (at most 2^-8 of each weight, either way: together about out's own rounding), the sums
// of its values are formed in fp32 before that.
//
// Items differ in length by orders of magnitude, so a CTA per SM takes an equal run of the whole batch's work,
// item by item, and may begin and end inside one; what it leaves of those, unnormalised, a second launch joins in a
// fixed order.  Between two items nothing hides what they need once: an item's rows go out behind the next one's first
// weights, while the tensor cores go on (eight prompts of 512 to 4096 tokens, 32 heads on 4: 437 -> 426 us), and the
// code of all roles is kept small, as 16 to 20 warps at different places of it fetch it anew for every item (with
// 184 KB, two thirds of it the walk over the items, 64 prompts of 200 to 400 tokens took 151 us; with 64 KB 113).
#include <string.h>

#include <algorithm>
#include <mutex>

#include "la_attn.cuh"

namespace la {
namespace {

using namespace attn;

constexpr int kRowTile = 128;
constexpr int kItemRows = 2 * kRowTile;
constexpr int kSlots = 5;  // tiles of keys and values in shared memory
constexpr int kThreads = 640;
constexpr int kMmaWarp = 16, kLoadWarp = 17, kValueWarp = 18;
constexpr int kRegsSoftmax = 104, kRegsRest = 64;  // a thread, by warp groups
static_assert(4 * kRegsSoftmax + kRegsRest <= 5 * 96, "register split");
constexpr int kItems = 4;  // items ahead
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffKV = kOffQ + 2 * kTileBytes;
constexpr uint32_t kOffBars = kOffKV + kSlots * kTileBytes;

// A partial result: of every group of 32 rows (a lane each) O in pieces of four columns, lane by lane, so that stores and
// loads of a warp are contiguous, then m and l of all rows.
constexpr int kPieceFloats = kItemRows * (kHeadDim + 2);

// What a CTA's warps have to know of an item.
struct Rec {
    int b, t0, n, kv_len, kvh, tok0;  // request, its first row, tokens, positions; kv head; first token
    int j0, j1, whole;             // tiles of keys that the CTA takes (none: the end of its run), all that there are
    int sound;                     // no parent out of range
};

constexpr uint8_t kNoParent = 255;

struct Bars {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full, q_empty, s_full[2], p_full[2][2], o_full[2], o_free[2], drain;
    uint64_t item_full[kItems], item_empty[kItems];
    Rec items[kItems];
    uint8_t parent[kItems][kMaxDrafts];  // of a tree's drafts; kNoParent: the context
    union {
        // Between a row's threads: [row tile][half][row].  Largest scores, then sums; between a thread's read and the other's
        // next write there is a barrier of the pair.
        float swap[2][2][kRowTile];
        long long work[kMmaWarp];    // of groups of requests, until the first item is known
    };
    int loads[2];  // of keys and of values, at the end
    uint32_t tmem_base;
};
constexpr uint32_t kSmemBytes = kOffBars + sizeof(Bars);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

constexpr uint32_t kTmS = 0, kTmO = 256, kTmCols = 512;

// Geometry of request b, and whether it is sound.
struct Request {
    int t0, n, kv_len;
};
__device__ __forceinline__ bool request_of(const AttnParams &p, int b, Request &r) {
    r.kv_len = p.cache.kv_lens[b];
    if (p.cu_seqlens == nullptr) {  // N drafts each
        r.t0 = b * p.N;
        r.n = p.N;
        return r.kv_len >= p.N && r.kv_len <= (long long)p.cache.max_pages * p.cache.page_size;
    }
    r.t0 = p.cu_seqlens[b];
    const int t1 = p.cu_seqlens[b + 1];
    r.n = t1 - r.t0;
    return r.t0 >= 0 && t1 >= r.t0 && t1 <= p.T && r.n <= p.max_seqlen && r.kv_len >= r.n &&
           r.kv_len <= (long long)p.cache.max_pages * p.cache.page_size;
}

// Work of a kv head's first `items` items of a request: the keys that they see and kItemKeys each for what an item
// costs besides, or one each where items are not cut.  (Eight prompts of 512 to 4096 tokens: 430 us with 200, 414 with
// 260, 417 with 320, 422 with 400.)
constexpr int kItemKeys = 260;
static_assert(kItemKeys >= kKeyTile, "an item's work covers its tiles");
__device__ __forceinline__ long long work_of(const AttnParams &p, const Request &r, long long items, long long tok) {
    if (!p.split) return items;
    return items * (r.kv_len - r.n + kItemKeys) + tok * (items * (items + 1) / 2);
}
// The tile at which the first `done` of an item's work end; what it costs besides counts as its end.
__device__ __forceinline__ int cut(long long done, int tiles) {
    return done <= 0 ? 0 : (int)min((long long)tiles, done / kKeyTile);
}
// Tokens of an item, and a request's items of a kv head.
__device__ __forceinline__ int tokens_of(const AttnParams &p) { return 2 * (kRowTile / p.group); }
__device__ __forceinline__ int items_of(const Request &r, int tok) {
    return (int)(((uint32_t)r.n + tok - 1) / (uint32_t)tok);
}

// Work of a request; with `report` a faulty one, which has none, is reported.
__device__ __forceinline__ long long request_work(const AttnParams &p, int b, int tok, bool report) {
    Request r;
    if (request_of(p, b, r)) return work_of(p, r, items_of(r, tok), tok) * p.Hkv;
    if (report && (p.cu_seqlens != nullptr || r.kv_len != 0)) atomicOr(p.err, ERR_BIT_SEQLENS);
    return 0;
}

// An item: rows of request b from token tok0 on, kv head kvh, its work [at, at + size), its tiles of keys.
struct Item {
    Request r = {};
    int b = 0, kvh = 0, t = 0, tok0 = 0, tiles = 0;
    int tok = 1, count = 0;  // tokens of an item, items of the request
    long long at = 0, size = 0;
    // the item whose work holds place x of request b, whose work begins at `first`
    __device__ __forceinline__ void find(const AttnParams &p, int b_, long long first, long long x) {
        b = b_;
        request_of(p, b, r);
        count = items_of(r, tok);
        const long long head = work_of(p, r, count, tok);
        kvh = (int)((x - first) / head);
        const long long rem = x - first - kvh * head;
        int lo = 0, hi = count - 1;
        while (lo < hi) {  // the last t whose work begins at rem or before
            const int mid = (lo + hi + 1) >> 1;
            if (work_of(p, r, mid, tok) <= rem)
                lo = mid;
            else
                hi = mid - 1;
        }
        t = lo;
        at = first + kvh * head + work_of(p, r, lo, tok);
    }
    __device__ __forceinline__ void measure(const AttnParams &p) {
        size = p.split ? r.kv_len - r.n + kItemKeys + (long long)tok * (t + 1) : 1;
        tok0 = t * tok;
        tiles = (r.kv_len - r.n + min(r.n, tok0 + tok) - 1) / kKeyTile + 1;
    }
    // the next one; false behind the last
    __device__ __forceinline__ bool next(const AttnParams &p) {
        at += size;
        if (++t < count) return true;
        t = 0;
        if (++kvh < p.Hkv) return true;
        kvh = 0;
        do {
            if (++b >= p.B) return false;
        } while (!request_of(p, b, r) || r.n == 0);
        count = items_of(r, tok);
        return true;
    }
};

// The items of a CTA's run, those of which it has no tile left out.  Its code is fetched anew for every item, so there is
// one copy of each step.
struct Walk {
    Item it;
    Runs runs;
    long long lo, hi;
    int j0, j1;
    bool begun = false;
    // one warp
    __device__ __forceinline__ Walk(const AttnParams &p, const long long (&sums)[kMmaWarp]) : runs(0, 1) {
        it.tok = tokens_of(p);
        const Place place(
            sums, p.B, [&](int x) { return request_work(p, x, it.tok, false); },
            [&](long long all) {
                runs = Runs(all, gridDim.x);
                lo = runs.start(blockIdx.x);
                hi = runs.start(blockIdx.x + 1);
                return lo;
            });
        if (place.b < 0) hi = lo;  // none behind the last (nor where somebody changes the lengths meanwhile)
        if (lo < hi) it.find(p, place.b, place.first, lo);
    }
    // The next item of which a tile is the CTA's; false: there is none.  tail(): the item is the one inside which the run
    // ends, and no earlier run does.
    template <class TailOf>
    __device__ __forceinline__ bool next(const AttnParams &p, TailOf tail) {
        while (true) {
            if (begun ? !it.next(p) || it.at >= hi : lo >= hi) return false;
            begun = true;
            it.measure(p);
            j0 = cut(lo - it.at, it.tiles);
            j1 = hi >= it.at + it.size ? it.tiles : cut(hi - it.at, it.tiles);
            if (it.at >= lo && it.at + it.size > hi) tail();
            if (j0 < j1) return true;
        }
    }
};

// A row's reference before it has seen a key: any score passes it, and -inf stays -inf against it.
constexpr float kUnseen = 1e30f;

// Columns 0 .. last of 32, a bit each.
__device__ __forceinline__ uint32_t columns_seen(int last) {
    return last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;
}

// 32 columns of which the first is draft d (those before draft 0 are seen by every row): a bit for each that is in `up`.
__device__ __forceinline__ uint32_t drafts_seen(const uint32_t (&up)[4], int d) {
    if (d <= -32) return 0xffffffffu;
    if (d < 0) return (up[0] << -d) | ((1u << -d) - 1u);
    const int q = d >> 5;
    const uint32_t lo = q == 0 ? up[0] : q == 1 ? up[1] : q == 2 ? up[2] : q == 3 ? up[3] : 0u;
    const uint32_t hi = q == 0 ? up[1] : q == 1 ? up[2] : q == 2 ? up[3] : 0u;
    return __funnelshift_r(lo, hi, d & 31);
}

// 32 scores of a row of which it sees those with a bit in `bits`.
__device__ __forceinline__ void mask_scores(uint32_t (&x)[32], uint32_t bits) {
#pragma unroll
    for (int y = 0; y < 32; ++y)
        if (!(bits & (1u << y))) x[y] = 0xff800000u;
}
__device__ __forceinline__ float largest(const uint32_t (&x)[32], float top) {
#pragma unroll
    for (int y = 0; y < 32; y += 2) top = max3(top, __uint_as_float(x[y]), __uint_as_float(x[y + 1]));
    return top;
}
// The scores as exponents against the reference.  Scalar arithmetic: a packed fma.f32x2 takes 4.3 cycles a warp, two
// fma.f32 2.6.
__device__ __forceinline__ void exponents(uint32_t (&x)[32], float c, float neg_m) {
#pragma unroll
    for (int y = 0; y < 32; ++y) x[y] = __float_as_uint(fmaf(__uint_as_float(x[y]), c, neg_m));
}
// Their weights, to tensor memory as bf16 pairs, and added to four partial sums.
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], uint32_t tp, float (&l)[4]) {
    uint32_t w[16];
#pragma unroll
    for (int y = 0; y < 16; ++y) {
        const float lo = ex2z(__uint_as_float(x[2 * y])), hi = ex2z(__uint_as_float(x[2 * y + 1]));
        l[(2 * y) & 3] += lo;
        l[(2 * y + 1) & 3] += hi;
        w[y] = pack_bf16x2(lo, hi);
    }
    tmem_st16(tp, w);
}

// The two warps that share 32 rows; whether any of their threads says so.
__device__ __forceinline__ bool pair_any(int pair, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(pair + 1)
        : "memory");
    return r != 0;
}

// Four rows' 64 bytes, a lane each in four pieces, to piece `lane % 4` of the four rows: rows of a quad are then
// stored 64 bytes at a time (16 at a time the stores of an item hold the SM's store path for 4096 cycles).
__device__ __forceinline__ void quad_transpose(uint4 (&x)[4], int lane) {
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        const bool up = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
            uint32_t *a = reinterpret_cast<uint32_t *>(&x[i]), *b = reinterpret_cast<uint32_t *>(&x[i + d]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a[y] : b[y], d);
                if (up)
                    a[y] = got;
                else
                    b[y] = got;
            }
        }
    }
}

template <bool kTree>
__device__ void softmax_role(const AttnParams &p, Bars *bars, uint32_t tbase, int warp, int lane, const Waiter &wait) {
    const int stage = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, pair = stage * 4 + quarter;
    const uint32_t lanes = (uint32_t)quarter << 21;  // in the address's upper half
    const uint32_t ts = tbase + kTmS + stage * 128 + half * 64 + lanes, to = tbase + kTmO + stage * 128 + half * 64 + lanes;
    const int row = quarter * 32 + lane;
    // the row's token and head of an item, 8 bits each; -1: it has none
    int mine = kRowTile / p.group;
    mine = row < mine * p.group ? (stage * mine + row / p.group) << 8 | row % p.group : -1;
    const float c = p.scale_log2;
    if (p.cu_seqlens == nullptr) {  // rows without keys: a request of no positions
        for (int b = blockIdx.x; b < p.B; b += gridDim.x)
            if (p.cache.kv_lens[b] == 0)
                for (int i = threadIdx.x; i < p.N * p.H * (kHeadDim / 8); i += kMmaWarp * 32)
                    reinterpret_cast<uint4 *>(p.out + (long long)b * p.N * p.H * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
    }
    bool ok = true;
    uint32_t tile = 0, item = 0;
    float done_l = 0.f, done_m = 0.f;  // the item before: the row's sum and minus its reference
    for (;; ++item) {
        ok = ok && __all_sync(0xffffffffu, wait(&bars->item_full[item % kItems], (item / kItems) & 1));
        const Rec it = bars->items[item % kItems];
        const bool live = it.j1 > it.j0;
        if (pair_any(pair, !ok)) return;
        const int tok = it.tok0 + (mine >> 8);
        const bool inside = mine >= 0 && tok < it.n;
        // Last column of this half, counted from the first key, that the row sees (rows that are not written take any),
        // and that all rows of the warp do.
        int limit = it.kv_len - it.n + (inside ? tok : it.n - 1) - half * 64, lo_limit;
        uint32_t up[4] = {0, 0, 0, 0};  // drafts that it sees, a bit each
        if constexpr (kTree) {
            for (uint32_t a = inside ? tok : live ? 0 : kNoParent; a != kNoParent; a = bars->parent[item % kItems][a])
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((a >> 5) == i) up[i] |= 1u << (a & 31);
            limit = it.kv_len - it.n - half * 64;  // where the drafts begin
            lo_limit = limit - 1;
        } else {
            lo_limit = __reduce_min_sync(0xffffffffu, limit);
        }
        float neg_m = kUnseen;
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
        int state = 0;  // of the last tile
        for (int j = it.j0; j == it.j0 || j < it.j1; ++j) {
            if (live) {
                ok = ok && __all_sync(0xffffffffu, wait(&bars->s_full[stage], tile & 1));
                tc_fence_after();
                const int last = limit - j * kKeyTile, lo_last = lo_limit - j * kKeyTile;
                auto seen = [&](int i) {
                    if constexpr (kTree)
                        return drafts_seen(up, i * 32 - last);
                    else
                        return columns_seen(last - i * 32);
                };
                // Against the reference that there is; with the item's first tile, and once more where a weight passes 2^8,
                // against a new one.
                uint32_t x[2][32];
                state = j == it.j0;  // 1: a new reference is to be found, 2: it has been
                while (true) {
                    tmem_ld32(ts, x[0]);
                    tmem_ld32(ts + 32, x[1]);
                    tmem_ld_wait_regs2(x[0], x[1]);
                    if (lo_last < 63) {
                        mask_scores(x[0], seen(0));
                        mask_scores(x[1], seen(1));
                    }
                    if (state == 1) {
                        float top = fmaxf(largest(x[0], -INFINITY), largest(x[1], -INFINITY));
                        bars->swap[stage][half][row] = top;
                        if (pair_any(pair, !ok)) return;
                        top = fmaxf(top, bars->swap[stage][half ^ 1][row]) * c;
                        float f = 1.f;
                        if (top > 8.f - neg_m) {
                            f = neg_m == kUnseen ? 0.f : ex2z(-neg_m - top);
                            neg_m = -top;
                        }
                        if (j > it.j0) {  // S(j) was issued behind O += P(j-1) V, which is complete
#pragma unroll
                            for (int i = 0; i < 4; ++i) l4[i] *= f;
#pragma unroll 1
                            for (int i = 0; i < 2; ++i) {
                                uint32_t o[32];
                                tmem_ld32(to + i * 32, o);
                                tmem_ld_wait_regs(o);
#pragma unroll
                                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                                tmem_st32(to + i * 32, o);
                            }
                            state = 2;
                            continue;
                        }
                    }
                    exponents(x[0], c, neg_m);
                    exponents(x[1], c, neg_m);
                    if (state) break;
                    const float top = fmaxf(largest(x[0], -INFINITY), largest(x[1], -INFINITY));
                    if (!pair_any(pair, top > 8.f || !ok)) break;
                    state = 1;
                }
                // a part of 32 keys at a time, so that the tensor cores begin with the first while the second is weighed
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    weigh(x[i], ts + i * 16, l4);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (elect()) mbar_arrive(&bars->p_full[stage][i]);
                }
                ++tile;
            }
            // the rows of the item before, whose O is complete or about to be
            if (j == it.j0 && item > 0) {
                const Rec &was = bars->items[(item - 1) % kItems];
                ok = ok && __all_sync(0xffffffffu, wait(&bars->o_full[stage], (item - 1) & 1));
                if (pair_any(pair, !ok)) return;
                tc_fence_after();
                const int wtok = was.tok0 + (mine >> 8);
                const bool valid = mine >= 0 && wtok < was.n && was.sound;
                const long long out_row = (long long)(was.t0 + wtok) * p.H + was.kvh * p.group + (mine & 255);
                const long long at = out_row * kHeadDim + half * 64;
                if (was.whole) {
                    const float f = 1.f / done_l;
                    uint4 w[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t o[32];
                        tmem_ld32(to + i * 32, o);
                        tmem_ld_wait_regs(o);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t y[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                y[z] = pack_bf16x2(__uint_as_float(o[8 * x + 2 * z]) * f,
                                                   __uint_as_float(o[8 * x + 2 * z + 1]) * f);
                            w[i][x] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (elect()) mbar_arrive(&bars->o_free[stage]);
                    quad_transpose(w[0], lane);
                    quad_transpose(w[1], lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int src = (lane & ~3) | k;
                        const long long to_row = __shfl_sync(0xffffffffu, at, src);
                        if (!__shfl_sync(0xffffffffu, (int)valid, src)) continue;
                        uint4 *dst = reinterpret_cast<uint4 *>(p.out + to_row) + (lane & 3);
                        dst[0] = w[0][k];
                        dst[4] = w[1][k];
                    }
                } else {
                    float *part = reinterpret_cast<float *>(static_cast<Tail *>(p.ws) + kAttnCtas) +
                                  (2ll * blockIdx.x + (was.j0 == 0)) * kPieceFloats;
                    uint4 *dst = reinterpret_cast<uint4 *>(part) + (pair * 32 + half * 16) * 32 + lane;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t o[32];
                        tmem_ld32(to + i * 32, o);
                        tmem_ld_wait_regs(o);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[(8 * i + x) * 32] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                    if (half == 0)
                        reinterpret_cast<float2 *>(part + kItemRows * kHeadDim)[pair * 32 + lane] =
                            make_float2(done_m == kUnseen ? -INFINITY : -done_m, done_l);
                    tc_fence_before();
                    __syncwarp();
                    if (elect()) mbar_arrive(&bars->o_free[stage]);
                }
                __syncwarp();
                if (elect()) mbar_arrive(&bars->item_empty[(item - 1) % kItems]);
            }
        }
        if (!live) return;
        done_l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
        done_m = neg_m;
        // The sums take the entries of the largest scores: where those were exchanged for the last tile, the other thread
        // has to have read them.  (For an earlier tile, the votes of the tiles behind it say so.)
        if (state && pair_any(pair, !ok)) return;
        bars->swap[stage][half][row] = done_l;
        if (pair_any(pair, !ok)) return;
        done_l += bars->swap[stage][half ^ 1][row];
    }
}

// What feeds an MMA is the same in every lane and known to be (values from shared memory through a shuffle,
// slots counted instead of divided), so that the uniform datapath forms the operands: otherwise an issue takes 95
// cycles, longer than the MMA (16,384 tokens, 32 heads on 8: 1750 us).
__device__ void mma_role(const AttnParams &p, Bars *bars, uint8_t *sm, uint32_t tbase, int lane,
                         const Waiter &wait) {
    const uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
    const uint32_t id_o = idesc_bf16_f32(128, 128, false, true);
    const uint64_t high = sdesc_sw128(0, 0, 1024);
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0) >> 4;
    const uint32_t q_base = base + (kOffQ >> 4), kv_base = base + (kOffKV >> 4);
    int slot = 0;  // the next tile to come
    uint32_t phase = 0;
    auto full = [&]() { return __all_sync(0xffffffffu, wait(&bars->full[slot], phase)); };
    auto next = [&]() {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
    };
    // S = Q K^T; with tile 1's the keys are done with, with the item's last Q too
    auto scores = [&](int stage, int at_slot, bool last) {
        const uint32_t a = q_base + stage * (kTileBytes >> 4) + (1u << 16);
        const uint32_t b = kv_base + (uint32_t)at_slot * (kTileBytes >> 4) + (1u << 16);
        if (elect()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t at = (k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2;
                mma_bf16(tbase + kTmS + stage * 128, high | (a + at), high | (b + at), id_s, k > 0);
            }
            mma_commit(&bars->s_full[stage]);
            if (stage == 1) {
                mma_commit(&bars->empty[at_slot]);
                if (last) mma_commit(&bars->q_empty);
            }
        }
        __syncwarp();
    };
    bool ok = true;
    uint32_t tile = 0, item = 0;
    while (true) {
        ok = __all_sync(0xffffffffu, wait(&bars->item_full[item % kItems], (item / kItems) & 1));
        if (!ok) break;
        const Rec &it = bars->items[item % kItems];
        const int j0 = __shfl_sync(0xffffffffu, it.j0, 0), nt = __shfl_sync(0xffffffffu, it.j1, 0) - j0;
        const int kv_len = __shfl_sync(0xffffffffu, it.kv_len, 0);
        const int end = kv_len & (p.cache.page_size - 1);
        if (nt <= 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[item % kItems]);
        ok = __all_sync(0xffffffffu, wait(&bars->q_full, item & 1)) && full();
        if (!ok) break;
        tc_fence_after();
        scores(0, slot, nt == 1);
        scores(1, slot, nt == 1);
        next();
        // rows of the last page behind the request's positions hold anything: zeros for the values
        const int last = (kv_len - 1) / kKeyTile - j0;
        for (int j = 0; j < nt && ok; ++j, ++tile) {
            ok = full();
            const int sv = slot;
            next();
            const int sk = slot;
            if (ok && end != 0 && j == last) {
                const int r0 = kv_len - (j0 + j) * kKeyTile, r1 = r0 - end + p.cache.page_size;
                uint8_t *v = sm + kOffKV + sv * kTileBytes;
                for (int r = r0 + (lane >> 4); r < r1; r += 2)
                    *reinterpret_cast<uint4 *>(v + ((lane >> 3) & 1) * kHalfBytes + r * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            const bool more = j + 1 < nt;
#pragma unroll
            for (int stage = 0; stage < 2; ++stage) {
                const uint32_t b = kv_base + (uint32_t)sv * (kTileBytes >> 4) + ((uint32_t)(kHalfBytes >> 4) << 16);
                if (ok && j == 0 && item > 0)  // the last item's O has been read
                    ok = __all_sync(0xffffffffu, wait(&bars->o_free[stage], (item - 1) & 1));
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // keys 0-31 and 64-95, then the others
                    ok = ok && __all_sync(0xffffffffu, wait(&bars->p_full[stage][part], tile & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int k = (x >> 1) * 4 + part * 2 + (x & 1);
                            const uint32_t weights = tbase + kTmS + stage * 128 + (k >> 2) * 64 + (k & 3) * 8;
                            mma_f16_tmem_a(tbase + kTmO + stage * 128, weights, high | (b + k * 128), id_o,
                                           j > 0 || part > 0 || x > 0);
                        }
                        if (part == 1) {
                            if (stage == 1) mma_commit(&bars->empty[sv]);
                            if (!more) mma_commit(&bars->o_full[stage]);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (more) {
                    if (stage == 0) ok = full();
                    if (!ok) break;
                    scores(stage, sk, j + 2 == nt);
                }
            }
            if (more) next();
        }
        if (!ok) break;
        ++item;
    }
    // everything issued is complete before tensor memory is freed
    __syncwarp();
    if (elect()) mma_commit(&bars->drain);
    wait.to_the_end()(&bars->drain, 0);
}

// The tiles that a loading warp fills, every other one of the ring: keys and values in turn.
struct Ring {
    int slot, count = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ Ring(int first) : slot(first) {}
    __device__ __forceinline__ bool load(const AttnParams &p, Bars *bars, uint8_t *sm, const CUtensorMap *map, int page,
                                         int head, const Waiter &wait) {
        // a slot's first phase is filled at once: the wait for the one before it returns
        if (!__all_sync(0xffffffffu, wait(&bars->empty[slot], phase ^ 1))) return false;
        load_tile(map, sm + kOffKV + slot * kTileBytes, &bars->full[slot], page, p.cache.page_size, head);
        ++count;
        slot += 2;
        if (slot >= kSlots) {
            slot -= kSlots;
            phase ^= 1;
        }
        return true;
    }
};

// No copy may be in flight when the CTA exits: the last load into every slot, of those that the two warps made.
__device__ void drain_ring(Bars *bars, const Waiter &wait) {
#pragma unroll 1
    for (int s = 0; s < kSlots; ++s) {
        int last = -1;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv)  // load n of warp kv is number 2 n + kv of the ring
#pragma unroll 1
            for (int n = max(0, bars->loads[kv] - kSlots); n < bars->loads[kv]; ++n)
                if ((2 * n + kv) % kSlots == s) last = max(last, 2 * n + kv);
        if (last >= 0) wait.to_the_end()(&bars->full[s], (uint32_t)(last / kSlots) & 1);
    }
}

// Parents of request b's drafts 4 lane .. 4 lane + 3, kNoParent for the context and for what is out of range; false if
// there is any of those.
__device__ __forceinline__ bool parents_of(const AttnParams &p, int b, int lane, int (&up)[4]) {
    bool sound = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * lane + i, x = t < p.N ? p.parents[(long long)b * p.N + t] : -1;
        const bool good = x >= 0 && x < t;
        sound &= good || x == -1;
        up[i] = good ? x : kNoParent;
    }
    return __all_sync(0xffffffffu, sound);
}

template <bool kTree>
__device__ void load_role(const AttnParams &p, const CUtensorMap *tq, const CUtensorMap *tk, Bars *bars, uint8_t *sm,
                          int lane, const Waiter &wait) {
    const int row_tok = kRowTile / p.group;
    const int box = row_tok * p.group * 128;  // bytes of a box: 64 columns
    uint32_t item = 0, asked = 0;
    Ring ring(0);
    bool ok = true;
    auto publish = [&](const Rec &r) {
        if (item >= kItems)
            ok = ok && __all_sync(0xffffffffu, wait(&bars->item_empty[item % kItems], (item / kItems - 1) & 1));
        if (ok && lane == 0) {
            bars->items[item % kItems] = r;
            mbar_arrive(&bars->item_full[item % kItems]);
        }
        __syncwarp();
    };
    Walk wk(p, bars->work);
    auto leave = [&](int tiles) {
        const Item &it = wk.it;
        if (p.split && lane == 0)
            static_cast<Tail *>(p.ws)[blockIdx.x] = {wk.runs, it.at,   it.size,   tiles, it.b,
                                                     it.kvh,  it.tok0, it.r.t0, it.r.n};
    };
    auto tail = [&]() {
        if constexpr (kTree) {
            int up[4];
            if (!parents_of(p, wk.it.b, lane, up)) return;  // left as it was
        }
        leave(wk.it.tiles);
    };
    leave(0);
    for (; ok && wk.next(p, tail); ++item) {
        const Item &it = wk.it;
        Pages pages;
        pages.fetch(p.cache, it.b, it.r.kv_len, wk.j0, lane);
        Rec r;
        r.b = it.b;
        r.t0 = it.r.t0;
        r.n = it.r.n;
        r.kv_len = it.r.kv_len;
        r.kvh = it.kvh;
        r.tok0 = it.tok0;
        r.j0 = wk.j0;
        r.j1 = wk.j1;
        r.whole = wk.j0 == 0 && wk.j1 == it.tiles;
        r.sound = 1;
        if constexpr (kTree) {
            int up[4];
            r.sound = parents_of(p, it.b, lane, up);
            if (!r.sound && lane == 0) atomicOr(p.err, ERR_BIT_PARENTS);
            if (item >= kItems)  // the slot's last item has been read
                ok = ok && __all_sync(0xffffffffu, wait(&bars->item_empty[item % kItems], (item / kItems - 1) & 1));
            if (ok)
#pragma unroll
                for (int i = 0; i < 4; ++i) bars->parent[item % kItems][4 * lane + i] = (uint8_t)up[i];
            __syncwarp();
        }
        publish(r);
        for (int j = wk.j0; j < wk.j1 && ok; ++j) {
            const int page = pages.check(p.cache, p.err);
            if (j + 1 < wk.j1) pages.fetch(p.cache, it.b, it.r.kv_len, j + 1, lane);
            ok = ring.load(p, bars, sm, tk, page, it.kvh, wait);
            if (j > wk.j0 || !ok) continue;
            // the item's first keys do not wait for the end of the last item's queries
            if (item > 0 && !(ok = __all_sync(0xffffffffu, wait(&bars->q_empty, (item - 1) & 1)))) break;
            if (elect()) {
                mbar_arrive_expect_tx(&bars->q_full, 4 * box);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    tma_load_4d(sm + kOffQ + (x >> 1) * kTileBytes + (x & 1) * kHalfBytes, tq, &bars->q_full, 0,
                                it.kvh * p.group, it.r.t0 + it.tok0 + (x >> 1) * row_tok, x & 1);
            }
            __syncwarp();
            asked = item + 1;
        }
    }
    Rec none = {};
    publish(none);
    // no copy may be in flight when the CTA exits
    if (asked > 0) wait.to_the_end()(&bars->q_full, (asked - 1) & 1);
    if (lane == 0) bars->loads[0] = ring.count;
}

__device__ void value_role(const AttnParams &p, const CUtensorMap *tv, Bars *bars, uint8_t *sm, int lane,
                           const Waiter &wait) {
    Ring ring(1);
    bool ok = true;
    for (uint32_t item = 0; ok; ++item) {
        if (!__all_sync(0xffffffffu, wait(&bars->item_full[item % kItems], (item / kItems) & 1))) break;
        const Rec it = bars->items[item % kItems];
        if (it.j1 <= it.j0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[item % kItems]);
        Pages pages;
        pages.fetch(p.cache, it.b, it.kv_len, it.j0, lane);
        for (int j = it.j0; j < it.j1 && ok; ++j) {
            const int page = pages.check(p.cache, p.err);
            if (j + 1 < it.j1) pages.fetch(p.cache, it.b, it.kv_len, j + 1, lane);
            ok = ring.load(p, bars, sm, tv, page, it.kvh, wait);
        }
    }
    if (lane == 0) bars->loads[1] = ring.count;
}

template <bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
    attn_extend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const AttnParams p) {
    extern __shared__ __align__(1024) uint8_t sm[];  // no room to align it by hand
    Bars *bars = reinterpret_cast<Bars *>(sm + kOffBars);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, kTmCols);
        tmem_relinquish();
    } else if (warp == kLoadWarp) {
        if (lane == 0) {
            for (int i = 0; i < kSlots; ++i) {
                mbar_init(&bars->full[i], 1);
                mbar_init(&bars->empty[i], 1);
            }
            mbar_init(&bars->q_full, 1);
            mbar_init(&bars->q_empty, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars->s_full[i], 1);
                mbar_init(&bars->p_full[i][0], 8);
                mbar_init(&bars->p_full[i][1], 8);
                mbar_init(&bars->o_full[i], 1);
                mbar_init(&bars->o_free[i], 8);
            }
            for (int i = 0; i < kItems; ++i) {
                mbar_init(&bars->item_full[i], 1);
                mbar_init(&bars->item_empty[i], kMmaWarp + 2);
            }
            mbar_init(&bars->drain, 1);
            fence_mbar_init();
        }
    }
    const int rows = kRowTile / p.group * p.group;
    if (warp < kMmaWarp && rows < kRowTile) {  // rows of Q that no box fills
        for (int i = threadIdx.x; i < 4 * (kRowTile - rows) * 8; i += kMmaWarp * 32) {
            const int block = i / ((kRowTile - rows) * 8), at = i - block * (kRowTile - rows) * 8;
            reinterpret_cast<uint4 *>(sm + kOffQ + block * kHalfBytes + rows * 128)[at] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    pdl_wait();
    if (warp < kMmaWarp)
        sum_groups<kMmaWarp>(p.B, bars->work, [&](int x) { return request_work(p, x, tokens_of(p), blockIdx.x == 0); });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    pdl_trigger();  // the join may wait for the end of this grid from here on
    const Waiter wait{p.wait_limit_ns, p.err};
    if (warp < kMmaWarp) {
        reg_inc<kRegsSoftmax>();
        softmax_role<kTree>(p, bars, tbase, warp, lane, wait);
    } else {
        reg_dec<kRegsRest>();
        if (warp == kMmaWarp)
            mma_role(p, bars, sm, tbase, lane, wait);
        else if (warp == kLoadWarp)
            load_role<kTree>(p, &tq, &tk, bars, sm, lane, wait);
        else if (warp == kValueWarp)
            value_role(p, &tv, bars, sm, lane, wait);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tbase, kTmCols);
    if (warp == kLoadWarp) drain_ring(bars, wait);
}

// Joins the items that several CTAs shared, block x the one that CTA x has left for it, block y 32 rows of it:
//     o = sum_i 2^{m_i - m} O_i / sum_i 2^{m_i - m} l_i   over the pieces i, in the CTAs' order.
// A lane has a row, a warp four pieces of four columns; rows go out through shared memory.
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p) {
    __shared__ int list[kAttnCtas], s_count;
    __shared__ __align__(16) uint2 rows[32][33];
    pdl_wait();
    pdl_trigger();
    const Tail t = static_cast<const Tail *>(p.ws)[blockIdx.x];
    if (t.tiles == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const int count = list_pieces(t, blockIdx.x, list, [&](long long done) {
            return done >= t.size ? t.tiles : cut(done, t.tiles);
        });
        if (lane == 0) s_count = count;
    }
    __syncthreads();
    const int count = s_count, row_tok = kRowTile / p.group;
    if (count == 0) return;
    const float *parts = reinterpret_cast<const float *>(static_cast<const Tail *>(p.ws) + kAttnCtas);
    float m = -INFINITY, l = 0.f;
    float4 o[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < count; ++i) {
        const float *part = parts + (long long)list[i] * kPieceFloats;
        const float2 ml = reinterpret_cast<const float2 *>(part + kItemRows * kHeadDim)[blockIdx.y * 32 + lane];
        float4 in[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            in[x] = reinterpret_cast<const float4 *>(part)[(blockIdx.y * 32 + warp * 4 + x) * 32 + lane];
        // a piece whose keys the row does not see has m = -inf and counts for nothing
        const float top = fmaxf(m, ml.x), f = m == -INFINITY ? 0.f : ex2z(m - top);
        const float g = ml.x == -INFINITY ? 0.f : ex2z(ml.x - top);
        m = top;
        l = l * f + ml.y * g;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            o[x].x = o[x].x * f + in[x].x * g;
            o[x].y = o[x].y * f + in[x].y * g;
            o[x].z = o[x].z * f + in[x].z * g;
            o[x].w = o[x].w * f + in[x].w * g;
        }
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        rows[lane][warp * 4 + x] =
            make_uint2(pack_bf16x2(o[x].x * inv, o[x].y * inv), pack_bf16x2(o[x].z * inv, o[x].w * inv));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (blockIdx.y & 3) * 32 + warp * 4 + i, stage = blockIdx.y >> 2;
        const int tok = t.first + stage * row_tok + row / p.group;
        if (row >= row_tok * p.group || tok >= t.n) continue;
        const int h = t.kvh * p.group + row % p.group;
        reinterpret_cast<uint2 *>(p.out + ((long long)(t.t0 + tok) * p.H + h) * kHeadDim)[lane] = rows[warp * 4 + i][lane];
    }
}

}  // namespace

bool make_pages_map(CUtensorMap *m, const void *pages, const CacheParams &c, int Hkv) {
    const unsigned long long extent[5] = {64, (unsigned long long)c.page_size, 2, (unsigned long long)Hkv,
                                          (unsigned long long)c.num_pages};
    const long long stride[5] = {1, kHeadDim, 64, (long long)c.page_size * kHeadDim, c.page_stride};
    const int box[5] = {64, c.page_size, 1, 1, 1};
    return make_bf16_map(m, pages, 5, extent, stride, box, true);
}

bool make_query_map(CUtensorMap *m, const void *q, long long rows, int H, long long row_stride, int group,
                    int tokens) {
    const unsigned long long extent[4] = {64, (unsigned long long)H, (unsigned long long)rows, 2};
    const long long stride[4] = {1, kHeadDim, row_stride, 64};
    const int box[4] = {64, group, tokens, 1};
    return make_bf16_map(m, q, 4, extent, stride, box, true);
}

// Items that see more than two tiles of keys may be cut; otherwise a CTA takes whole ones, in equal numbers.
AttnExtendPlan plan_attn_extend(long long B, long long T, int H, int Hkv, long long max_seqlen,
                                long long max_kvlen) {
    const long long tok = 2 * (kRowTile / (H / Hkv));
    const long long longest = std::min(max_seqlen, T);
    // one at least: where no request may have tokens, a CTA still finds and reports those that have
    const long long items = std::max(std::min(T / tok + std::min(B, T), B * ((longest + tok - 1) / tok)) * Hkv, 1ll);
    const long long pieces = (std::max(max_kvlen, longest) + 2 * kKeyTile - 1) / (2 * kKeyTile);  // of an item
    AttnExtendPlan plan;
    plan.split = pieces > 1;
    plan.ctas = (int)std::min<long long>(items * std::min<long long>(pieces, kAttnCtas), kAttnCtas);
    plan.whole_ctas = (int)std::min<long long>(items, kAttnCtas);
    plan.ws_bytes = plan.split ? kAttnCtas * sizeof(Tail) + 2ull * plan.ctas * kPieceFloats * 4 : 0;
    return plan;
}

cudaError_t launch_attn_extend(const AttnParams &p, const AttnExtendPlan &plan, cudaStream_t stream) {
    const int ctas = p.split ? plan.ctas : plan.whole_ctas;
    CUtensorMap tq, tk, tv;
    if (!make_query_map(&tq, p.q, p.T, p.H, p.q_rs, p.group, kRowTile / p.group) ||
        !make_pages_map(&tk, p.cache.k, p.cache, p.Hkv) || !make_pages_map(&tv, p.cache.v, p.cache, p.Hkv))
        return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::mutex mu;
    static bool configured[64] = {false};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!configured[dev]) {
            e = cudaFuncSetAttribute(attn_extend_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(attn_extend_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    e = launch_pdl(p.parents ? attn_extend_kernel<true> : attn_extend_kernel<false>, dim3((unsigned)ctas), dim3(kThreads),
                   kSmemBytes, stream, tq, tk, tv, p);
    if (e != cudaSuccess || !p.split || ctas == 1) return e;
    return launch_pdl(attn_join_kernel, dim3((unsigned)(ctas - 1), 8), dim3(256), 0, stream, p);
}

}  // namespace la
