// la_attn_verify.cu -- softmax attention of single tokens and of drafted trees over a paged key/value
// cache.  The N drafts of a request are its last N positions; draft t sees the positions before them, its
// ancestors and itself:
//     o_r = sum_j e^{s_rj - m_r} v_j / sum_j e^{s_rj - m_r},   s_rj = scale q_r . k_j
// for the R = (drafts) x (query heads of a kv head) rows r that share the keys, R at most 64 (with more, what is there to
// compute outweighs the loads: la_attn_extend.cu), each key read once.
//
// Bound by HBM: 512 bytes a key and kv head (128 requests of 500 to 8000 positions, 32 heads on 4: 181 to 187 us, 0.93 to
// 0.96 of the copy bandwidth; trees of 8 drafts, 64 requests of 1000 to 8000, 64 heads on 8: 189 to 196 us, 0.85 to
// 0.88, as an item's first tile has to find the references of 64 rows).  The work is the sequence of all tiles of 128 keys, request by
// request and head by head, cut into equal runs, one for each CTA: the SMs finish together whatever the
// lengths.  A run may begin or end inside a (request, head); those leave unnormalised sums, which a second
// launch joins in a fixed order.  Where contexts are short a (request, head) stays with the CTA in whose run it begins.
//
// With few rows the keys take the 128 lanes of the tensor cores: S^T = K Q^T and O^T += V^T P^T, both with
// N = R (padded to 16, 32 or 64), K and V as they lie in their pages.  Two threads share a key in the
// softmax, half of the rows each, and a column of v in the result.  The reference m_r is that of the first tile and
// follows only when a score passes it by more than 2^8, so that a tile takes no maximum, one test.  P goes into
// shared memory as bf16 pairs hi + lo (off by at most 2^-16), which the idle tensor cores take at no cost.
#include <string.h>

#include <algorithm>
#include <mutex>

#include "la_attn.cuh"

namespace la {
namespace {

using namespace attn;

constexpr int kThreads = 384;  // warps 0-7: softmax, 8: MMAs, 9: loads of queries and keys, 10: of values, 11: none
constexpr int kMmaWarp = 8, kLoadWarp = 9, kValueWarp = 10;
constexpr int kRegsSoftmax = 208, kRegsRest = 88;  // a thread, by warp groups, with 64 rows
static_assert(2 * kRegsSoftmax + kRegsRest <= 3 * 168, "register split");
constexpr int kBarSoftmax = 1;
constexpr int kMaxRuns = 2 * kAttnCtas;
constexpr float kUnseen = 1e30f;  // minus the reference of a row that has seen no key: any score passes it, -inf stays

// Two CTAs share an SM where contexts are short, so that one works where the other waits at an item's beginning or end.
template <int RP, int PER_SM>
struct Shape {
    static constexpr int kPerSm = PER_SM;
    static constexpr int kQBufs = 2, kPBufs = RP <= 32 && PER_SM == 1 ? 2 : 1;
    static constexpr int kSlots = PER_SM == 2 ? 3 : RP <= 32 ? 5 : 4;  // tiles of keys and values
    static constexpr int kExtra = RP <= 32 ? 1 : 2;  // tiles' time that an item takes besides its own
    static constexpr uint32_t kQBytes = RP * 256, kPart = kKeyTile * RP * 2, kPBytes = 2 * kPart;
    static constexpr uint32_t kOffKV = 0;
    static constexpr uint32_t kOffQ = kOffKV + kSlots * kTileBytes;
    static constexpr uint32_t kOffP = kOffQ + kQBufs * kQBytes;
    static constexpr uint32_t kOffBars = kOffP + kPBufs * kPBytes;
    static constexpr uint32_t kTmO = 2 * RP, kTmCols = 4 * RP;  // columns of tensor memory: S twice, O
};

// What a CTA's warps have to know of an item, published by the warp that loads the keys; no tiles: the run's end.
struct Rec {
    int b, kvh, kv_len, j0, j1, whole;
};
constexpr int kItems = 4;  // items ahead

template <int RP>
struct Bars {
    uint64_t item_full[kItems], item_empty[kItems];
    Rec items[kItems];
    uint64_t full[5], empty[5];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], p_empty[2], o_full, o_free, drain;
    alignas(16) float neg_m[RP];        // minus the references, in log 2
    alignas(16) float factor[RP];
    union {
        float top[4][RP];
        long long work[kMmaWarp];  // of groups of requests, until the first item is known
    };
    uint8_t tok_of[RP];
    uint32_t below[RP][2];              // below[a] bit t: draft t is a or descends from it
    int loads[2];                       // of keys and of values, at the end
    uint32_t tmem_base;
};

// Tiles of a (request, kv head); 0: no keys, or lengths that do not fit.
__device__ __forceinline__ int tiles_of(const AttnParams &p, int b) {
    const int kv = p.cache.kv_lens[b];
    if (kv < p.N || kv > (long long)p.cache.max_pages * p.cache.page_size) return 0;
    return (kv + kKeyTile - 1) / kKeyTile;
}

// An item is a (request, kv head); its work is its tiles and `extra` more for its beginning and end.
__device__ __forceinline__ int work_of(int tiles, int extra) { return tiles ? tiles + extra : 0; }
// The tile at which the first `done` of an item's work end.
__device__ __forceinline__ int cut(long long done, int tiles) {
    return done <= 0 ? 0 : (int)min((long long)tiles, done);
}

// Work of a request.
__device__ __forceinline__ long long request_work(const AttnParams &p, int b, int extra) {
    return (long long)work_of(tiles_of(p, b), extra) * p.Hkv;
}

// The items of a CTA's run, those of which it has no tile left out.
struct Walk {
    int b, kvh, tiles, j0, j1, kv_len, extra;
    Runs runs;
    long long at, lo, hi;  // where the item begins; the run
    bool begun = false;
    int tail_tiles = 0, tail_b = 0, tail_kvh = 0;  // the item inside which the run ends, if an earlier one does not
    long long tail_at = 0;
    // one warp
    __device__ __forceinline__ Walk(const AttnParams &p, int extra_, const long long (&sums)[kMmaWarp])
        : extra(extra_), runs(0, 1) {
        const Place place(
            sums, p.B, [&](int x) { return request_work(p, x, extra); },
            [&](long long all) {
                runs = Runs(all, (int)max(1ll, min((long long)gridDim.x, all)));
                lo = runs.start(min((int)blockIdx.x, runs.ctas));
                hi = runs.start(min((int)blockIdx.x + 1, runs.ctas));
                return lo;
            });
        if (place.b < 0) hi = lo;  // none behind the last (nor where somebody changes the lengths meanwhile)
        if (lo >= hi) return;
        b = place.b;
        tiles = tiles_of(p, b);
        kv_len = p.cache.kv_lens[b];
        kvh = (int)((lo - place.first) / work_of(tiles, extra));
        at = place.first + (long long)kvh * work_of(tiles, extra);
    }
    __device__ __forceinline__ bool advance(const AttnParams &p) {
        at += work_of(tiles, extra);
        if (at >= hi) return false;
        if (++kvh < p.Hkv) return true;
        kvh = 0;
        do {
            if (++b >= p.B) return false;
            tiles = tiles_of(p, b);
        } while (tiles == 0);
        kv_len = p.cache.kv_lens[b];
        return true;
    }
    // the next item of which a tile is the CTA's; false: there is none
    __device__ __forceinline__ bool next(const AttnParams &p) {
        while (true) {
            if (begun ? !advance(p) : lo >= hi) return false;
            begun = true;
            j0 = p.split ? cut(lo - at, tiles) : at < lo ? tiles : 0;
            j1 = p.split ? cut(hi - at, tiles) : tiles;
            if (at >= lo && at + work_of(tiles, extra) > hi) {
                tail_tiles = tiles;
                tail_b = b;
                tail_kvh = kvh;
                tail_at = at;
            }
            if (j0 < j1) return true;
        }
    }
};

__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kBarSoftmax)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() {
    asm volatile("barrier.cta.sync %0, 256;" ::"n"(kBarSoftmax) : "memory");
}
__device__ __forceinline__ float redux_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Which drafts descend from which; false if a parent is out of range.  256 threads.
template <int RP>
__device__ bool build_tree(const AttnParams &p, Bars<RP> *bars, int b, int tid) {
    softmax_sync();  // the last request's table is not read any more
    if (tid < RP) bars->below[tid][0] = bars->below[tid][1] = 0;
    softmax_sync();
    bool bad = false;
    if (tid < p.N) {
        const int32_t *par = p.parents + (long long)b * p.N;
        int a = tid;
        while (true) {
            atomicOr(&bars->below[a][tid >> 5], 1u << (tid & 31));
            const int up = par[a];
            if (up == -1) break;
            if (up < 0 || up >= a) {
                bad = true;
                break;
            }
            a = up;
        }
    }
    return !softmax_any(bad);
}

// n (8 or a multiple of 16) columns of tensor memory.
template <int n>
__device__ __forceinline__ void tmem_get(uint32_t at, float (&x)[n]) {
    if constexpr (n == 8) {
        uint32_t r[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(at)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < n; i += 16) {
            uint32_t r[16];
            tmem_ld16(at + i, r);
            tmem_ld_wait_regs(r);
#pragma unroll
            for (int y = 0; y < 16; ++y) x[i + y] = __uint_as_float(r[y]);
        }
    }
}
template <int n>
__device__ __forceinline__ void tmem_put(uint32_t at, const float (&x)[n]) {
#pragma unroll
    for (int i = 0; i < n; i += 8) {
        uint32_t r[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) r[y] = __float_as_uint(x[i + y]);
        tmem_st8(at + i, r);
    }
    tmem_st_wait();
}

// Two threads a key: warps 0-3 have the first half of the rows, warps 4-7 the other.
template <int RP, int PER_SM>
__device__ void softmax_role(const AttnParams &p, Bars<RP> *bars, uint8_t *sm, uint32_t tbase, int warp, int lane,
                             const Waiter &wait) {
    using S = Shape<RP, PER_SM>;
    constexpr int R = RP / 2;  // rows of a thread
    const int tid = warp * 32 + lane, key = tid & 127, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const int r0 = half * R;
    const float c = p.scale_log2;
    // rows without keys: a request of no positions
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int kv = p.cache.kv_lens[b];
        if (kv == 0) {
            for (int i = tid; i < p.N * p.H * (kHeadDim / 8); i += 256)
                reinterpret_cast<uint4 *>(p.out + (long long)b * p.N * p.H * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
        } else if (tiles_of(p, b) == 0 && tid == 0) {
            atomicOr(p.err, ERR_BIT_PAGE);
        }
    }
    int tile = 0, tree_of = -1;
    bool ok = true, sound = true;
    float sum[R];  // of this thread's key
    for (int item = 0;; ++item) {
        ok = ok && __all_sync(0xffffffffu, wait(&bars->item_full[item % kItems], (uint32_t)(item / kItems) & 1));
        const Rec w = bars->items[item % kItems];
        if (softmax_any(!ok) || w.j1 <= w.j0) return;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[item % kItems]);
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r] = 0.f;
        if (p.parents && tree_of != w.b) {
            sound = build_tree(p, bars, w.b, tid);
            if (!sound && tid == 0) atomicOr(p.err, ERR_BIT_PARENTS);
            tree_of = w.b;
        }
        const int ctx = w.kv_len - p.N;
        for (int j = w.j0; j < w.j1; ++j, ++tile) {
            const int buf = tile & 1, pbuf = tile % S::kPBufs;
            ok = ok && __all_sync(0xffffffffu, wait(&bars->s_full[buf], (uint32_t)(tile >> 1) & 1));
            tc_fence_after();
            float s[R];  // the scores, then the exponents
            auto fetch = [&]() {
                tmem_get<R>(tbase + lanes + buf * RP + r0, s);
                if ((j + 1) * kKeyTile <= ctx) return;
                // the tile holds drafts, or ends behind the request
                const int d = j * kKeyTile + key - ctx;
                if (d >= p.N) {
#pragma unroll
                    for (int r = 0; r < R; ++r) s[r] = -INFINITY;
                } else if (d >= 0 && p.parents) {
                    const uint32_t see[2] = {bars->below[d][0], bars->below[d][1]};
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int t = min((int)bars->tok_of[r0 + r], kVerifyRows - 1);
                        const uint32_t word = t < 32 ? see[0] : see[1];
                        if (!((word >> (t & 31)) & 1u)) s[r] = -INFINITY;
                    }
                }
            };
            auto exponents = [&]() {
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(&bars->neg_m[r0 + r]);
                    s[r] = fmaf(s[r], c, m.x);
                    s[r + 1] = fmaf(s[r + 1], c, m.y);
                    s[r + 2] = fmaf(s[r + 2], c, m.z);
                    s[r + 3] = fmaf(s[r + 3], c, m.w);
                }
            };
            fetch();
            // against the rows' references; new ones with the first tile and where one is passed by more than 2^8
            const bool first = j == w.j0;
            float far = first ? INFINITY : -INFINITY;
            if (!first) {
                exponents();
#pragma unroll
                for (int r = 0; r < R; r += 4) far = max3(max3(far, s[r], s[r + 1]), s[r + 2], s[r + 3]);
            }
            if (softmax_any(far > 8.f || !ok)) {
                if (!first) fetch();
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float t = redux_max(s[r]);
                    if (lane == 0) bars->top[warp & 3][r0 + r] = t * c;
                }
                if (softmax_any(!ok)) {
                    ok = false;
                    break;
                }
                if (tid < RP) {
                    const float old = first ? kUnseen : bars->neg_m[tid];
                    const float t = fmaxf(fmaxf(bars->top[0][tid], bars->top[1][tid]),
                                          fmaxf(bars->top[2][tid], bars->top[3][tid]));
                    const bool follow = t > -old;  // never where no key is seen
                    bars->factor[tid] = !follow ? 1.f : old == kUnseen ? 0.f : ex2z(-old - t);
                    bars->neg_m[tid] = follow ? -t : old;
                }
                softmax_sync();
                exponents();
#pragma unroll
                for (int r = 0; r < R; ++r) sum[r] *= bars->factor[r0 + r];
                if (!first) {  // O, once the last tile is in it
                    ok = __all_sync(0xffffffffu, wait(&bars->p_empty[(tile - 1) % S::kPBufs],
                                                      (uint32_t)((tile - 1) / S::kPBufs) & 1));
                    tc_fence_after();
                    if (ok) {
                        float o[R];
                        tmem_get<R>(tbase + lanes + S::kTmO + r0, o);
#pragma unroll
                        for (int r = 0; r < R; ++r) o[r] *= bars->factor[r0 + r];
                        tmem_put<R>(tbase + lanes + S::kTmO + r0, o);
                    }
                }
            }
            if (tile >= S::kPBufs)
                ok = ok && __all_sync(0xffffffffu, wait(&bars->p_empty[pbuf], (uint32_t)(tile / S::kPBufs - 1) & 1));
            // groups of 16 rows are 4 KB apart, a key's 32 bytes in pieces of 16, swapped in every other four keys
            uint8_t *ph = sm + S::kOffP + pbuf * S::kPBytes + key * 32;
            const uint32_t turn = ((uint32_t)key >> 2 & 1u) << 4;
#pragma unroll
            for (int g = 0; g < R; g += 8) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int x = 0; x < 8; x += 2) {
                    const float e0 = ex2z(s[g + x]), e1 = ex2z(s[g + x + 1]);
                    sum[g + x] += e0;
                    sum[g + x + 1] += e1;
                    const uint32_t h = pack_bf16x2(e0, e1);
                    hi[x / 2] = h;
                    lo[x / 2] = pack_bf16x2(e0 - __uint_as_float(h << 16), e1 - __uint_as_float(h & 0xffff0000u));
                }
                const int row = r0 + g;
                uint8_t *at = ph + (row >> 4) * 4096 + (turn ^ ((row & 8) ? 16u : 0u));
                *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(at + S::kPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[pbuf]);
        }
        // Where a wait ran out in some warps only, all go on to the next vote: the barriers until there count every thread.
        // The item's sums: over the lanes, each step with half the rows, then over the warps.
        int row = r0;
#pragma unroll
        for (int d = 16, n = R; d > 0; d >>= 1) {
            if (n > 1) {
                n >>= 1;
                const bool up = (lane & d) != 0;
                if (up) row += n;
#pragma unroll
                for (int i = 0; i < R / 2; ++i)
                    if (i < n) {
                        const float mine = up ? sum[i + n] : sum[i], other = up ? sum[i] : sum[i + n];
                        sum[i] = mine + __shfl_xor_sync(0xffffffffu, other, d);
                    }
            } else {
                sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], d);
            }
        }
        bars->top[warp & 3][row] = sum[0];
        softmax_sync();
        // this thread holds column `key` of v
        ok = ok && __all_sync(0xffffffffu, wait(&bars->o_full, (uint32_t)item & 1));
        tc_fence_after();
        const int rows = p.N * p.group;
        const long long piece = 2ll * blockIdx.x + (w.j0 == 0 ? 1 : 0);
        float *po = reinterpret_cast<float *>(static_cast<Tail *>(p.ws) + kMaxRuns) + piece * RP * (kHeadDim + 2);
        if (ok) {
            float o[R], l[R];
            tmem_get<R>(tbase + lanes + S::kTmO + r0, o);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->o_free);
#pragma unroll
            for (int r = 0; r < R; ++r)
                l[r] = (bars->top[0][r0 + r] + bars->top[1][r0 + r]) + (bars->top[2][r0 + r] + bars->top[3][r0 + r]);
            if (!sound) {
            } else if (w.whole) {
                __nv_bfloat16 *to = p.out + ((long long)w.b * p.N * p.H + w.kvh * p.group) * kHeadDim + key;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r0 + r >= rows) break;
                    to[(r0 + r + (int)bars->tok_of[r0 + r] * (p.H - p.group)) * kHeadDim] =
                        __float2bfloat16_rn(l[r] == 0.f ? 0.f : o[r] / l[r]);
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r0 + r >= rows) break;
                    po[(r0 + r) * kHeadDim + key] = o[r];
                }
                if (tid < rows) {
                    const float m = bars->neg_m[tid];
                    reinterpret_cast<float2 *>(po + RP * kHeadDim)[tid] =
                        make_float2(m == kUnseen ? -INFINITY : -m,
                                    (bars->top[0][tid] + bars->top[1][tid]) + (bars->top[2][tid] + bars->top[3][tid]));
                }
            }
        }
        softmax_sync();  // neg_m and the sums are read until here
    }
}

// What feeds an MMA is the same in every lane and known to be (values from shared memory through a shuffle,
// slots counted instead of divided), so that the uniform datapath forms the operands: otherwise an issue takes 100
// cycles, several times the MMA (128 requests of 500-8000 positions, 32 heads on 4: 304 us).
template <int RP, int PER_SM>
__device__ void mma_role(const AttnParams &p, Bars<RP> *bars, uint8_t *sm, uint32_t tbase, int lane,
                         const Waiter &wait) {
    using S = Shape<RP, PER_SM>;
    const uint32_t id_s = idesc_bf16_f32(128, RP, false, false);
    const uint32_t id_o = idesc_bf16_f32(128, RP, true, true);
    const uint64_t high = sdesc_sw128(0, 0, 1024), high32 = sdesc_sw32(0, 0, 256);
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0) >> 4;
    const uint32_t kv_base = base + (S::kOffKV >> 4), q_base = base + (S::kOffQ >> 4);
    const uint32_t p_base = base + (S::kOffP >> 4);
    bool ok = true;
    int slot = 0, qb = 0, pb = 0;  // the next tile, Q and P to come, and the parities of their barriers
    uint32_t slot_par = 0, q_par = 0, p_par = 0;
    uint32_t s_buf = 0;            // of S, for the next scores
    auto next_slot = [&]() {
        if (++slot == S::kSlots) {
            slot = 0;
            slot_par ^= 1;
        }
    };
    // S^T of the next tile; with an item's first tile Q has to be there, with its last Q is done with
    auto scores = [&](bool first, bool last) {
        if (first) ok = ok && __all_sync(0xffffffffu, wait(&bars->q_full[qb], q_par));
        ok = ok && __all_sync(0xffffffffu, wait(&bars->full[slot], slot_par));
        if (!ok) return;
        tc_fence_after();
        const uint32_t a = kv_base + (uint32_t)slot * (kTileBytes >> 4) + (1u << 16);
        const uint32_t b = q_base + (uint32_t)qb * (S::kQBytes >> 4) + (1u << 16);
        if (elect()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_bf16(tbase + s_buf * RP, high | (a + (k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2),
                         high | (b + (k >> 2) * (S::kQBytes >> 5) + (k & 3) * 2), id_s, k > 0);
            mma_commit(&bars->s_full[s_buf]);
            if (last) mma_commit(&bars->q_empty[qb]);
        }
        __syncwarp();
        s_buf ^= 1;
        next_slot();
        if (last) {
            if (++qb == S::kQBufs) {
                qb = 0;
                q_par ^= 1;
            }
        }
    };
    int j0 = 0, j1 = 0, kv_len = 0;
    auto read_item = [&](int x) {  // j1 = j0: there is none
        ok = ok && __all_sync(0xffffffffu, wait(&bars->item_full[x % kItems], (uint32_t)(x / kItems) & 1));
        const Rec &it = bars->items[x % kItems];
        j0 = __shfl_sync(0xffffffffu, it.j0, 0);
        j1 = ok ? __shfl_sync(0xffffffffu, it.j1, 0) : j0;
        kv_len = __shfl_sync(0xffffffffu, it.kv_len, 0);
        __syncwarp();
        if (j0 < j1 && lane == 0) mbar_arrive(&bars->item_empty[x % kItems]);
    };
    int item = 0;
    read_item(0);
    if (j0 < j1) {
        scores(true, j1 - j0 == 1);
        if (elect()) mma_commit(&bars->empty[0]);
        __syncwarp();
    }
    while (j0 < j1 && ok) {
        const int from = j0, to = j1;
        const int end = kv_len & (p.cache.page_size - 1), last = (kv_len - 1) / kKeyTile;
        const int r0 = kv_len - last * kKeyTile, r1 = r0 - end + p.cache.page_size;
        for (int j = from; j < to && ok; ++j) {
            const int sv = slot;  // this tile's values, then the next tile's keys
            const uint32_t sv_par = slot_par;
            next_slot();
            const int sk = slot;
            // the next tile's scores run under this one's softmax; its S was read before the P before was full
            const bool more = j + 1 < to;
            if (!more) read_item(item + 1);
            const bool follows = more || j0 < j1;
            if (follows) scores(!more, more ? j + 2 == to : j1 - j0 == 1);
            ok = ok && __all_sync(0xffffffffu, wait(&bars->full[sv], sv_par));
            if (!ok) break;
            if (end != 0 && j == last) {  // rows of the last page behind the request's positions: zeros
                uint8_t *v = sm + S::kOffKV + sv * kTileBytes;
                for (int r = r0 + (lane >> 4); r < r1; r += 2)
                    *reinterpret_cast<uint4 *>(v + ((lane >> 3) & 1) * kHalfBytes + r * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, wait(&bars->p_full[pb], p_par));
            if (ok && j == from && item > 0)  // the last item's sums have been read
                ok = __all_sync(0xffffffffu, wait(&bars->o_free, (uint32_t)(item - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = kv_base + (uint32_t)sv * (kTileBytes >> 4) + ((uint32_t)(kHalfBytes >> 4) << 16);
            const uint32_t b = p_base + (uint32_t)pb * (S::kPBytes >> 4) + ((4096u >> 4) << 16);
            if (elect()) {
#pragma unroll
                for (int x = 0; x < 2; ++x)  // hi, lo
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t bk = b + x * (S::kPart >> 4) + k * 32;
                        mma_bf16(tbase + S::kTmO, high | (a + k * 128), high32 | bk, id_o, j > from || x + k > 0);
                    }
                // Slots go back in the ring's order, although the keys were done with first: the loading warps, which fill
                // every other one, tell a slot's phases apart by that.
                mma_commit(&bars->empty[sv]);
                if (follows) mma_commit(&bars->empty[sk]);
                mma_commit(&bars->p_empty[pb]);
                if (!more) mma_commit(&bars->o_full);
            }
            __syncwarp();
            if (++pb == S::kPBufs) {
                pb = 0;
                p_par ^= 1;
            }
        }
        ++item;
    }
    __syncwarp();
    if (elect()) mma_commit(&bars->drain);
    wait.to_the_end()(&bars->drain, 0);
}

// The tiles that a loading warp fills, every other one of the ring: keys (kv 0) and values (1).
template <int RP, int PER_SM>
struct Ring {
    using S = Shape<RP, PER_SM>;
    int slot, count = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ Ring(int kv) : slot(kv) {}
    __device__ __forceinline__ bool load(const AttnParams &p, Bars<RP> *bars, uint8_t *sm, const CUtensorMap *map,
                                         int page, int head, const Waiter &wait) {
        // a slot's first phase is filled at once: the wait for the one before it returns
        if (!__all_sync(0xffffffffu, wait(&bars->empty[slot], phase ^ 1))) return false;
        load_tile(map, sm + S::kOffKV + slot * kTileBytes, &bars->full[slot], page, p.cache.page_size, head);
        ++count;
        slot += 2;
        if (slot >= S::kSlots) {
            slot -= S::kSlots;
            phase ^= 1;
        }
        return true;
    }
};

template <int RP, int PER_SM>
__device__ void load_role(const AttnParams &p, const CUtensorMap *tq, const CUtensorMap *tk, Bars<RP> *bars,
                          uint8_t *sm, int lane, const Waiter &wait) {
    using S = Shape<RP, PER_SM>;
    const uint32_t box = (uint32_t)(p.N * p.group) * 128;
    int item = 0, asked = 0;
    Ring<RP, PER_SM> ring(0);
    bool ok = true;
    auto publish = [&](const Rec &r) {
        if (item >= kItems)
            ok = ok && __all_sync(0xffffffffu, wait(&bars->item_empty[item % kItems], (uint32_t)(item / kItems - 1) & 1));
        if (ok && lane == 0) {
            bars->items[item % kItems] = r;
            mbar_arrive(&bars->item_full[item % kItems]);
        }
        __syncwarp();
    };
    Walk w(p, S::kExtra, bars->work);
    for (; ok && w.next(p); ++item) {
        Pages pages;
        pages.fetch(p.cache, w.b, w.kv_len, w.j0, lane);
        publish({w.b, w.kvh, w.kv_len, w.j0, w.j1, w.j0 == 0 && w.j1 == w.tiles});
        const int qb = item % S::kQBufs;
        // a buffer's first phase is filled at once: the wait for the one before it returns
        if (!(ok = ok && __all_sync(0xffffffffu, wait(&bars->q_empty[qb], (uint32_t)(item / S::kQBufs + 1) & 1)))) break;
        if (elect()) {
            mbar_arrive_expect_tx(&bars->q_full[qb], 2 * box);
#pragma unroll
            for (int x = 0; x < 2; ++x)
                tma_load_4d(sm + S::kOffQ + qb * S::kQBytes + x * (S::kQBytes / 2), tq, &bars->q_full[qb], 0,
                            w.kvh * p.group, w.b * p.N, x);
        }
        __syncwarp();
        asked = item + 1;
        for (int j = w.j0; j < w.j1 && ok; ++j) {
            const int page = pages.check(p.cache, p.err);
            if (j + 1 < w.j1) pages.fetch(p.cache, w.b, w.kv_len, j + 1, lane);
            ok = ring.load(p, bars, sm, tk, page, w.kvh, wait);
        }
    }
    if (p.split && lane == 0)
        static_cast<Tail *>(p.ws)[blockIdx.x] = {w.runs, w.tail_at, work_of(w.tail_tiles, w.extra), w.tail_tiles, w.tail_b,
                                                 w.tail_kvh, 0, w.tail_b * p.N, p.N};
    publish({});
    // no copy may be in flight when the CTA exits
    for (int x = asked > S::kQBufs ? asked - S::kQBufs : 0; x < asked; ++x)
        wait.to_the_end()(&bars->q_full[x % S::kQBufs], (uint32_t)(x / S::kQBufs) & 1);
    if (lane == 0) bars->loads[0] = ring.count;
}

template <int RP, int PER_SM>
__device__ void value_role(const AttnParams &p, const CUtensorMap *tv, Bars<RP> *bars, uint8_t *sm, int lane,
                           const Waiter &wait) {
    Ring<RP, PER_SM> ring(1);
    bool ok = true;
    for (int item = 0; ok; ++item) {
        if (!__all_sync(0xffffffffu, wait(&bars->item_full[item % kItems], (uint32_t)(item / kItems) & 1))) break;
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

// The last load into every slot, of those that the two warps made.
template <int RP, int PER_SM>
__device__ void drain_ring(Bars<RP> *bars, const Waiter &wait) {
    constexpr int n_slots = Shape<RP, PER_SM>::kSlots;
#pragma unroll 1
    for (int s = 0; s < n_slots; ++s) {
        int last = -1;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv)  // load n of warp kv is number 2 n + kv of the ring
#pragma unroll 1
            for (int n = max(0, bars->loads[kv] - n_slots); n < bars->loads[kv]; ++n)
                if ((2 * n + kv) % n_slots == s) last = max(last, 2 * n + kv);
        if (last >= 0) wait.to_the_end()(&bars->full[s], (uint32_t)(last / n_slots) & 1);
    }
}

template <int RP, int PER_SM>
__global__ void __launch_bounds__(kThreads, Shape<RP, PER_SM>::kPerSm)
    attn_verify_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const AttnParams p) {
    using S = Shape<RP, PER_SM>;
    extern __shared__ __align__(1024) uint8_t sm[];  // no room to align it by hand
    Bars<RP> *bars = reinterpret_cast<Bars<RP> *>(sm + S::kOffBars);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (warp < kMmaWarp) {
        // rows of Q that no box fills
        for (int i = threadIdx.x; i < (int)(S::kQBufs * S::kQBytes / 16); i += 256)
            reinterpret_cast<uint4 *>(sm + S::kOffQ)[i] = make_uint4(0, 0, 0, 0);
        for (int r = threadIdx.x; r < RP; r += 256) bars->tok_of[r] = (uint8_t)(r / p.group);
        fence_proxy_async_smem();
    } else if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, S::kTmCols);
        tmem_relinquish();
    } else if (warp == kLoadWarp) {
        if (lane == 0) {
            for (int i = 0; i < S::kSlots; ++i) {
                mbar_init(&bars->full[i], 1);
                mbar_init(&bars->empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars->q_full[i], 1);
                mbar_init(&bars->q_empty[i], 1);
                mbar_init(&bars->s_full[i], 1);
                mbar_init(&bars->p_full[i], 8);
                mbar_init(&bars->p_empty[i], 1);
            }
            for (int i = 0; i < kItems; ++i) {
                mbar_init(&bars->item_full[i], 1);
                mbar_init(&bars->item_empty[i], kMmaWarp + 2);
            }
            mbar_init(&bars->o_full, 1);
            mbar_init(&bars->o_free, 8);
            mbar_init(&bars->drain, 1);
            fence_mbar_init();
        }
    }
    pdl_wait();
    if (warp < kMmaWarp) sum_groups<kMmaWarp>(p.B, bars->work, [&](int x) { return request_work(p, x, S::kExtra); });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const Waiter wait{p.wait_limit_ns, p.err};
    if (warp < kMmaWarp) {
        if (RP == 64) reg_inc<kRegsSoftmax>();
        softmax_role<RP, PER_SM>(p, bars, sm, tbase, warp, lane, wait);
    } else {
        if (RP == 64) reg_dec<kRegsRest>();
        if (warp == kMmaWarp)
            mma_role<RP, PER_SM>(p, bars, sm, tbase, lane, wait);
        else if (warp == kLoadWarp)
            load_role<RP, PER_SM>(p, &tq, &tk, bars, sm, lane, wait);
        else if (warp == kValueWarp)
            value_role<RP, PER_SM>(p, &tv, bars, sm, lane, wait);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tbase, S::kTmCols);
    if (warp == kLoadWarp) drain_ring<RP, PER_SM>(bars, wait);
}

// A row's partial results joined: o = sum_i 2^{m_i - m} O_i / sum_i 2^{m_i - m} l_i over the pieces of the list, a lane per
// piece and step, four of their rows in flight; lane l gets columns 4 l .. 4 l + 3.  row(i): where piece i's O row is;
// m and l follow `to_ml` floats behind it.
template <class Row>
__device__ __forceinline__ uint2 join_row(const int *list, int count, long long to_ml, int lane, Row row) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < count; i0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (i0 + lane < count) ml = *reinterpret_cast<const float2 *>(row(list[i0 + lane]) + to_ml);
        float top = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m);
        // a piece whose keys the row does not see has m = -inf and counts for nothing
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
        const int n = min(32, count - i0);
        for (int i = 0; i < n; i += 4) {
            float4 x[4];
            float g[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[k] = __shfl_sync(0xffffffffu, w, (i + k) & 31);  // 0 past the last
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i + k < n && g[k] > 0.f) x[k] = reinterpret_cast<const float4 *>(row(list[i0 + i + k]))[lane];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i + k >= n) break;
                o.x += g[k] * x[k].x;
                o.y += g[k] * x[k].y;
                o.z += g[k] * x[k].z;
                o.w += g[k] * x[k].w;
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    return make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// Joins the items that several CTAs shared, block x the one that CTA x has left for it, a warp per row.  rp: the
// padded rows of a partial result.
__global__ void __launch_bounds__(256) attn_verify_join_kernel(const AttnParams p, int rp) {
    __shared__ int list[kMaxRuns], s_count;
    pdl_wait();
    pdl_trigger();
    const Tail t = static_cast<const Tail *>(p.ws)[blockIdx.x];
    if (t.tiles == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        int count = list_pieces(t, blockIdx.x, list, [&](long long done) { return cut(done, t.tiles); });
        if (p.parents) {  // a request with a parent out of range is left as it was
            bool bad = false;
            for (int i = lane; i < p.N; i += 32) {
                const int up = p.parents[(long long)t.b * p.N + i];
                bad |= up < -1 || up >= i;
            }
            if (__any_sync(0xffffffffu, bad)) count = 0;
        }
        if (lane == 0) s_count = count;
    }
    __syncthreads();
    const int count = s_count;
    if (count == 0) return;
    const int rows = p.N * p.group;
    const float *parts = reinterpret_cast<const float *>(static_cast<const Tail *>(p.ws) + kMaxRuns);
    for (int r = blockIdx.y * 8 + warp; r < rows; r += gridDim.y * 8) {
        const uint2 w = join_row(list, count, (long long)rp * kHeadDim - r * (kHeadDim - 2), lane, [&](int piece) {
            return parts + (long long)piece * rp * (kHeadDim + 2) + r * kHeadDim;
        });
        const int tok = r / p.group, head = t.kvh * p.group + r - tok * p.group;
        reinterpret_cast<uint2 *>(p.out + (((long long)t.t0 + tok) * p.H + head) * kHeadDim)[lane] = w;
    }
}

template <int RP, int PER_SM>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const AttnParams &p,
                   cudaStream_t stream) {
    constexpr uint32_t smem = Shape<RP, PER_SM>::kOffBars + sizeof(Bars<RP>);
    static_assert(Shape<RP, PER_SM>::kPerSm * (smem + 1024) <= 228 * 1024, "shared memory");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::mutex mu;
    static bool configured[64] = {false};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!configured[dev]) {
            e = cudaFuncSetAttribute(attn_verify_kernel<RP, PER_SM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    return launch_pdl(attn_verify_kernel<RP, PER_SM>, dim3(kAttnCtas * Shape<RP, PER_SM>::kPerSm), dim3(kThreads), smem,
                      stream, tq, tk, tv, p);
}

int padded_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// One CTA an SM or two, by what a row of the page table can hold.  One / two, us, 32 heads on 4, 262,144 positions in
// requests of 64 (the first 1024): 95 / 68, 128: 122 / 104, 256: 149 / 135, 384: 129 / 118, 512: 119 / 112, 768: 108 / 106,
// 1024: 103.3 / 102.7, 2048: 98.4 / 99.6; 128 requests of 500-8000: 187 / 189, 2 of 115,000 on 8 heads: 146 / 151.
constexpr long long kShortKeys = 1280;
int per_sm(int rows, long long max_kvlen) { return rows <= 16 && max_kvlen <= kShortKeys ? 2 : 1; }

// Whole (request, head)s, and no second launch, by the same.  Shared out / whole, us in a graph, 32 heads on 8: 1 request of 100
// positions 7.9 / 6.2, of 256 9.0 / 8.8, of 512 9.7 / 11.4, 8 requests 8.4 / 6.7, 10.6 / 10.5, 12.1 / 13.4, 2 trees of 8
// drafts 10.4 / 8.1, 12.2 / 10.3, 13.8 / 12.6; 1024 requests of 128, 32 heads on 4, 89 / 87.
constexpr long long kWholeKeys = 256;

}  // namespace

unsigned long long attn_verify_ws_bytes(int rows, long long max_kvlen) {
    if (max_kvlen <= kWholeKeys) return 0;
    return kMaxRuns * sizeof(Tail) +
           2ull * per_sm(rows, max_kvlen) * kAttnCtas * padded_rows(rows) * (kHeadDim + 2) * 4;
}

cudaError_t launch_attn_verify(const AttnParams &p, cudaStream_t stream) {
    CUtensorMap tq, tk, tv;
    if (!make_query_map(&tq, p.q, (long long)p.B * p.N, p.H, p.q_rs, p.group, p.N) ||
        !make_pages_map(&tk, p.cache.k, p.cache, p.Hkv) || !make_pages_map(&tv, p.cache.v, p.cache, p.Hkv))
        return cudaErrorInvalidValue;
    const int rows = p.N * p.group, rp = padded_rows(rows);
    const int ctas = kAttnCtas * per_sm(rows, (long long)p.cache.max_pages * p.cache.page_size);
    const cudaError_t e = ctas > kAttnCtas ? launch<16, 2>(tq, tk, tv, p, stream)
                          : rp == 16       ? launch<16, 1>(tq, tk, tv, p, stream)
                          : rp == 32       ? launch<32, 1>(tq, tk, tv, p, stream)
                                           : launch<64, 1>(tq, tk, tv, p, stream);
    if (e != cudaSuccess || !p.split) return e;
    return launch_pdl(attn_verify_join_kernel, dim3((unsigned)(ctas - 1), (unsigned)(rp / 16)), dim3(256), 0, stream, p,
                      rp);
}

}  // namespace la
