// la_attn_extend.cu -- softmax attention of packed prompts over a paged key/value cache (causal,
// grouped heads): for query row i of a request, with the keys at and before its position,
//     o_i = sum_j e^{s_ij - m_i} v_j / sum_j e^{s_ij - m_i},   s_ij = scale q_i . k_j
// in one pass over the keys, m_i a running reference.
//
// A CTA owns two tiles of up to 128 rows -- consecutive tokens x the query heads of one kv head, so
// that the heads of a group share its keys -- and goes over tiles of 128 keys.  Per key tile and row
// tile, S = Q K^T (tcgen05, fp32 in tensor memory), P = exp2(S scale log2 e - m) by one thread per row
// (bf16, back into S's columns), O += P V (P from tensor memory, V as it lies in its page).  While one
// tile's softmax runs, the tensor cores work on the other tile:
//     S0(j) S1(j) | O0 += P0 V, S0(j+1) | O1 += P1 V, S1(j+1) | ...
// Warps 0-3 and 4-7: softmax of tile 0 and 1; warp 8 issues the MMAs; warp 9 loads (TMA, a box per page).
//
// The reference m_i follows the running maximum only when it falls behind by more than 2^8, so that O,
// which lies in tensor memory, is rarely rescaled: P is at most 2^8 and sums stay far inside fp32.
// P is rounded to bf16 (2^-9 of each weight, independent errors: as much as out's own rounding), the sums
// of its values are formed in fp32 before that.
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
constexpr int kThreads = 384;  // warps 10 and 11 wait for the end: registers are shared out by warp groups
constexpr int kRegsSoftmax = 208, kRegsRest = 80;
static_assert(2 * kRegsSoftmax + kRegsRest <= 3 * 168, "register split");
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffKV = kOffQ + 2 * kTileBytes;
constexpr uint32_t kOffBars = kOffKV + kSlots * kTileBytes;

struct Item {
    int b, kvh, t0, n, kv_len, tok0;  // request, kv head, its first row, tokens, positions, first token
    int j0, j1;                       // tiles of keys
    int row_tok;                      // tokens per row tile
    long long index;                  // of the item, for partial results
};

struct Bars {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full, s_full[2], p_full[2], o_full[2], drain;
    Item item;
    int ok;
    uint32_t tmem_base;
};
constexpr uint32_t kSmemBytes = kOffBars + sizeof(Bars) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

constexpr uint32_t kTmS = 0, kTmO = 256, kTmCols = 512;

// Geometry of request b, and whether it is sound.
__device__ __forceinline__ bool request_ok(const AttnParams &p, int b, int &t0, int &n, int &kv_len) {
    t0 = p.cu_seqlens[b];
    const int t1 = p.cu_seqlens[b + 1];
    n = t1 - t0;
    kv_len = p.cache.kv_lens[b];
    return t0 >= 0 && t1 >= t0 && t1 <= p.T && n <= p.max_seqlen && kv_len >= n &&
           kv_len <= (long long)p.cache.max_pages * p.cache.page_size;
}

// The x-th (tile of rows) of the batch, by request and from a request's last tile to its first: one warp.
// CTA 0 goes over all requests and reports the faulty ones.
__device__ bool find_tile(const AttnParams &p, int x, int tok_item, bool report, Item &it) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int t0 = 0, n = 0, kv_len = 0, tiles = 0;
        if (b < p.B) {
            if (request_ok(p, b, t0, n, kv_len))
                tiles = (n + tok_item - 1) / tok_item;
            else if (report)
                atomicOr(p.err, ERR_BIT_SEQLENS);
        }
        int upto = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        upto += before;
        const unsigned hit = __ballot_sync(0xffffffffu, x >= upto - tiles && x < upto);
        if (hit && !found) {
            found = true;
            if (hit & (1u << lane)) {
                it.b = b;
                it.t0 = t0;
                it.n = n;
                it.kv_len = kv_len;
                it.tok0 = (upto - 1 - x) * tok_item;
            }
            const int src = __ffs(hit) - 1;
            it.b = __shfl_sync(0xffffffffu, it.b, src);
            it.t0 = __shfl_sync(0xffffffffu, it.t0, src);
            it.n = __shfl_sync(0xffffffffu, it.n, src);
            it.kv_len = __shfl_sync(0xffffffffu, it.kv_len, src);
            it.tok0 = __shfl_sync(0xffffffffu, it.tok0, src);
        }
        if (found && !report) break;
        before = __shfl_sync(0xffffffffu, upto, 31);
    }
    return found;
}

__device__ void softmax_role(const AttnParams &p, Bars *bars, uint32_t tbase, int stage, int warp, int lane,
                             const Waiter &wait) {
    const Item &it = bars->item;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane quarter, in the address's upper half
    const uint32_t ts = tbase + kTmS + stage * 128 + lanes, to = tbase + kTmO + stage * 128 + lanes;
    const int row = (warp & 3) * 32 + lane;
    const int tok = it.tok0 + stage * it.row_tok + row / p.group, head = row % p.group;
    const bool valid = row < it.row_tok * p.group && tok < it.n;
    // last position that the row sees; rows that are not written take any
    const int limit = it.kv_len - it.n + (valid ? tok : it.n - 1);
    const uint64_t c2 = f2(p.scale_log2, p.scale_log2);
    float m = -INFINITY;
    uint64_t l2[4] = {0, 0, 0, 0};
    bool ok = true;
    for (int j = it.j0; j < it.j1; ++j) {
        ok = __all_sync(0xffffffffu, wait(&bars->s_full[stage], (j - it.j0) & 1));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + i * 32, s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_wait_regs(s[i]);
        const int last = limit - j * kKeyTile;  // columns up to this one are seen
        if (__any_sync(0xffffffffu, last < kKeyTile - 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (i * 32 + x > last) s[i][x] = 0xff800000u;
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top[i] = __uint_as_float(s[i][0]);
#pragma unroll
            for (int x = 1; x < 32; ++x) top[i] = fmaxf(top[i], __uint_as_float(s[i][x]));
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
        const bool behind = mx > m + 8.f;
        if (__any_sync(0xffffffffu, behind)) {
            const float f = behind ? ex2(m - mx) : 1.f;  // 0 from the first visible keys on
            if (behind) m = mx;
            const uint64_t ff = f2(f, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) l2[i] = mul2(l2[i], ff);
            if (j > it.j0) {  // S(j) comes after O += P(j-1) V, which is complete
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    tmem_ld32(to + i * 32, o);
                    tmem_ld_wait_regs(o);
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                    tmem_st32(to + i * 32, o);
                }
            }
        }
        const float sub = m == -INFINITY ? 0.f : -m;
        const uint64_t m2 = f2(sub, sub);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const uint64_t a = fma2(f2(__uint_as_float(s[i][2 * x]), __uint_as_float(s[i][2 * x + 1])), c2, m2);
                float lo, hi;
                f2_get(a, lo, hi);
                lo = ex2(lo);
                hi = ex2(hi);
                l2[x & 3] = add2(l2[x & 3], f2(lo, hi));
                w[x] = pack_bf16x2(lo, hi);
            }
            tmem_st16(ts + i * 16, w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[stage]);
    }
    float la, lb, l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f2_get(l2[i], la, lb);
        l += la + lb;
    }
    const bool any = it.j1 > it.j0;
    if (any) ok = ok && __all_sync(0xffffffffu, wait(&bars->o_full[stage], 0));
    if (!ok) return;
    tc_fence_after();
    if (p.nsplit == 1) {
        const float inv = 1.f / l;
        __nv_bfloat16 *dst = p.out + ((long long)(it.t0 + tok) * p.H + it.kvh * p.group + head) * kHeadDim;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[32];
            tmem_ld32(to + i * 32, o);
            tmem_ld_wait_regs(o);
            if (valid) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        w[y] = pack_bf16x2(__uint_as_float(o[8 * x + 2 * y]) * inv,
                                           __uint_as_float(o[8 * x + 2 * y + 1]) * inv);
                    reinterpret_cast<uint4 *>(dst)[4 * i + x] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        return;
    }
    const long long piece = blockIdx.x, pieces = gridDim.x;
    float *po = static_cast<float *>(p.ws) + (piece * kItemRows + stage * kRowTile + row) * kHeadDim;
    float *ml = static_cast<float *>(p.ws) + pieces * kItemRows * kHeadDim +
                (piece * kItemRows + stage * kRowTile + row) * 2;
    if (valid) *reinterpret_cast<float2 *>(ml) = make_float2(any ? m : -INFINITY, l);
    if (!any) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t o[32];
        tmem_ld32(to + i * 32, o);
        tmem_ld_wait_regs(o);
        if (valid) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                reinterpret_cast<uint4 *>(po)[8 * i + x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
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
    const int j0 = __shfl_sync(0xffffffffu, bars->item.j0, 0), nt = __shfl_sync(0xffffffffu, bars->item.j1, 0) - j0;
    const int kv_len = __shfl_sync(0xffffffffu, bars->item.kv_len, 0);
    int slot = 0;  // the next tile to come
    uint32_t phase = 0;
    auto full = [&]() { return __all_sync(0xffffffffu, wait(&bars->full[slot], phase)); };
    auto next = [&]() {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
    };
    auto scores = [&](int stage, int at_slot) {  // S = Q K^T
        const uint32_t a = q_base + stage * (kTileBytes >> 4) + (1u << 16);
        const uint32_t b = kv_base + (uint32_t)at_slot * (kTileBytes >> 4) + (1u << 16);
        if (elect()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t at = (k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2;
                mma_bf16(tbase + kTmS + stage * 128, high | (a + at), high | (b + at), id_s, k > 0);
            }
            mma_commit(&bars->s_full[stage]);
            if (stage == 1) mma_commit(&bars->empty[at_slot]);
        }
        __syncwarp();
    };
    bool ok = nt > 0 && __all_sync(0xffffffffu, wait(&bars->q_full, 0)) && full();
    if (ok) {
        scores(0, 0);
        scores(1, 0);
        next();
    }
    // rows of the last page behind the request's positions hold anything: zeros for the values
    const int end = kv_len % p.cache.page_size, last = (kv_len - 1) / kKeyTile - j0;
    for (int j = 0; j < nt && ok; ++j) {
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
            ok = ok && __all_sync(0xffffffffu, wait(&bars->p_full[stage], j & 1));
            if (!ok) break;
            tc_fence_after();
            const uint32_t b = kv_base + (uint32_t)sv * (kTileBytes >> 4) + ((uint32_t)(kHalfBytes >> 4) << 16);
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_tmem_a(tbase + kTmO + stage * 128, tbase + kTmS + stage * 128 + k * 8,
                                   high | (b + k * 128), id_o, j > 0 || k > 0);
                if (stage == 1) mma_commit(&bars->empty[sv]);
                if (!more) mma_commit(&bars->o_full[stage]);
            }
            __syncwarp();
            if (more) {
                if (stage == 0) ok = full();
                if (!ok) break;
                scores(stage, sk);
            }
        }
        if (more) next();
    }
    // everything issued is complete before tensor memory is freed
    __syncwarp();
    if (elect()) mma_commit(&bars->drain);
    wait(&bars->drain, 0);
}

__device__ void load_role(const AttnParams &p, const CUtensorMap *tq, const CUtensorMap *tk,
                          const CUtensorMap *tv, Bars *bars, uint8_t *sm, int lane, const Waiter &wait) {
    const Item &it = bars->item;
    const int nt = it.j1 - it.j0;
    if (nt <= 0) return;
    const int box = it.row_tok * p.group * 128;  // bytes of a box: 64 columns
    if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, 4 * box);
        for (int x = 0; x < 4; ++x)
            tma_load_4d(sm + kOffQ + (x >> 1) * kTileBytes + (x & 1) * kHalfBytes, tq, &bars->q_full, 0,
                        it.kvh * p.group, it.t0 + it.tok0 + (x >> 1) * it.row_tok, x & 1);
    }
    int page = page_of(p.cache, it.b, it.kv_len, it.j0, lane, p.err);
    int i = 0;
    bool ok = true;
    for (int j = it.j0; j < it.j1 && ok; ++j) {
        const int next = j + 1 < it.j1 ? page_of(p.cache, it.b, it.kv_len, j + 1, lane, p.err) : 0;
        for (int kv = 0; kv < 2; ++kv, ++i) {
            const int slot = i % kSlots;
            if (i >= kSlots &&
                !(ok = __all_sync(0xffffffffu, wait(&bars->empty[slot], (uint32_t)(i / kSlots - 1) & 1))))
                break;
            load_tile(kv ? tv : tk, sm + kOffKV + slot * kTileBytes, &bars->full[slot], page,
                      p.cache.page_size, it.kvh, lane);
        }
        page = next;
    }
    // no copy may be in flight when the CTA exits
    wait(&bars->q_full, 0);
    for (int x = i > kSlots ? i - kSlots : 0; x < i; ++x) wait(&bars->full[x % kSlots], (uint32_t)(x / kSlots) & 1);
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_extend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const AttnParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars *bars = reinterpret_cast<Bars *>(sm + kOffBars);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    pdl_wait();
    if (warp == 0) {
        Item it;
        it.row_tok = kRowTile / p.group;
        const int split = blockIdx.x % p.nsplit;
        it.index = blockIdx.x / p.nsplit;
        it.kvh = (int)(it.index % p.Hkv);
        const bool ok = find_tile(p, (int)(it.index / p.Hkv), 2 * it.row_tok, blockIdx.x == 0, it);
        if (ok) {
            const int last = min(it.n, it.tok0 + 2 * it.row_tok) - 1;
            const int tiles = (it.kv_len - it.n + last) / kKeyTile + 1;
            it.j0 = (int)((long long)tiles * split / p.nsplit);
            it.j1 = (int)((long long)tiles * (split + 1) / p.nsplit);
        }
        if (lane == 0) {
            if (ok) bars->item = it;
            bars->ok = ok;
        }
    } else if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, kTmCols);
        tmem_relinquish();
    } else if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        mbar_init(&bars->q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->o_full[i], 1);
        }
        mbar_init(&bars->drain, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const Waiter wait{p.wait_limit_ns, p.err};
    if (bars->ok) {
        if (warp < kMmaWarp) {
            reg_inc<kRegsSoftmax>();
            softmax_role(p, bars, tbase, warp >> 2, warp, lane, wait);
        } else {
            reg_dec<kRegsRest>();
            if (warp == kMmaWarp)
                mma_role(p, bars, sm, tbase, lane, wait);
            else if (warp == kLoadWarp)
                load_role(p, &tq, &tk, &tv, bars, sm, lane, wait);
        }
    }
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tbase, kTmCols);
}

// The partial results of a tile's rows, joined: o = sum_s 2^{m_s - m} O_s / sum_s 2^{m_s - m} l_s.  A warp
// per row, in a fixed order.
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p) {
    __shared__ Item item;
    __shared__ int found;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row_tok = kRowTile / p.group;
    const long long index = blockIdx.x;
    if (warp == 0) {
        Item it;
        const bool ok = find_tile(p, (int)(index / p.Hkv), 2 * row_tok, false, it);
        if (lane == 0) {
            if (ok) item = it;
            found = ok;
        }
    }
    __syncthreads();
    if (!found) return;
    const long long pieces = (long long)gridDim.x * p.nsplit;
    const float *po = static_cast<const float *>(p.ws);
    const float2 *ml = reinterpret_cast<const float2 *>(po + pieces * kItemRows * kHeadDim);
    for (int r = blockIdx.y * 8 + warp; r < kItemRows; r += gridDim.y * 8) {
        const int row = r % kRowTile;
        const int tok = item.tok0 + (r / kRowTile) * row_tok + row / p.group;
        if (row >= row_tok * p.group || tok >= item.n) continue;
        // a lane per piece; at most 32 of them
        const float2 mine = lane < p.nsplit ? ml[(index * p.nsplit + lane) * kItemRows + r]
                                            : make_float2(-INFINITY, 0.f);
        float m = mine.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float w = mine.x == -INFINITY ? 0.f : ex2(mine.x - m);
        float l = w * mine.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.nsplit; ++s) {
            const float ws = __shfl_sync(0xffffffffu, w, s);
            if (ws == 0.f) continue;
            const float4 x = reinterpret_cast<const float4 *>(po + ((index * p.nsplit + s) * kItemRows + r) * kHeadDim)[lane];
            o.x += ws * x.x;
            o.y += ws * x.y;
            o.z += ws * x.z;
            o.w += ws * x.w;
        }
        const float inv = 1.f / l;
        const int h = (int)(index % p.Hkv) * p.group + row % p.group;
        const uint2 w2 = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        reinterpret_cast<uint2 *>(p.out + ((long long)(item.t0 + tok) * p.H + h) * kHeadDim)[lane] = w2;
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

// One CTA per pair of row tiles and kv head; where that leaves SMs idle, the keys of each are shared out
// among up to 32 CTAs and a second launch joins their results.
AttnExtendPlan plan_attn_extend(long long B, long long T, int H, int Hkv, long long max_seqlen,
                                long long max_kvlen) {
    const long long tok = 2 * (kRowTile / (H / Hkv));
    const long long longest = std::min(max_seqlen, T);
    const long long tiles = std::min(T / tok + std::min(B, T), B * ((longest + tok - 1) / tok));
    AttnExtendPlan plan;
    plan.items = tiles * Hkv;
    plan.nsplit = 1;
    if (plan.items > 0 && plan.items < kAttnCtas) {
        const long long most = (std::max(max_kvlen, longest) + kKeyTile - 1) / kKeyTile / 4;
        plan.nsplit = (int)std::max(1ll, std::min({kAttnCtas / plan.items, most, 32ll}));
    }
    plan.ws_bytes = plan.nsplit > 1 ? (unsigned long long)plan.items * plan.nsplit * kItemRows * (kHeadDim + 2) * 4 : 0;
    return plan;
}

cudaError_t launch_attn_extend(const AttnParams &p, const AttnExtendPlan &plan, cudaStream_t stream) {
    if (plan.items <= 0) return cudaSuccess;
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
            e = cudaFuncSetAttribute(attn_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    AttnParams pw = p;
    pw.nsplit = plan.nsplit;
    e = launch_pdl(attn_extend_kernel, dim3((unsigned)(plan.items * plan.nsplit)), dim3(kThreads), kSmemBytes,
                   stream, tq, tk, tv, pw);
    if (e != cudaSuccess || plan.nsplit == 1) return e;
    return launch_pdl(attn_join_kernel, dim3((unsigned)plan.items, 4), dim3(256), 0, stream, pw);
}

}  // namespace la
