// la_attn.h -- softmax attention over a paged key/value cache: the launchers of its kernels and
// their parameters (not part of the ABI).
#pragma once

#include "la_internal.h"

// The entry points have checked all sizes, alignments and strides, and the grids fit.
namespace la {

// The cache: position j of request b is row j % page_size of page page_table[b][j / page_size]; element
// (page, kv head, row, d) of k and v is at page * page_stride + (head * page_size + row) * 128 + d.
struct CacheParams {
    __nv_bfloat16 *k, *v;
    long long page_stride;       // elements from one page to the next, both caches
    const int32_t *page_table;   // [B][max_pages]
    const int32_t *kv_lens;      // [B]: positions held, the call's own tokens among them
    int num_pages, page_size, max_pages;
};

// Rotary positions of q and k rows; k (rotated) and v go to cache rows where loc is given, k to k_out
// otherwise.
struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    long long q_rs, k_rs, v_rs;  // elements from one token's row to the next
    const int32_t *positions;    // [T]
    const double *inv_freq;      // [rot / 2], radians per position
    __nv_bfloat16 *q_out, *k_out;
    long long qo_rs, ko_rs;
    CacheParams cache;           // k, v, page_stride, num_pages, page_size
    const int32_t *loc;          // [T]: page * page_size + row, -1: not stored; null: k to k_out, no v
    unsigned int *err;
    float mscale;
    int T, H, Hkv, rot, interleaved;
};
cudaError_t launch_rope(const RopeParams &p, cudaStream_t stream);

struct AttnParams {
    const __nv_bfloat16 *q;      // rows of H heads; query head h reads kv head h / group
    long long q_rs;
    CacheParams cache;
    const int32_t *cu_seqlens;   // [B + 1] (extend), null: N rows per request
    const int32_t *parents;      // [B][N] (tree), null: single tokens
    __nv_bfloat16 *out;          // [T][H * 128]
    void *ws;
    unsigned int *err;
    float scale_log2;            // scale * log2 e, positive
    int B, T, H, Hkv, group, N, max_seqlen;
    int split;                   // whether CTAs may share the keys of a tile of rows, or of a request and kv head
    unsigned long long wait_limit_ns;
};
// Prompts: the tokens of a request are its last positions, each sees those at and before it.
struct AttnExtendPlan {
    int split;                   // with a workspace of ws_bytes
    int ctas, whole_ctas;        // grids with and without
    unsigned long long ws_bytes;
};
AttnExtendPlan plan_attn_extend(long long B, long long T, int H, int Hkv, long long max_seqlen,
                                long long max_kvlen);
cudaError_t launch_attn_extend(const AttnParams &p, const AttnExtendPlan &plan, cudaStream_t stream);

// N drafts (or one token) per request, the last N positions, N * group at most kVerifyRows; more go to
// launch_attn_extend, with cu_seqlens null.  split: where there is a workspace to have (attn_verify_ws_bytes, 0: none).
constexpr int kVerifyRows = 64;
unsigned long long attn_verify_ws_bytes(int rows, long long max_kvlen);
cudaError_t launch_attn_verify(const AttnParams &p, cudaStream_t stream);

struct KvCommitParams {
    CacheParams cache;
    const int32_t *parents;      // [B][N]
    const int32_t *accept_idx;   // [B]
    int32_t *new_lens;           // [B]
    unsigned int *err;
    int B, N, Hkv;
    int keep_lens;               // a skipped request's new_lens is its kv_lens; 0: not written
};
cudaError_t launch_kv_commit(const KvCommitParams &p, cudaStream_t stream);

constexpr int kAttnCtas = 152;       // SMs of a GB300: what schedules and workspaces go by
constexpr int kMaxDrafts = 128;      // drafts of a tree, and query heads that share a kv head
constexpr int kKeyTile = 128;        // keys of a tile
constexpr int kMaxHeads = 1 << 16;   // query heads: 32 bits hold a place among the rows of a request's drafts

}  // namespace la
