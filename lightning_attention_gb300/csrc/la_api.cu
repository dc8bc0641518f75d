// la_api.cu -- the extern "C" entry points of the seg_la library (declared in include/la.h):
// host-side argument checks, the per-device error word, and kernel dispatch.  No entry point
// allocates device memory or synchronises, except la_poll_error, which synchronises by design.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "la.h"
#include "la_attn.h"
#include "la_delta.h"
#include "la_extend_bal.h"
#include "la_internal.h"

namespace {

// The extend kernel runs one CTA per (request, head, segment) (la_extend_w.cu).
constexpr int kExtendCtasPerHead = 1;

// Per-device error word: kernels OR bits into it when they find a fault the host cannot see
// (out-of-range slot, inconsistent cu_seqlens, a bounded wait that ran out).  Module-scope
// device variable; its address is looked up once per device and passed to kernels.
__device__ unsigned int g_error_word;

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
unsigned int *g_err_ptr[kMaxDevices] = {nullptr};
std::atomic<unsigned long long> g_wait_limit{0};
std::atomic<int> g_column_split{1};
std::atomic<int> g_persistent{1};
std::atomic<int> g_balanced{1};

// Default bound on a device wait: far above any legitimate wait inside one CTA (microseconds),
// short enough that a lost arrival ends the kernel in about two seconds instead of hanging.
constexpr unsigned long long kDefaultWaitLimitUs = 2000000ull;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// int32, fp32 and uint8 arrays are read element by element: 4-byte alignment (1 for uint8)
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

la_status error_word_ptr(unsigned int **out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return LA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_err_ptr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) return LA_ERR_CUDA;
        g_err_ptr[dev] = static_cast<unsigned int *>(p);
    }
    *out = g_err_ptr[dev];
    return LA_OK;
}

la_status launch_status(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

int g_num_sms[kMaxDevices] = {0};

la_status num_sms(int *out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return LA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_num_sms[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return LA_ERR_CUDA;
        g_num_sms[dev] = n;
    }
    *out = g_num_sms[dev];
    return LA_OK;
}

}  // namespace

extern "C" {

const char *la_status_string(la_status status) {
    switch (status) {
        case LA_OK: return "LA_OK";
        case LA_ERR_INVALID: return "LA_ERR_INVALID: invalid argument";
        case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED: unsupported configuration";
        case LA_ERR_CUDA: return "LA_ERR_CUDA: CUDA runtime or launch error";
        case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT: a bounded device wait ran out";
        case LA_ERR_DEVICE_INPUT:
            return "LA_ERR_DEVICE_INPUT: a device-side index (slot, cu_seqlens, parent, accept "
                   "or track entry, page, cache row or kv_lens) was out of range";
    }
    return "LA_ERR_UNKNOWN";
}

la_status la_slopes(int H, int layer_id, int L, float *host_out) {
    if (H < 1 || L < 1 || layer_id < 0 || layer_id >= L || host_out == nullptr)
        return LA_ERR_INVALID;
    // Per-layer factor from the page's slope rule; ALiBi geometric base 2^(-8 (i+1) / H).
    const double factor =
        (L == 1) ? (1.0 + 1e-5) : (1.0 - (double)layer_id / (double)(L - 1) + 1e-5);
    for (int i = 0; i < H; ++i)
        host_out[i] = (float)(exp2(-8.0 * (double)(i + 1) / (double)H) * factor);
    return LA_OK;
}

void la_set_wait_limit(uint64_t microseconds) { g_wait_limit.store(microseconds); }

void la_set_column_split(int enable) { g_column_split.store(enable ? 1 : 0); }

void la_set_persistent(int enable) { g_persistent.store(enable ? 1 : 0); }

void la_set_balanced(int enable) { g_balanced.store(enable ? 1 : 0); }

la_status la_poll_error(la_stream stream) {
    // The error word is per device, so every kernel that may write it -- on any stream of the
    // device -- has to be finished before it is read: synchronise the stream given (which may
    // belong to another context's default) and then the whole device.
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return LA_ERR_CUDA;
    if (cudaDeviceSynchronize() != cudaSuccess) return LA_ERR_CUDA;
    if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
    unsigned int *err = nullptr;
    la_status st = error_word_ptr(&err);
    if (st != LA_OK) return st;
    unsigned int word = 0;
    if (cudaMemcpy(&word, err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
        return LA_ERR_CUDA;
    if (word != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpy(err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
            return LA_ERR_CUDA;
    }
    if (word & la::ERR_BIT_TIMEOUT) return LA_ERR_TIMEOUT;
    if (word & (la::ERR_BIT_SLOT_RANGE | la::ERR_BIT_SEQLENS | la::ERR_BIT_PARENTS |
                la::ERR_BIT_ACCEPT | la::ERR_BIT_TRACK | la::ERR_BIT_PAGE))
        return LA_ERR_DEVICE_INPUT;
    return LA_OK;
}

la_status la_decode(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, const float *slopes,
                    float *state_pool, int num_slots, const int32_t *state_idx, la_bf16 *out,
                    int B, int H, int D, la_stream stream) {
    if (B < 0 || H < 1 || D < 1 || num_slots < 1) return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !slopes || !state_pool || !state_idx || !out) return LA_ERR_INVALID;
    // the kernel moves q, k, v, the states and out with 16-byte vector accesses
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_pool) ||
        !aligned16(out) || !aligned4(slopes) || !aligned4(state_idx))
        return LA_ERR_INVALID;
    la::RecurParams p{};
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p.v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p.slopes = slopes;
    p.pool = state_pool;
    p.state_idx = state_idx;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.B = B;
    p.H = H;
    p.N = 1;
    p.num_slots = num_slots;
    la_status st = error_word_ptr(&p.err);
    if (st != LA_OK) return st;
    return launch_status(la::launch_recurrent(la::RECUR_DECODE, p, static_cast<cudaStream_t>(stream)));
}

la_status la_verify_chain(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v,
                          const float *slopes, const float *state_pool, int num_slots,
                          const int32_t *state_idx, float *inter_states, la_bf16 *out, int B,
                          int N, int H, int D, la_stream stream) {
    if (B < 0 || N < 1 || H < 1 || D < 1 || num_slots < 1) return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if ((long long)B * N > 0x7fffffffLL) return LA_ERR_INVALID;
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !slopes || !state_pool || !state_idx || !inter_states || !out)
        return LA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_pool) ||
        !aligned16(inter_states) || !aligned16(out) || !aligned4(slopes) || !aligned4(state_idx))
        return LA_ERR_INVALID;
    la::RecurParams p{};
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p.v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p.slopes = slopes;
    p.pool = const_cast<float *>(state_pool);  // read only in verify mode
    p.state_idx = state_idx;
    p.inter = inter_states;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.B = B;
    p.H = H;
    p.N = N;
    p.num_slots = num_slots;
    la_status st = error_word_ptr(&p.err);
    if (st != LA_OK) return st;
    return launch_status(la::launch_recurrent(la::RECUR_VERIFY, p, static_cast<cudaStream_t>(stream)));
}

la_status la_verify_tree(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v,
                         const float *slopes, const float *state_pool, int num_slots,
                         const int32_t *state_idx, const int32_t *parents, float *inter_states,
                         la_bf16 *out, int B, int N, int H, int D, la_stream stream) {
    if (B < 0 || N < 1 || H < 1 || D < 1 || num_slots < 1) return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if ((long long)B * N > 0x7fffffffLL) return LA_ERR_INVALID;
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !slopes || !state_pool || !state_idx || !parents || !inter_states || !out)
        return LA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_pool) ||
        !aligned16(inter_states) || !aligned16(out) || !aligned4(slopes) || !aligned4(state_idx) ||
        !aligned4(parents))
        return LA_ERR_INVALID;
    la::RecurParams p{};
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p.v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p.slopes = slopes;
    p.pool = const_cast<float *>(state_pool);  // read only in tree mode
    p.state_idx = state_idx;
    p.parents = parents;
    p.inter = inter_states;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.B = B;
    p.H = H;
    p.N = N;
    p.num_slots = num_slots;
    la_status st = error_word_ptr(&p.err);
    if (st != LA_OK) return st;
    return launch_status(la::launch_recurrent(la::RECUR_TREE, p, static_cast<cudaStream_t>(stream)));
}

la_status la_commit_accepted(const float *inter_states, const int32_t *accept_idx,
                             float *state_pool, int num_slots, const int32_t *state_idx, int B,
                             int N, int H, int D, la_stream stream) {
    if (B < 0 || N < 1 || H < 1 || D < 1 || num_slots < 1) return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!inter_states || !accept_idx || !state_pool || !state_idx) return LA_ERR_INVALID;
    if (!aligned16(inter_states) || !aligned16(state_pool) || !aligned4(accept_idx) ||
        !aligned4(state_idx))
        return LA_ERR_INVALID;
    la::CommitParams p{};
    p.inter = inter_states;
    p.accept_idx = accept_idx;
    p.pool = state_pool;
    p.state_idx = state_idx;
    p.B = B;
    p.N = N;
    p.H = H;
    p.num_slots = num_slots;
    la_status st = error_word_ptr(&p.err);
    if (st != LA_OK) return st;
    return launch_status(la::launch_commit(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Scratch of an extend call: the split plan's block states and initial-state copies, and for a
// grouped call (Hkv < H) at least the initial-state copies.
struct ExtendScratch {
    la::SplitPlan plan;        // seg_len == 0: no sequence split
    unsigned long long full;   // bytes with the split, before the order array
    unsigned long long copies; // bytes of the initial-state copies alone (grouped calls)
    unsigned long long order;  // bytes of the longest-first order array (large batches), after
                               // `full`
    unsigned long long recs;   // bytes of the persistent extend's request records (batches of
                               // more than one wave), after the order array
    unsigned long long bal;    // bytes of the balanced extend's plan (one-wave batches without a
                               // sequence split), after the records
};

// A one-wave batch runs balanced when its longest request (max_seqlen) is at least this many times
// the mean length T / B.  Balancing reads the keys and values before each cut a second time and
// keeps every SM streaming, which slows each chunk (3.4-3.6 us against 3.05 us); on batches of
// lengths within a factor of about two of each other the column split does as well or better.
constexpr long long kBalancedSkew = 2;

// Up to this many requests every extend CTA ranks the batch itself; above it, a pre-pass ranks
// it once into the workspace.
constexpr int kInCtaRankedRequests = 256;

la_status extend_scratch(int B, int T, int H, int Hkv, int max_seqlen, ExtendScratch *out) {
    *out = ExtendScratch{la::SplitPlan{0, 0, 1, 0, 0ull}, 0ull, 0ull, 0ull, 0ull, 0ull};
    const unsigned long long mat = (unsigned long long)la::kHeadDim * la::kHeadDim * sizeof(float);
    if (Hkv < H) out->copies = (unsigned long long)B * Hkv * mat;
    out->full = out->copies;
    if (B == 0 || T == 0) return LA_OK;
    if (B > kInCtaRankedRequests && B <= la::kMaxRankedRequests)
        out->order = ((unsigned long long)B * sizeof(int32_t) + 15ull) & ~15ull;
    int sms = 0;
    la_status st = num_sms(&sms);
    if (st != LA_OK) return st;
    if (Hkv == H && (long long)B * H > sms && B <= la::kMaxRankedRequests)
        out->recs = (unsigned long long)B * sizeof(la::ItemRec);
    const la::SplitPlan pl = la::plan_split(B, H, max_seqlen, sms, kExtendCtasPerHead);
    if (pl.seg_len > 0) {
        out->plan = pl;
        out->full = (unsigned long long)B * Hkv * (unsigned long long)(1 + pl.nblk) * mat;
    } else if (Hkv == H && B >= 2 && B <= la::kMaxBalRequests && (long long)B * H <= sms &&
               (long long)max_seqlen * B >= kBalancedSkew * (long long)T) {
        out->bal = la::bal_scratch_bytes(B, H);
    }
    return LA_OK;
}

la_status extend_impl(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, const float *slopes,
                      float *state_pool, int num_slots, const int32_t *state_idx,
                      const int32_t *cu_seqlens, const uint8_t *prefix_mask,
                      const int32_t *track_lens, const int32_t *track_state_idx, la_bf16 *out,
                      long long out_rs, long long out_hs, int B, int T, int H, int Hkv, int D,
                      int max_seqlen, void *workspace, size_t workspace_bytes, la_stream stream) {
    if (B < 0 || T < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || D < 1 || num_slots < 1 ||
        max_seqlen < 0)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    // output layout: 16-byte aligned rows and heads that do not overlap (rows of heads, or heads
    // of rows), all inside the 2^40-element range the kernels index
    if (out_rs == 0) out_rs = (long long)H * D;
    if (out_hs == 0) out_hs = D;
    if (out_rs < 0 || out_hs < 0 || out_rs % 8 != 0 || out_hs % 8 != 0) return LA_ERR_INVALID;
    if (out_rs < (long long)(H - 1) * out_hs + D && out_hs < (long long)(T > 0 ? T - 1 : 0) * out_rs + D)
        return LA_ERR_INVALID;
    if (out_rs >= (1ll << 40) || out_hs >= (1ll << 40) ||
        (long long)(T > 0 ? T - 1 : 0) * out_rs + (long long)(H - 1) * out_hs + D >= (1ll << 40))
        return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!slopes || !state_pool || !state_idx || !cu_seqlens || !prefix_mask) return LA_ERR_INVALID;
    if (T > 0 && (!q || !k || !v || !out)) return LA_ERR_INVALID;
    if ((long long)T * H * D >= (1ll << 40)) return LA_ERR_UNSUPPORTED;
    if (workspace != nullptr && !aligned16(workspace)) return LA_ERR_INVALID;
    if (!aligned16(state_pool) || (T > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) ||
                                             !aligned16(out))))
        return LA_ERR_INVALID;
    if (!aligned4(slopes) || !aligned4(state_idx) || !aligned4(cu_seqlens) ||
        (track_lens && (!aligned4(track_lens) || !aligned4(track_state_idx))))
        return LA_ERR_INVALID;
    la_status st;
    la::ExtendParams p{};
    if ((st = error_word_ptr(&p.err)) != LA_OK) return st;
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p.v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p.slopes = slopes;
    p.pool = state_pool;
    p.state_idx = state_idx;
    p.cu_seqlens = cu_seqlens;
    p.prefix_mask = prefix_mask;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.B = B;
    p.T = T;
    p.H = H;
    p.Hkv = Hkv;
    p.group = H / Hkv;
    p.num_slots = num_slots;
    p.max_seqlen = max_seqlen;
    const unsigned long long us = g_wait_limit.load();
    p.wait_limit_ns = (us == 0 ? kDefaultWaitLimitUs : us) * 1000ull;
    p.seg_len = 0;
    p.blk_len = 0;
    p.nseg = 1;
    p.nblk = 0;
    p.ws = nullptr;
    p.lpt = (B > 1 && B <= kInCtaRankedRequests) ? 1 : 0;
    p.order = nullptr;
    p.track_lens = track_lens;
    p.track_idx = track_state_idx;
    p.out_rs = out_rs;
    p.out_hs = out_hs;
    ExtendScratch scr;
    if ((st = extend_scratch(B, T, H, Hkv, max_seqlen, &scr)) != LA_OK) return st;
    // a grouped call cannot run without its initial-state copies
    if (p.group > 1 && (workspace == nullptr || (unsigned long long)workspace_bytes < scr.copies))
        return LA_ERR_INVALID;
    if (p.group > 1) p.ws = static_cast<float *>(workspace);
    if (workspace != nullptr && scr.plan.seg_len > 0 &&
        (unsigned long long)workspace_bytes >= scr.full) {
        p.seg_len = scr.plan.seg_len;
        p.blk_len = scr.plan.blk_len;
        p.nseg = scr.plan.nseg;
        p.nblk = scr.plan.nblk;
        p.ws = static_cast<float *>(workspace);
    }
    // a large batch is taken longest first when the workspace has room for its order
    int32_t *order = nullptr;
    if (workspace != nullptr && scr.order > 0 &&
        (unsigned long long)workspace_bytes >= scr.full + scr.order) {
        order = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + scr.full);
        p.order = order;
        p.lpt = 1;
    }
    // Persistent grid: a batch of more (request, head) pairs than SMs runs on one CTA per SM
    // when the workspace has room for the request records.
    la::ItemRec *recs = nullptr;
    int many_ctas = 0;
    if (workspace != nullptr && scr.recs > 0 && g_persistent.load() &&
        (unsigned long long)workspace_bytes >= scr.full + scr.order + scr.recs) {
        int sms = 0;
        if ((st = num_sms(&sms)) != LA_OK) return st;
        recs = reinterpret_cast<la::ItemRec *>(static_cast<char *>(workspace) + scr.full +
                                               scr.order);
        many_ctas = sms;
    }
    // Column split: SMs that one CTA per (request, head) leaves idle take the second value-column
    // half of the longest requests, H CTAs per request.
    p.csplit = 0;
    if (p.seg_len == 0 && T > 0 && g_column_split.load() && (B == 1 || p.lpt)) {
        int sms = 0;
        if ((st = num_sms(&sms)) != LA_OK) return st;
        const long long spare = (long long)sms - (long long)B * H;
        if (spare >= H) p.csplit = (int)std::min<long long>(B, spare / H);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.recs = nullptr;
    // Balanced grid: a one-wave batch whose requests differ in length runs as segments planned
    // on the device, on one CTA per SM, when the workspace has room for the plan.
    if (workspace != nullptr && scr.bal > 0 && g_balanced.load() && p.seg_len == 0 &&
        p.group == 1 && T > 0 &&
        (unsigned long long)workspace_bytes >= scr.full + scr.order + scr.recs + scr.bal) {
        int sms = 0;
        if ((st = num_sms(&sms)) != LA_OK) return st;
        void *plan = static_cast<char *>(workspace) + scr.full + scr.order + scr.recs;
        return launch_status(la::launch_extend_bal(p, plan, sms, s));
    }
    if (many_ctas > 0 && p.seg_len == 0 && p.csplit == 0 && p.group == 1)
        return launch_status(la::launch_extend_many(p, recs, many_ctas, s));
    if (order != nullptr && la::launch_rank_requests(cu_seqlens, B, order, s) != cudaSuccess)
        return LA_ERR_CUDA;
    if (p.seg_len > 0 || p.group > 1) {
        cudaError_t e = la::launch_block_states(p, s);
        if (e == cudaSuccess) e = la::launch_state_scan(p, s);
        if (e != cudaSuccess) return LA_ERR_CUDA;
    }
    return launch_status(la::launch_extend_wide(p, s));
}

}  // namespace

extern "C" {

la_status la_extend(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, const float *slopes,
                    float *state_pool, int num_slots, const int32_t *state_idx,
                    const int32_t *cu_seqlens, const uint8_t *prefix_mask, la_bf16 *out, int B,
                    int T, int H, int D, int max_seqlen, void *workspace, size_t workspace_bytes,
                    la_stream stream) {
    return extend_impl(q, k, v, slopes, state_pool, num_slots, state_idx, cu_seqlens, prefix_mask,
                       nullptr, nullptr, out, 0, 0, B, T, H, H, D, max_seqlen, workspace,
                       workspace_bytes, stream);
}

la_status la_extend_gqa(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, const float *slopes,
                        float *state_pool, int num_slots, const int32_t *state_idx,
                        const int32_t *cu_seqlens, const uint8_t *prefix_mask, la_bf16 *out,
                        int B, int T, int H, int Hkv, int D, int max_seqlen, void *workspace,
                        size_t workspace_bytes, la_stream stream) {
    return extend_impl(q, k, v, slopes, state_pool, num_slots, state_idx, cu_seqlens, prefix_mask,
                       nullptr, nullptr, out, 0, 0, B, T, H, Hkv, D, max_seqlen, workspace,
                       workspace_bytes, stream);
}

la_status la_extend_gqa_workspace_size(int B, int T, int H, int Hkv, int D, int max_seqlen,
                                       size_t *bytes) {
    if (B < 0 || T < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || D < 1 || max_seqlen < 0 ||
        bytes == nullptr)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    ExtendScratch scr;
    const la_status st = extend_scratch(B, T, H, Hkv, max_seqlen, &scr);
    if (st != LA_OK) return st;
    *bytes = (size_t)(scr.full + scr.order + scr.recs + scr.bal);
    return LA_OK;
}

la_status la_decode_gqa(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, const float *slopes,
                        float *state_pool, int num_slots, const int32_t *state_idx, la_bf16 *out,
                        int B, int H, int Hkv, int D, la_stream stream) {
    if (B < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || D < 1 || num_slots < 1)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if (Hkv == H)  // one query head per state: the plain decode
        return la_decode(q, k, v, slopes, state_pool, num_slots, state_idx, out, B, H, D, stream);
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !slopes || !state_pool || !state_idx || !out) return LA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_pool) ||
        !aligned16(out) || !aligned4(slopes) || !aligned4(state_idx))
        return LA_ERR_INVALID;
    la::RecurParams p{};
    p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p.k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p.v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p.slopes = slopes;
    p.pool = state_pool;
    p.state_idx = state_idx;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.B = B;
    p.H = Hkv;
    p.G = H / Hkv;
    p.N = 1;
    p.num_slots = num_slots;
    la_status st = error_word_ptr(&p.err);
    if (st != LA_OK) return st;
    return launch_status(la::launch_decode_grouped(p, static_cast<cudaStream_t>(stream)));
}

la_status la_extend_ex(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, const float *slopes,
                       float *state_pool, int num_slots, const int32_t *state_idx,
                       const int32_t *cu_seqlens, const uint8_t *prefix_mask,
                       const int32_t *track_lens, const int32_t *track_state_idx, la_bf16 *out,
                       int64_t out_row_stride, int64_t out_head_stride, int B, int T, int H, int D,
                       int max_seqlen, void *workspace, size_t workspace_bytes, la_stream stream) {
    if ((track_lens == nullptr) != (track_state_idx == nullptr)) return LA_ERR_INVALID;
    return extend_impl(q, k, v, slopes, state_pool, num_slots, state_idx, cu_seqlens, prefix_mask,
                       track_lens, track_state_idx, out, (long long)out_row_stride,
                       (long long)out_head_stride, B, T, H, H, D, max_seqlen, workspace,
                       workspace_bytes, stream);
}

la_status la_extend_workspace_size(int B, int T, int H, int D, int max_seqlen, size_t *bytes) {
    if (B < 0 || T < 0 || H < 1 || D < 1 || max_seqlen < 0 || bytes == nullptr)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    ExtendScratch scr;
    const la_status st = extend_scratch(B, T, H, H, max_seqlen, &scr);
    if (st != LA_OK) return st;
    *bytes = (size_t)(scr.full + scr.order + scr.recs + scr.bal);
    return LA_OK;
}

}  // extern "C"

namespace {

// Row stride of a token row of `width` elements: 0 means packed; rows may not overlap and start on
// 16-byte boundaries.  The stride of a single row does not matter.
bool row_stride_ok(int64_t *rs, long long rows, long long width) {
    if (*rs == 0 || rows <= 1) *rs = width;
    return *rs >= width && *rs % 8 == 0;
}

// The grids have B * H CTAs, four times as many, or one per chunk and head.
bool delta_grid_ok(long long B, long long tokens, long long H) {
    return B * H <= 0x1fffffffLL && (tokens / 64 + B) * H <= 0x7fff0000LL;
}

// The checks and the marshalling that the delta entry points share.  `tokens` is their number of
// token rows; work == false: nothing to launch.
la_status delta_params(la::DeltaParams *p, bool *work, const la_bf16 *q, const la_bf16 *k,
                       const la_bf16 *v, int64_t q_rs, int64_t k_rs, int64_t v_rs, const float *g,
                       const float *beta, const float *state_pool, int num_slots,
                       const int32_t *state_idx, la_bf16 *out, int B, long long tokens, int H,
                       int Hk, int D, int qk_l2norm) {
    *work = false;
    if (B < 0 || tokens < 0 || H < 1 || Hk < 1 || H % Hk != 0 || D < 1 || num_slots < 1)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if (tokens > 0x7fffffffLL) return LA_ERR_INVALID;
    if (!row_stride_ok(&q_rs, tokens, (long long)Hk * D) ||
        !row_stride_ok(&k_rs, tokens, (long long)Hk * D) ||
        !row_stride_ok(&v_rs, tokens, (long long)H * D))
        return LA_ERR_INVALID;
    const long long widest = std::max<long long>(std::max<long long>(q_rs, k_rs), v_rs);
    if (widest >= (1ll << 38) || tokens * widest >= (1ll << 40)) return LA_ERR_UNSUPPORTED;
    if (!delta_grid_ok(B, tokens, H)) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!state_pool || !state_idx) return LA_ERR_INVALID;
    if (tokens > 0 && (!q || !k || !v || !g || !beta || !out)) return LA_ERR_INVALID;
    if (!aligned16(state_pool) || !aligned4(state_idx)) return LA_ERR_INVALID;
    if (tokens > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
                       !aligned4(g) || !aligned4(beta)))
        return LA_ERR_INVALID;
    *p = la::DeltaParams{};
    p->q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p->k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p->v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p->q_rs = q_rs;
    p->k_rs = k_rs;
    p->v_rs = v_rs;
    p->g = g;
    p->beta = beta;
    p->pool = const_cast<float *>(state_pool);
    p->state_idx = state_idx;
    p->out = reinterpret_cast<__nv_bfloat16 *>(out);
    p->B = B;
    p->T = (int)tokens;
    p->H = H;
    p->Hk = Hk;
    p->N = 1;
    p->group = H / Hk;
    p->num_slots = num_slots;
    p->l2norm = qk_l2norm != 0;
    const unsigned long long us = g_wait_limit.load();
    p->wait_limit_ns = (us == 0 ? kDefaultWaitLimitUs : us) * 1000ull;
    *work = true;
    return LA_OK;
}

la_status pack_params(la::PackParams *p, bool *work, const float *state_pool, int num_slots,
                      const int32_t *state_idx, const int8_t *codes, const uint8_t *scales,
                      int entries, const int32_t *store_idx, int B, int H, int D) {
    *work = false;
    if (B < 0 || H < 1 || D < 1 || num_slots < 1 || entries < 1) return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if ((long long)B * H > 0x7fffffffLL) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!state_pool || !state_idx || !codes || !scales || !store_idx) return LA_ERR_INVALID;
    if (!aligned16(state_pool) || !aligned16(codes) || !aligned4(scales) || !aligned4(state_idx) ||
        !aligned4(store_idx))
        return LA_ERR_INVALID;
    *p = la::PackParams{};
    p->pool = const_cast<float *>(state_pool);
    p->state_idx = state_idx;
    p->codes = const_cast<int8_t *>(codes);
    p->scales = const_cast<uint8_t *>(scales);
    p->store_idx = store_idx;
    p->B = B;
    p->H = H;
    p->num_slots = num_slots;
    p->entries = entries;
    const la_status st = error_word_ptr(&p->err);
    if (st != LA_OK) return st;
    *work = true;
    return LA_OK;
}

}  // namespace

extern "C" {

la_status la_delta_extend(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, int64_t q_row_stride,
                          int64_t k_row_stride, int64_t v_row_stride, const float *g,
                          const float *beta, float *state_pool, int num_slots,
                          const int32_t *state_idx, const int32_t *cu_seqlens,
                          const uint8_t *prefix_mask, la_bf16 *out, int B, int T, int H, int Hk,
                          int D, int max_seqlen, int qk_l2norm, void *workspace,
                          size_t workspace_bytes, la_stream stream) {
    la::DeltaParams p;
    bool work;
    if (max_seqlen < 0) return LA_ERR_INVALID;
    la_status st = delta_params(&p, &work, q, k, v, q_row_stride, k_row_stride, v_row_stride, g, beta,
                                state_pool, num_slots, state_idx, out, B, T, H, Hk, D, qk_l2norm);
    if (st != LA_OK || !work) return st;
    if (!cu_seqlens || !prefix_mask || !aligned4(cu_seqlens)) return LA_ERR_INVALID;
    // a few tokens a request: token by token, without chunks
    const bool serial = std::min(max_seqlen, T) <= la::kSerialTokens;
    const unsigned long long need = serial ? 0ull : la::delta_scratch_bytes(B, T, H);
    if (need > 0 && (!workspace || !aligned16(workspace) || (unsigned long long)workspace_bytes < need))
        return LA_ERR_INVALID;
    p.cu_seqlens = cu_seqlens;
    p.prefix_mask = prefix_mask;
    p.max_seqlen = max_seqlen;
    int sms = 0;
    if ((st = error_word_ptr(&p.err)) != LA_OK || (st = num_sms(&sms)) != LA_OK) return st;
    if (serial)
        return launch_status(la::launch_delta_recurrent(la::DELTA_SERIAL, p, sms,
                                                        static_cast<cudaStream_t>(stream)));
    return launch_status(la::launch_delta_extend(p, workspace, sms, static_cast<cudaStream_t>(stream)));
}

la_status la_delta_extend_workspace_size(int B, int T, int H, int D, size_t *bytes) {
    if (B < 0 || T < 0 || H < 1 || D < 1 || bytes == nullptr) return LA_ERR_INVALID;
    if (D != la::kHeadDim || !delta_grid_ok(B, T, H)) return LA_ERR_UNSUPPORTED;
    *bytes = (size_t)la::delta_scratch_bytes(B, T, H);
    return LA_OK;
}

la_status la_delta_decode(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, int64_t q_row_stride,
                          int64_t k_row_stride, int64_t v_row_stride, const float *g,
                          const float *beta, float *state_pool, int num_slots,
                          const int32_t *state_idx, la_bf16 *out, int B, int H, int Hk, int D,
                          int qk_l2norm, la_stream stream) {
    la::DeltaParams p;
    bool work;
    la_status st = delta_params(&p, &work, q, k, v, q_row_stride, k_row_stride, v_row_stride, g, beta,
                                state_pool, num_slots, state_idx, out, B, B, H, Hk, D, qk_l2norm);
    if (st != LA_OK || !work) return st;
    int sms = 0;
    if ((st = error_word_ptr(&p.err)) != LA_OK || (st = num_sms(&sms)) != LA_OK) return st;
    return launch_status(la::launch_delta_recurrent(la::DELTA_DECODE, p, sms,
                                                    static_cast<cudaStream_t>(stream)));
}

la_status la_delta_verify_chain(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v,
                                int64_t q_row_stride, int64_t k_row_stride, int64_t v_row_stride,
                                const float *g, const float *beta, const float *state_pool,
                                int num_slots, const int32_t *state_idx, float *inter_states,
                                la_bf16 *out, int B, int N, int H, int Hk, int D, int qk_l2norm,
                                la_stream stream) {
    la::DeltaParams p;
    bool work;
    if (N < 1) return LA_ERR_INVALID;
    la_status st = delta_params(&p, &work, q, k, v, q_row_stride, k_row_stride, v_row_stride, g, beta,
                                state_pool, num_slots, state_idx, out, B, (long long)B * N, H, Hk, D,
                                qk_l2norm);
    if (st != LA_OK || !work) return st;
    if (!inter_states || !aligned16(inter_states)) return LA_ERR_INVALID;
    p.N = N;
    p.inter = inter_states;
    int sms = 0;
    if ((st = error_word_ptr(&p.err)) != LA_OK || (st = num_sms(&sms)) != LA_OK) return st;
    return launch_status(la::launch_delta_recurrent(la::DELTA_VERIFY, p, sms,
                                                    static_cast<cudaStream_t>(stream)));
}

la_status la_pack_states(const float *state_pool, int num_slots, const int32_t *state_idx,
                         int8_t *codes, uint8_t *scales, int entries, const int32_t *store_idx, int B,
                         int H, int D, la_stream stream) {
    la::PackParams p;
    bool work;
    const la_status st = pack_params(&p, &work, state_pool, num_slots, state_idx, codes, scales,
                                     entries, store_idx, B, H, D);
    if (st != LA_OK || !work) return st;
    return launch_status(la::launch_pack_states(p, static_cast<cudaStream_t>(stream)));
}

la_status la_unpack_states(const int8_t *codes, const uint8_t *scales, int entries,
                           const int32_t *store_idx, float *state_pool, int num_slots,
                           const int32_t *state_idx, int B, int H, int D, la_stream stream) {
    la::PackParams p;
    bool work;
    const la_status st = pack_params(&p, &work, state_pool, num_slots, state_idx, codes, scales,
                                     entries, store_idx, B, H, D);
    if (st != LA_OK || !work) return st;
    return launch_status(la::launch_unpack_states(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// A cache's checks that need no device.  `lists`: whether the call has a page table and lengths.
la_status cache_params(la::CacheParams *c, const la_bf16 *k_pages, const la_bf16 *v_pages,
                       int64_t page_stride, int num_pages, int page_size, const int32_t *page_table,
                       int max_pages, const int32_t *kv_lens, int Hkv, int D, bool lists) {
    if (num_pages < 1 || page_size < 1 || Hkv < 1 || D < 1 || (lists && max_pages < 1)) return LA_ERR_INVALID;
    if (D != la::kHeadDim) return LA_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return LA_ERR_UNSUPPORTED;
    const long long page = (long long)Hkv * page_size * la::kHeadDim;
    if (page_stride == 0) page_stride = page;
    if (page_stride < page || page_stride % 8 != 0) return LA_ERR_INVALID;
    if (page_stride >= (1ll << 38) || (long long)num_pages * page_stride >= (1ll << 44)) return LA_ERR_UNSUPPORTED;
    if (lists && (long long)max_pages * page_size > (1ll << 30)) return LA_ERR_UNSUPPORTED;
    *c = la::CacheParams{};
    c->k = reinterpret_cast<__nv_bfloat16 *>(const_cast<la_bf16 *>(k_pages));
    c->v = reinterpret_cast<__nv_bfloat16 *>(const_cast<la_bf16 *>(v_pages));
    c->page_stride = page_stride;
    c->page_table = page_table;
    c->kv_lens = kv_lens;
    c->num_pages = num_pages;
    c->page_size = page_size;
    c->max_pages = max_pages;
    return LA_OK;
}

bool cache_pointers_ok(const la::CacheParams &c, bool lists) {
    if (!c.k || !c.v || !aligned16(c.k) || !aligned16(c.v)) return false;
    return !lists || (c.page_table && c.kv_lens && aligned4(c.page_table) && aligned4(c.kv_lens));
}

la_status rope_params(la::RopeParams *p, const la_bf16 *q, const la_bf16 *k, int64_t q_rs, int64_t k_rs,
                      const int32_t *positions, const double *inv_freq, int rot_dim, int interleaved,
                      float mscale, la_bf16 *q_out, int64_t qo_rs, int T, int H, int Hkv, int D) {
    if (T < 0 || H < 1 || Hkv < 1 || D < 1 || rot_dim < 0 || rot_dim > D || !isfinite(mscale))
        return LA_ERR_INVALID;
    if (D != la::kHeadDim || rot_dim % 16 != 0) return LA_ERR_UNSUPPORTED;
    const long long rows = (long long)H + 2ll * Hkv;  // of a token, at most
    if (rows > 0x7fff0000LL / la::kHeadDim || rows * T > (1ll << 36)) return LA_ERR_UNSUPPORTED;
    if (!row_stride_ok(&q_rs, T, (long long)H * D) || !row_stride_ok(&k_rs, T, (long long)Hkv * D) ||
        !row_stride_ok(&qo_rs, T, (long long)H * D))
        return LA_ERR_INVALID;
    *p = la::RopeParams{};
    p->q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p->k = reinterpret_cast<const __nv_bfloat16 *>(k);
    p->q_rs = q_rs;
    p->k_rs = k_rs;
    p->positions = positions;
    p->inv_freq = inv_freq;
    p->q_out = reinterpret_cast<__nv_bfloat16 *>(q_out);
    p->qo_rs = qo_rs;
    p->mscale = mscale;
    p->T = T;
    p->H = H;
    p->Hkv = Hkv;
    p->rot = rot_dim;
    p->interleaved = interleaved != 0;
    return LA_OK;
}

bool rope_pointers_ok(const la::RopeParams &p) {
    if (!p.q || !p.k || !p.q_out || !p.positions || (p.rot > 0 && !p.inv_freq)) return false;
    return aligned16(p.q) && aligned16(p.k) && aligned16(p.q_out) && aligned4(p.positions) &&
           (reinterpret_cast<uintptr_t>(p.inv_freq) & 7u) == 0;
}

constexpr float kLog2e = 1.4426950408889634f;

// Checks shared by the attention calls, of `tokens` rows; work == false: nothing to launch.
la_status attn_params(la::AttnParams *p, bool *work, const la_bf16 *q, int64_t q_rs, const la::CacheParams &c,
                      la_bf16 *out, int B, long long tokens, int H, int Hkv, float scale) {
    *work = false;
    if (B < 0 || tokens < 0 || H < 1 || H % Hkv != 0 || !(scale > 0.f) || !isfinite(scale * kLog2e))
        return LA_ERR_INVALID;
    if (tokens > 0x7fffffffLL) return LA_ERR_INVALID;
    if (H > la::kMaxHeads || H / Hkv > la::kMaxDrafts) return LA_ERR_UNSUPPORTED;
    if (!row_stride_ok(&q_rs, tokens, (long long)H * la::kHeadDim)) return LA_ERR_INVALID;
    if (q_rs >= (1ll << 38)) return LA_ERR_UNSUPPORTED;
    if (B == 0 || tokens == 0) return LA_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out) || !cache_pointers_ok(c, true)) return LA_ERR_INVALID;
    *p = la::AttnParams{};
    p->q = reinterpret_cast<const __nv_bfloat16 *>(q);
    p->q_rs = q_rs;
    p->cache = c;
    p->out = reinterpret_cast<__nv_bfloat16 *>(out);
    p->scale_log2 = scale * kLog2e;
    p->B = B;
    p->T = (int)tokens;
    p->H = H;
    p->Hkv = Hkv;
    p->group = H / Hkv;
    p->N = 1;
    const unsigned long long us = g_wait_limit.load();
    p->wait_limit_ns = (us == 0 ? kDefaultWaitLimitUs : us) * 1000ull;
    *work = true;
    return LA_OK;
}

la_status attn_verify(const la_bf16 *q, int64_t q_rs, const la_bf16 *k_pages, const la_bf16 *v_pages,
                      int64_t page_stride, int num_pages, int page_size, const int32_t *page_table, int max_pages,
                      const int32_t *kv_lens, const int32_t *parents, bool tree, la_bf16 *out, int B, int N, int H,
                      int Hkv, int D, float scale, void *workspace, size_t workspace_bytes, la_stream stream) {
    la::CacheParams c;
    la::AttnParams p;
    bool work;
    la_status st = cache_params(&c, k_pages, v_pages, page_stride, num_pages, page_size, page_table, max_pages,
                                kv_lens, Hkv, D, true);
    if (st != LA_OK) return st;
    if (N < 1) return LA_ERR_INVALID;
    if (N > la::kMaxDrafts) return LA_ERR_UNSUPPORTED;
    st = attn_params(&p, &work, q, q_rs, c, out, B, (long long)B * N, H, Hkv, scale);
    if (st != LA_OK || !work) return st;
    if (tree && (!parents || !aligned4(parents))) return LA_ERR_INVALID;
    const bool few = N * p.group <= la::kVerifyRows;
    const la::AttnExtendPlan plan = la::plan_attn_extend(B, p.T, H, Hkv, N, (long long)max_pages * page_size);
    const unsigned long long need =
        few ? la::attn_verify_ws_bytes(N * p.group, (long long)max_pages * page_size) : plan.ws_bytes;
    if (!aligned16(workspace) || (need > 0 && (!workspace || (unsigned long long)workspace_bytes < need)))
        return LA_ERR_INVALID;
    p.parents = tree ? parents : nullptr;
    p.N = N;
    p.ws = workspace;
    p.max_seqlen = N;
    p.split = need > 0;
    if ((st = error_word_ptr(&p.err)) != LA_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_status(few ? la::launch_attn_verify(p, s) : la::launch_attn_extend(p, plan, s));
}

}  // namespace

extern "C" {

la_status la_rope_freqs(int rot_dim, double base, la_rope_scaling scaling, double factor, int orig_len,
                        double beta_fast, double beta_slow, double *host_inv_freq, float *host_mscale) {
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !isfinite(base) || !host_inv_freq || !host_mscale)
        return LA_ERR_INVALID;
    if (scaling < LA_ROPE_PLAIN || scaling > LA_ROPE_YARN) return LA_ERR_INVALID;
    if (scaling != LA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return LA_ERR_INVALID;
    if (scaling == LA_ROPE_YARN &&
        (orig_len < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0) || !isfinite(beta_fast)))
        return LA_ERR_INVALID;
    if (scaling == LA_ROPE_NTK && rot_dim > 2) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    // the (real) index of the pair that turns `turns` times over the original length
    auto index_of = [&](double turns) {
        return rot_dim * log(orig_len / (turns * 6.283185307179586477)) / (2.0 * log(base));
    };
    double lo = 0.0, hi = 0.0;
    if (scaling == LA_ROPE_YARN) {
        lo = std::max(floor(index_of(beta_fast)), 0.0);
        hi = std::min(ceil(index_of(beta_slow)), (double)(rot_dim - 1));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == LA_ROPE_LINEAR) f /= factor;
        if (scaling == LA_ROPE_YARN) {
            // behind the ramp everything is interpolated, where it ends before pair 0 too
            const double ramp = i >= hi ? 1.0 : std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        host_inv_freq[i] = f;
    }
    *host_mscale = scaling == LA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return LA_OK;
}

la_status la_rope(const la_bf16 *q, const la_bf16 *k, int64_t q_row_stride, int64_t k_row_stride,
                  const int32_t *positions, const double *inv_freq, int rot_dim, int interleaved, float mscale,
                  la_bf16 *q_out, la_bf16 *k_out, int64_t q_out_row_stride, int64_t k_out_row_stride, int T, int H,
                  int Hkv, int D, la_stream stream) {
    la::RopeParams p;
    const la_status st = rope_params(&p, q, k, q_row_stride, k_row_stride, positions, inv_freq, rot_dim, interleaved,
                                     mscale, q_out, q_out_row_stride, T, H, Hkv, D);
    if (st != LA_OK) return st;
    if (!row_stride_ok(&k_out_row_stride, T, (long long)Hkv * D)) return LA_ERR_INVALID;
    if (T == 0) return LA_OK;
    if (!rope_pointers_ok(p) || !k_out || !aligned16(k_out)) return LA_ERR_INVALID;
    p.k_out = reinterpret_cast<__nv_bfloat16 *>(k_out);
    p.ko_rs = k_out_row_stride;
    return launch_status(la::launch_rope(p, static_cast<cudaStream_t>(stream)));
}

la_status la_kv_store(const la_bf16 *q, const la_bf16 *k, const la_bf16 *v, int64_t q_row_stride,
                      int64_t k_row_stride, int64_t v_row_stride, const int32_t *positions, const double *inv_freq,
                      int rot_dim, int interleaved, float mscale, la_bf16 *q_out, int64_t q_out_row_stride,
                      la_bf16 *k_pages, la_bf16 *v_pages, int64_t page_stride, int num_pages, int page_size,
                      const int32_t *loc, int T, int H, int Hkv, int D, la_stream stream) {
    la::RopeParams p;
    la_status st = rope_params(&p, q, k, q_row_stride, k_row_stride, positions, inv_freq, rot_dim, interleaved, mscale,
                               q_out, q_out_row_stride, T, H, Hkv, D);
    if (st != LA_OK) return st;
    st = cache_params(&p.cache, k_pages, v_pages, page_stride, num_pages, page_size, nullptr, 0, nullptr, Hkv, D, false);
    if (st != LA_OK) return st;
    if (!row_stride_ok(&v_row_stride, T, (long long)Hkv * D)) return LA_ERR_INVALID;
    if (T == 0) return LA_OK;
    if (!rope_pointers_ok(p) || !v || !aligned16(v) || !loc || !aligned4(loc) || !cache_pointers_ok(p.cache, false))
        return LA_ERR_INVALID;
    p.v = reinterpret_cast<const __nv_bfloat16 *>(v);
    p.v_rs = v_row_stride;
    p.loc = loc;
    if ((st = error_word_ptr(&p.err)) != LA_OK) return st;
    return launch_status(la::launch_rope(p, static_cast<cudaStream_t>(stream)));
}

la_status la_attn_extend_workspace_size(int B, int T, int H, int Hkv, int D, int max_seqlen, int max_kvlen,
                                        size_t *bytes) {
    if (B < 0 || T < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || D < 1 || max_seqlen < 0 || max_kvlen < 0 ||
        bytes == nullptr)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim || H > la::kMaxHeads || H / Hkv > la::kMaxDrafts) return LA_ERR_UNSUPPORTED;
    *bytes = (size_t)la::plan_attn_extend(B, T, H, Hkv, max_seqlen, max_kvlen).ws_bytes;
    return LA_OK;
}

la_status la_attn_extend(const la_bf16 *q, int64_t q_row_stride, const la_bf16 *k_pages, const la_bf16 *v_pages,
                         int64_t page_stride, int num_pages, int page_size, const int32_t *page_table, int max_pages,
                         const int32_t *cu_seqlens, const int32_t *kv_lens, la_bf16 *out, int B, int T, int H,
                         int Hkv, int D, int max_seqlen, int max_kvlen, float scale, void *workspace,
                         size_t workspace_bytes, la_stream stream) {
    la::CacheParams c;
    la::AttnParams p;
    bool work;
    la_status st = cache_params(&c, k_pages, v_pages, page_stride, num_pages, page_size, page_table, max_pages,
                                kv_lens, Hkv, D, true);
    if (st != LA_OK) return st;
    if (max_seqlen < 0 || max_kvlen < 0) return LA_ERR_INVALID;
    st = attn_params(&p, &work, q, q_row_stride, c, out, B, T, H, Hkv, scale);
    if (st != LA_OK || !work) return st;
    if (!cu_seqlens || !aligned4(cu_seqlens) || !aligned16(workspace)) return LA_ERR_INVALID;
    const la::AttnExtendPlan plan = la::plan_attn_extend(B, T, H, Hkv, max_seqlen, max_kvlen);
    p.split = plan.split && workspace && (unsigned long long)workspace_bytes >= plan.ws_bytes;
    p.cu_seqlens = cu_seqlens;
    p.max_seqlen = max_seqlen;
    p.ws = workspace;
    if ((st = error_word_ptr(&p.err)) != LA_OK) return st;
    return launch_status(la::launch_attn_extend(p, plan, static_cast<cudaStream_t>(stream)));
}

la_status la_attn_verify_workspace_size(int B, int N, int H, int Hkv, int D, int max_kvlen, size_t *bytes) {
    if (B < 0 || N < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || D < 1 || max_kvlen < 0 || bytes == nullptr)
        return LA_ERR_INVALID;
    if (D != la::kHeadDim || N > la::kMaxDrafts || H > la::kMaxHeads || H / Hkv > la::kMaxDrafts)
        return LA_ERR_UNSUPPORTED;
    const int rows = N * (H / Hkv);
    *bytes = (size_t)(B == 0                      ? 0
                      : rows <= la::kVerifyRows ? la::attn_verify_ws_bytes(rows, max_kvlen)
                                                  : la::plan_attn_extend(B, (long long)B * N, H, Hkv, N, max_kvlen).ws_bytes);
    return LA_OK;
}

la_status la_attn_decode(const la_bf16 *q, int64_t q_row_stride, const la_bf16 *k_pages, const la_bf16 *v_pages,
                         int64_t page_stride, int num_pages, int page_size, const int32_t *page_table, int max_pages,
                         const int32_t *kv_lens, la_bf16 *out, int B, int H, int Hkv, int D, float scale,
                         void *workspace, size_t workspace_bytes, la_stream stream) {
    return attn_verify(q, q_row_stride, k_pages, v_pages, page_stride, num_pages, page_size, page_table, max_pages,
                       kv_lens, nullptr, false, out, B, 1, H, Hkv, D, scale, workspace, workspace_bytes, stream);
}

la_status la_attn_verify_tree(const la_bf16 *q, int64_t q_row_stride, const la_bf16 *k_pages, const la_bf16 *v_pages,
                              int64_t page_stride, int num_pages, int page_size, const int32_t *page_table,
                              int max_pages, const int32_t *kv_lens, const int32_t *parents, la_bf16 *out, int B,
                              int N, int H, int Hkv, int D, float scale, void *workspace, size_t workspace_bytes,
                              la_stream stream) {
    return attn_verify(q, q_row_stride, k_pages, v_pages, page_stride, num_pages, page_size, page_table, max_pages,
                       kv_lens, parents, true, out, B, N, H, Hkv, D, scale, workspace, workspace_bytes, stream);
}

la_status la_kv_commit(la_bf16 *k_pages, la_bf16 *v_pages, int64_t page_stride, int num_pages, int page_size,
                       const int32_t *page_table, int max_pages, const int32_t *kv_lens, const int32_t *parents,
                       const int32_t *accept_idx, int32_t *new_lens, int B, int N, int Hkv, int D,
                       la_stream stream) {
    return la_kv_commit_ex(k_pages, v_pages, page_stride, num_pages, page_size, page_table, max_pages, kv_lens, parents,
                           accept_idx, new_lens, 0, B, N, Hkv, D, stream);
}

la_status la_kv_commit_ex(la_bf16 *k_pages, la_bf16 *v_pages, int64_t page_stride, int num_pages, int page_size,
                          const int32_t *page_table, int max_pages, const int32_t *kv_lens, const int32_t *parents,
                          const int32_t *accept_idx, int32_t *new_lens, int keep_lens, int B, int N, int Hkv, int D,
                          la_stream stream) {
    la::KvCommitParams p = la::KvCommitParams{};
    la_status st = cache_params(&p.cache, k_pages, v_pages, page_stride, num_pages, page_size, page_table, max_pages,
                                kv_lens, Hkv, D, true);
    if (st != LA_OK) return st;
    if (B < 0 || N < 1) return LA_ERR_INVALID;
    if (N > la::kMaxDrafts) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!cache_pointers_ok(p.cache, true) || !parents || !accept_idx || !new_lens || !aligned4(parents) ||
        !aligned4(accept_idx) || !aligned4(new_lens))
        return LA_ERR_INVALID;
    p.parents = parents;
    p.accept_idx = accept_idx;
    p.new_lens = new_lens;
    p.B = B;
    p.N = N;
    p.Hkv = Hkv;
    p.keep_lens = keep_lens != 0;
    if ((st = error_word_ptr(&p.err)) != LA_OK) return st;
    return launch_status(la::launch_kv_commit(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
