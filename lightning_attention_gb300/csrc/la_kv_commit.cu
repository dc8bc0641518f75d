// la_kv_commit.cu -- the accepted drafts of a tree become the end of their request's context: the key and
// value rows on the path to the last accepted draft move to the positions right behind the context.
//
// A path's drafts ascend, its i-th is draft i or a later one, so rows move towards the front and a row is
// only overwritten by a move that comes no earlier than its own.  A thread takes 16 bytes of every row of
// the path, eight rows read before they are written.  A copy of a few rows: bound by latency (the walk up the path,
// then the page table, then the rows).
#include "la_attn.h"

namespace la {
namespace {

constexpr int kThreads = 256;  // a warp per kv head: 16 pieces of a key row, 16 of a value row

__global__ void __launch_bounds__(kThreads) kv_commit_kernel(const KvCommitParams p) {
    __shared__ int path[kMaxDrafts], parent[kMaxDrafts];
    __shared__ long long from[kMaxDrafts], to[kMaxDrafts];
    __shared__ int count;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x, tid = threadIdx.x;
    const CacheParams &c = p.cache;
    const int kv = c.kv_lens[b], last = p.accept_idx[b];
    const bool report = tid == 0;  // writes new_lens, which may be kv_lens, once all threads have read them
    auto skip = [&](unsigned int fault) {
        if (!report) return;
        atomicOr(p.err, fault);
        if (p.keep_lens) p.new_lens[b] = kv;
    };
    if (kv == 0) {  // a request without positions; new_lens may hold that already
        if (report) p.new_lens[b] = 0;
        return;
    }
    if (kv < p.N || kv > (long long)c.max_pages * c.page_size) {
        skip(ERR_BIT_PAGE);
        return;
    }
    if (last < -1 || last >= p.N) {
        skip(ERR_BIT_ACCEPT);
        return;
    }
    if (tid < p.N) parent[tid] = p.parents[(long long)b * p.N + tid];
    __syncthreads();
    if (tid == 0) {
        int n = 0, a = last;
        while (a >= 0) {  // a falls with every step
            path[n++] = a;
            const int up = parent[a];
            if (up < -1 || up >= a) {
                n = -1;
                break;
            }
            a = up;
        }
        count = n;
    }
    __syncthreads();
    const int n = count;
    if (n < 0) {
        skip(ERR_BIT_PARENTS);
        return;
    }
    const int ctx = kv - p.N;
    bool bad = false;
    if (tid < n) {
        const int32_t *table = c.page_table + (long long)b * c.max_pages;
        const int x = ctx + path[n - 1 - tid], y = ctx + tid;
        const int px = table[x / c.page_size], py = table[y / c.page_size];
        bad = px < 0 || px >= c.num_pages || py < 0 || py >= c.num_pages;
        from[tid] = px * c.page_stride + (long long)(x % c.page_size) * kHeadDim;
        to[tid] = py * c.page_stride + (long long)(y % c.page_size) * kHeadDim;
    }
    if (__syncthreads_or(bad)) {
        skip(ERR_BIT_PAGE);
        return;
    }
    if (report) p.new_lens[b] = ctx + n;
    for (int head = tid >> 5; head < p.Hkv; head += kThreads / 32) {
        __nv_bfloat16 *pages = (tid & 16 ? c.v : c.k) + (long long)head * c.page_size * kHeadDim + (tid & 15) * 8;
        for (int i0 = 0; i0 < n; i0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < n) x[i] = *reinterpret_cast<const uint4 *>(pages + from[i0 + i]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < n && from[i0 + i] != to[i0 + i]) *reinterpret_cast<uint4 *>(pages + to[i0 + i]) = x[i];
        }
    }
}

}  // namespace

cudaError_t launch_kv_commit(const KvCommitParams &p, cudaStream_t stream) {
    return launch_pdl(kv_commit_kernel, dim3((unsigned)p.B), dim3(kThreads), 0, stream, p);
}

}  // namespace la
