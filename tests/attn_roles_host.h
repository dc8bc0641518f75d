// What the roles of the attention kernels call, for the host: a fiber per thread, and barriers that count.
// Shared entries that threads exchange are Cells: they know who touched them since which barrier.  A barrier that
// can never be complete, accesses of two threads with no barrier between them, and copies or MMAs that are under way
// when all roles have ended and that nobody has waited for to the end, end the program with a message.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <set>
#include <vector>

#define __device__
#define __host__
#define __forceinline__ inline
using std::max;
using std::min;

struct uint2 { unsigned x, y; };
struct uint4 { unsigned x, y, z, w; };
struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
struct Dim { int x, y, z; };
inline uint4 make_uint4(unsigned a, unsigned b, unsigned c, unsigned d) { return {a, b, c, d}; }
inline float2 make_float2(float a, float b) { return {a, b}; }
struct __nv_bfloat16 { uint16_t bits; };

struct Fiber {
    ucontext_t ctx;
    std::vector<char> stack;
    Dim tid;
    bool done;
    int barriers;  // that this thread has passed
    int waits;     // of this thread so far
    int fetched;   // reads of scores
};
static std::vector<Fiber> fibers;
static Fiber *self;
static ucontext_t scheduler;
static long progress;
#define threadIdx (self->tid)
static Dim blockIdx = {0, 0, 0}, gridDim = {2, 1, 1};
static int fail_warp = -1, fail_at = -1, failed;  // the wait that runs out
static bool rising;                               // whether every tile's scores pass those before
static const char *scenario = "";

[[noreturn]] static void broken(const char *what, int a, int b) {
    printf("%s: %s (%d, %d); wait %d of warp %d ran out\n", scenario, what, a, b, fail_at, fail_warp);
    fflush(stdout);
    _Exit(1);
}
static void yield() { swapcontext(&self->ctx, &scheduler); }
template <class F>
static void until(F done) {
    while (!done()) yield();
    ++progress;
}

// A meeting of `count` threads, each with a value; all get all values.
struct Meeting {
    long gen = 0;
    int here = 0;
    std::vector<uint64_t> value[2];
    int who[2][1024];
    const std::vector<uint64_t> &meet(int place, int count, uint64_t x) {
        const long g = gen;
        std::vector<uint64_t> &v = value[g & 1];
        if (here == 0) v.assign(count, 0);
        v[place] = x;
        ++progress;
        if (++here == count) {
            here = 0;
            ++gen;
        }
        until([&] { return gen != g; });
        return v;
    }
};
static Meeting warps[32], named[16];
static int lane_of() { return threadIdx.x & 31; }
static int named_place(int id);  // of this thread among those that meet at barrier `id`
static int named_count(int id);
static bool named_any(int id, bool x) {
    const std::vector<uint64_t> &v = named[id].meet(named_place(id), named_count(id), x);
    bool any = false;
    for (uint64_t y : v) any |= y != 0;
    ++self->barriers;
    return any;
}

template <class T>
static T lane_value(T x, int src) {
    uint64_t bits = 0;
    memcpy(&bits, &x, sizeof x);
    const uint64_t got = warps[threadIdx.x >> 5].meet(lane_of(), 32, bits)[src & 31];
    T y;
    memcpy(&y, &got, sizeof y);
    return y;
}
template <class T>
static T __shfl_sync(unsigned, T x, int src) { return lane_value(x, src); }
template <class T>
static T __shfl_xor_sync(unsigned, T x, int d) { return lane_value(x, lane_of() ^ d); }
static const std::vector<uint64_t> &lanes(uint64_t x) { return warps[threadIdx.x >> 5].meet(lane_of(), 32, x); }
static bool __all_sync(unsigned, bool x) {
    bool all = true;
    for (uint64_t y : lanes(x)) all &= y != 0;
    return all;
}
static int __reduce_min_sync(unsigned, int x) {
    int least = x;
    for (uint64_t y : lanes((uint64_t)(int64_t)x)) least = min(least, (int)(int64_t)y);
    return least;
}
static unsigned __ballot_sync(unsigned, bool x) {
    const std::vector<uint64_t> &v = lanes(x);
    unsigned bits = 0;
    for (int i = 0; i < 32; ++i) bits |= (unsigned)(v[i] != 0) << i;
    return bits;
}
template <class T>
static T __shfl_up_sync(unsigned, T x, int d) { return lane_value(x, lane_of() < d ? lane_of() : lane_of() - d); }
static int __clz(unsigned x) { return x ? __builtin_clz(x) : 32; }
static int __ffs(unsigned x) { return __builtin_ffs((int)x); }
static void __syncwarp() { lanes(0); }
static bool elect() { return lane_of() == 0; }
static unsigned __funnelshift_r(unsigned lo, unsigned hi, int d) {
    return (unsigned)(((uint64_t)hi << 32 | lo) >> (d & 31));
}
template <class T>
static T as(const void *p) { T x; memcpy(&x, p, sizeof x); return x; }
static float __uint_as_float(unsigned x) { return as<float>(&x); }
static unsigned __float_as_uint(float x) { return as<unsigned>(&x); }
static void atomicOr(unsigned *p, unsigned x) { *p |= x; }
static __nv_bfloat16 __float2bfloat16_rn(float x) { return {(uint16_t)(__float_as_uint(x) >> 16)}; }
static uint32_t pack_bf16x2(float a, float b) { return __float_as_uint(a) >> 16 | (__float_as_uint(b) & 0xffff0000u); }
static float ex2z(float x) { return exp2f(x); }
static float max3(float a, float b, float c) { return fmaxf(a, fmaxf(b, c)); }
static float redux_max(float x) {
    float top = x;
    for (uint64_t y : lanes(__float_as_uint(x))) top = fmaxf(top, __uint_as_float((unsigned)y));
    return top;
}

// Scores: those of a tile alike, or above all that the thread has read before.
static float score() { return rising ? 40.f * ++self->fetched : 0.f; }
template <int n>
static void tmem_ld32(uint32_t, uint32_t (&r)[n]) { const float s = score(); for (uint32_t &x : r) x = __float_as_uint(s); }
template <int n>
static void tmem_get(uint32_t, float (&r)[n]) { const float s = score(); for (float &x : r) x = s; }
template <int n>
static void tmem_put(uint32_t, const float (&)[n]) {}
static void tmem_st16(uint32_t, const uint32_t (&)[16]) {}
static void tmem_st32(uint32_t, const uint32_t (&)[32]) {}
template <class A>
static void tmem_ld_wait_regs(A &) {}
template <class A>
static void tmem_ld_wait_regs2(A &, A &) {}
static void tmem_st_wait() {}
static void tc_fence_after() {}
static void tc_fence_before() {}
static void fence_proxy_async_smem() {}
static void mbar_arrive(uint64_t *) {}

// What a wait is for is there at once, or never comes; copies and MMAs are waited for to the end with a limit that
// nobody has set (a second and more).
static std::set<uint64_t *> copies;  // barriers of those under way
static uint64_t *committed;          // that of the last MMAs
static bool mmas;
static bool mbar_wait(uint64_t *bar, uint32_t, uint64_t limit_ns) {
    if (limit_ns < 1000000000ull && (int)(threadIdx.x >> 5) == fail_warp && self->waits++ == fail_at) {
        failed = 1;
        return false;
    }
    copies.erase(bar);
    if (bar == committed) mmas = false;
    return true;
}
static void mbar_arrive_expect_tx(uint64_t *bar, uint32_t) { copies.insert(bar); }
static void mma_commit(uint64_t *bar) { committed = bar; }
template <class... A>
static void mma_bf16(A...) { mmas = true; committed = nullptr; }
template <class... A>
static void mma_f16_tmem_a(A...) { mmas = true; committed = nullptr; }
struct CUtensorMap {};
template <class... A>
static void tma_load_4d(A...) {}
template <class... A>
static void tma_load_5d(A...) {}
template <class... A>
static uint32_t idesc_bf16_f32(A...) { return 0; }
template <class... A>
static uint64_t sdesc_sw128(A...) { return 0; }
template <class... A>
static uint64_t sdesc_sw32(A...) { return 0; }
static uint32_t smem_u32(const void *) { return 0; }

// Writes of one thread and accesses of another need a barrier between them; lanes of a warp may write the same value.
struct Cell {
    float v;
    int wrote_at, wrote, read_at, read;  // barriers passed plus one, thread; read -1: several threads
    operator float() {
        const int t = threadIdx.x, at = self->barriers + 1;
        if (wrote_at == at && wrote != t) broken("an entry is read beside another thread's write", t, wrote);
        read = read_at == at && read != t ? -1 : t;
        read_at = at;
        return v;
    }
    float operator=(float x) {
        const int t = threadIdx.x, at = self->barriers + 1;
        if (wrote_at == at && wrote != t && (wrote >> 5 != t >> 5 || v != x))
            broken("an entry is written by two threads", t, wrote);
        if (read_at == at && read != t) broken("an entry is written beside another thread's read", t, read);
        wrote = t;
        wrote_at = at;
        return v = x;
    }
};
static float4 load4(Cell *c) { return {c[0], c[1], c[2], c[3]}; }

static std::function<void()> body;
static void enter() {
    body();
    self->done = true;
    ++progress;
    swapcontext(&self->ctx, &scheduler);
}
// Runs `f` on the threads of the given warps to their end.
static void run(const std::vector<int> &which, std::function<void()> f) {
    body = f;
    failed = 0;
    copies.clear();
    mmas = false;
    for (auto &w : warps) w = Meeting();
    for (auto &b : named) b = Meeting();
    fibers.resize(which.size() * 32);
    for (size_t i = 0; i < fibers.size(); ++i) {
        Fiber &x = fibers[i];
        x.stack.resize(64 << 10);
        x.tid = {which[i / 32] * 32 + (int)(i % 32), 0, 0};
        x.done = false;
        x.barriers = x.waits = x.fetched = 0;
        getcontext(&x.ctx);
        x.ctx.uc_stack.ss_sp = x.stack.data();
        x.ctx.uc_stack.ss_size = x.stack.size();
        x.ctx.uc_link = nullptr;
        makecontext(&x.ctx, enter, 0);
    }
    while (true) {
        const long before = progress;
        size_t left = 0;
        for (Fiber &x : fibers) {
            if (x.done) continue;
            ++left;
            self = &x;
            swapcontext(&scheduler, &x.ctx);
        }
        if (left == 0 && (mmas || !copies.empty())) broken("under way at the end: MMAs, copies", mmas, (int)copies.size());
        if (left == 0) return;
        if (progress == before) broken("threads wait for others that have left", (int)left, (int)fibers.size());
    }
}
// `f` with no wait that runs out, then with each wait of each of the warps `out`.
static void every_wait(const std::vector<int> &which, const std::vector<int> &out, std::function<void()> f) {
    fail_warp = -1;
    run(which, f);
    for (int w : out)
        for (fail_at = 0, fail_warp = w;; ++fail_at) {
            run(which, f);
            if (!failed) break;
        }
    fail_warp = fail_at = -1;
}
