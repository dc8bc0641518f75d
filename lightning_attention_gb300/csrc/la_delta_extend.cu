// la_delta_extend.cu -- chunked gated delta rule on the 5th-generation tensor cores, one CTA per
// (request, value head), or several where there are few.
//
// Per request and head, token by token: S <- e^{g} S; u = beta (v - S^T k); S <- S + k u^T;
// o = D^-0.5 S^T q (q, k divided by their 2-norms first if asked).  Over a chunk of C = 64 tokens with
// S the state before it, G_i the running sum of g, gamma_i = e^{G_i}, rk, rq the inverse norms (or 1):
//   X     = [K; Q] S
//   R_i   = beta_i v_i - beta_i gamma_i rk_i X^K_i
//   A_ij  = beta_i rk_i rk_j e^{G_i - G_j} (k_i . k_j)            j < i, else 0
//   T     = (I + A)^-1 = I + T'                                    (strictly lower T')
//   U     = T R = R + T' R
//   P_ij  = D^-0.5 rq_i rk_j e^{G_i - G_j} (q_i . k_j)             j <= i, else 0
//   o_i   = D^-0.5 gamma_i rq_i X^Q_i + (P U)_i,   P U = (P T) R
//   S     <- gamma_C S + K^T diag(e^{G_C - G_j} rk_j) U
// Every exponent is formed as a difference of sums that are kept as fp32 pairs, so that steep decays lose
// nothing; factors are at most 1.
//
// Two kernels.  T and P T of a chunk depend on nothing before it, so a first kernel forms them for all
// chunks at once (delta_t_kernel, a CTA of four warps per chunk and head), with the chunk's coefficients,
// into the workspace; the second runs the chain over the chunks, one CTA per (request, head)
// (delta_extend_kernel; a long request among few is split, see Split).  One kernel with T warps beside the
// chain took 393 us on 8 requests of 512-4096 tokens x 16 heads, the two take 220: while tcgen05.mma
// instructions stream, warp-level MMAs are starved (four take 1,764 cycles in place of 79), so T held the
// chain up.
//
// The chain is computed transposed: lanes of tensor memory are the 128 value columns.
//   X^T = S^T [K; Q]^T,   [U; O']^T = R^T [T'; P T]^T,   dS^T = U^T K
// so the three operands that it computes (S, R, U) are the A operands, which a tcgen05.mma takes from
// tensor memory: a warp converts its lanes where they lie, without a trip through shared memory, and the
// B operands (the stacked [K; Q] tile, the stacked [T'; P T] tile, K) come in by TMA ahead of the chain.
// The stacking keeps the products with S and U at M = N = 128 (65 cycles an instruction; one of N = 64 takes
// 45-50); the one with R leaves out the rows of T' and P T that are zero, so its k-steps have N = 128, 96, 64, 32.
// P T makes the output a product with R, so nothing of it waits for U.
//
// Precision.  Products run in bf16 with fp32 accumulation.  K and Q are used as loaded; the operands
// that are computed (S, R, T', P T, U) are bf16 pairs hi + lo, off by at most 2^-16 and about a sixth of
// that in the mean; U takes R itself in fp32 and only T' R through pairs; products of two pairs leave out that
// of the lo parts, but for those of the inverse; the state stays in fp32 registers and is never accumulated in
// tensor memory (which does not round to nearest).  Decays come from ex2.approx (off by 2^-22) and norms from
// rsqrtf (2 units in the last place), both far below the pairs.  The state is off by 3.2e-6 of its norm, of which U's
// pair is 2.8e-6: a third part of U leaves 1.6e-6 and takes the mixed batch above from 218.5 to 230.8 us, one request
// of 32,768 tokens x 32 heads from 840 to 895; third parts of S, R and U and a finer inverse would be needed for less
// than 1e-6, at half again the chain's MMAs.  The outputs are rounded to bf16, 1.7e-3, and show none of it.
// Where a chunk's sums cancel (keys nearly the same, beta |k|^2 near 2, no decay) the pairs' errors show more: 1.2e-4
// of the norm at keys within 8 degrees.
//
// Roles of the chain kernel (384 threads, one CTA per SM):
//   warps 0-7   E: the state (32 v rows x 64 k columns a warp) and the passes R, U, O and S;
//   warp 8      finds the items (below) and issues their loads; warp 9 tensor-memory owner and MMA issuer;
//   warp 10     zeroes the K rows past the end of the request's last chunk (they hold the next
//               request's keys, and 0 x NaN is NaN).
// Per chunk the chain is X -> R -> T' R -> U -> U^T K -> S; the output pass runs under U^T K.  A chunk takes
// about 2.4 us: 36 MMAs, 24 of 65 cycles and 12 of 65 down to 45 or less, are half of it, the passes between them
// (wait, tensor memory to registers, pair split, back, barrier) the other half; no two of them overlap along the
// chain, and a second chain on the SM has room neither in tensor memory (512 columns) nor in shared memory (171 KB).
// More items than SMs: a CTA per SM takes several in turn, longest first, each from a common count, and warp 8
// runs ahead of the item that is worked on.  256 requests of 32-512 tokens x 16 heads: 641 us; items dealt out
// in turn 19 more, a CTA per item 67 more.
//
// Every wait ends: mbarrier waits have a deadline (the named barriers below end with them); one that runs out
// sets the error word and an abort flag that ends every role, then the CTA waits for its copies and MMAs,
// frees tensor memory and exits.
#include <cuda.h>

#include <mutex>

#include "la_delta.h"
#include "la_delta_plan.h"
#include "la_sm100.cuh"

namespace la {

namespace {

using namespace sm100;

constexpr int C = kDeltaChunk;
constexpr int kEWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kFixWarp = 10;
constexpr int kThreads = 384;
// Registers per thread of the warp groups: 2 x 184 (E) + 136 = 3 x 168, the launch's share.  (E at 200: the
// same times; at 216 2% more on the batch above.)
constexpr int kRegsE = 184, kRegsRest = 136;
static_assert(2 * kRegsE + kRegsRest <= 3 * 168, "register split");
constexpr int kTThreads = 128;
constexpr float kScale = 0.08838834764831845f;  // 128^-0.5

constexpr uint32_t kTmemCols = 512;
// The operands S, R and U are kept per k-step (16 values of the contraction) as 8 columns of hi parts,
// two to a column, and 8 of lo parts.  X: [K | Q] tokens, R replaces the K part 16 tokens by 16; Y: per 16
// tokens [U | O'], U likewise.
constexpr uint32_t TM_S = 0, TM_X = 128, TM_Y = 256, TM_D = 384;

// What the first kernel leaves per chunk and head: T' and P T as their hi and their lo parts, then the
// coefficients: beta, -beta gamma rk, lam rk and scale gamma rq per token, gamma_C.  T' and P T are stacked
// by blocks of 16 rows (T' of tokens 16 a .., then P T of them, a = 0 .. 3), and a part is cut by k-steps kk
// of 16 columns, of which only the row blocks a >= kk are not zero: 128 - 32 kk rows of 32 bytes, with the
// 16-byte pieces of a row swapped where the row's bit 2 is set (the 32-byte swizzle that the MMA reads).
constexpr uint32_t SZ_PART = 10240;
constexpr uint32_t SZ_COEF = 4 * 256 + 16;
constexpr uint32_t SZ_SLOT = 2 * SZ_PART + SZ_COEF;
// The words behind gamma_C are spare; the first one of the workspace's first slot says whether cu_seqlens
// decreases somewhere.
constexpr uint32_t OFF_DISORDER = 2 * SZ_PART + 4 * 257;
static_assert(OFF_DISORDER + 4 <= SZ_SLOT, "a spare word");
// Offset within a part of step kk.
__host__ __device__ constexpr uint32_t part_ofs(int kk) { return (uint32_t)(4096 * kk - 512 * kk * (kk - 1)); }
static_assert(part_ofs(4) == SZ_PART, "part layout");
// Chunk slots of a batch: request b's start at floor(cu_seqlens[b] / C) + b, far enough from the next
// request's for its ceil(length / C) chunks.
__host__ __device__ inline long long chunk_slots(long long T, long long B) { return T / C + B; }

// Shared memory of the chain kernel, from a 1024-byte aligned base.
constexpr int kStages = 3;
constexpr uint32_t SZ_KQ = 32768;                          // [64 K rows; 64 Q rows][128], swizzled
constexpr uint32_t OFF_KQ = 0;
constexpr uint32_t OFF_V = OFF_KQ + kStages * SZ_KQ;       // 2 x [64][128], rows of 256 bytes
constexpr uint32_t OFF_T = OFF_V + 2 * 16384;              // 2 x a slot
constexpr uint32_t SZ_T = (SZ_SLOT + 255) / 256 * 256;     // whole swizzle atoms
constexpr uint32_t OFF_COEF = OFF_T + 2 * SZ_PART;         // a slot's coefficients
constexpr uint32_t OFF_BAR = OFF_T + 2 * SZ_T;
constexpr uint32_t SZ_BAR = 512;
constexpr uint32_t kSmemBytes = OFF_BAR + SZ_BAR + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

// What a CTA's roles need of the item (a chain, or a segment of one) they are on.
struct Item {
    const float *from;  // the start state; null: zero, or the identity for a transition
    float *to;          // where the end state goes; null: not kept
    int t0, n, h;       // first token, tokens, value head
    int transition;     // PLANNED: V counts as zero
    int emit;           // PLANNED: outputs are written
};
constexpr int kItems = 4;
// The kernel's kinds: several items a CTA; one (without the loop over items in the E warps' code, which costs
// the chunk loop 2%); one that is a segment; several that are segments of a plan.
enum Kind : int { MANY, ONE, SEGMENT, PLANNED };

struct Bars {
    uint64_t kq_full[kStages];
    uint64_t kq_empty[kStages];  // the chunk's products done; warp 10 past it (2)
    uint64_t kq_ready[kStages];  // warp 10: K rows past the request's end zeroed
    uint64_t v_full[2], t_full[2];
    uint64_t y_done[2];    // the product with T's tile done: tile and V buffer free
    uint64_t c_free[2];    // E warps: the chunk's coefficients read (8)
    uint64_t item_full[kItems];
    uint64_t item_empty[kItems];  // read by the E warps, the MMA warp and warp 10 (10)
    uint64_t x_full, y_full, d_full;
    uint64_t o_free;       // E warps (8): X^Q and O' read
    uint64_t drain;
    Item items[kItems];
    uint32_t tmem_base;
    int abort_flag;
    int go[2];             // the MMA warp's word to the E warps: on to the next item
};
static_assert(sizeof(Bars) <= SZ_BAR, "barrier block");

// Shared memory of the T kernel (five CTAs per SM).  16 x 16 blocks of the inversion are two panels of 8
// columns x 16 rows x 16 bytes: the blocks of A below the diagonal (hi, lo) and the diagonal blocks of T
// (hi, lo; before that A's, transposed, and T's in fp32).  The slot's two parts (P before P T) and the blocks
// take the place of K and Q.  (Six CTAs fit, at 80 registers: 227 us in place of 222 on the mixed batch.)
constexpr uint32_t TK_KQ = 0;                              // [64 K rows; 64 Q rows][128]
constexpr uint32_t TK_AB = 2 * SZ_PART;                    // 6 x (512 hi + 512 lo)
constexpr uint32_t TK_TD = TK_AB + 6 * 1024;               // 4 x (512 hi + 512 lo)
constexpr uint32_t TK_TOK = TK_KQ + SZ_KQ;                 // per token: ghi, glo, rk, beta rk, scale rq
static_assert(TK_TD + 4 * 1024 <= SZ_KQ, "blocks in place of K and Q");
constexpr uint32_t kTSmemBytes = TK_TOK + 5 * 256 + 1024;

// Named barriers between the E warps, which arrive, and the MMA warp, which waits: k-steps y and 4 + y of S
// (kBarS + y), y and 2 + y of R and U (kBarR + y, kBarU + y) are in place.  A test of an
// mbarrier takes about 113 cycles when eight warps poll, a named barrier about 30.  They have no deadline of
// their own: the E warps arrive at every one of every chunk, whether their own (bounded) waits succeed or
// not, so the MMA warp's waits end when theirs do.  At kBarItem all of them meet before an item: the MMA warp,
// which waits (with a deadline) for the item, says there whether it is still to be run.
constexpr int kBarS = 1, kBarR = 5, kBarU = 7, kBarItem = 9;
constexpr int kBarThreads = (kEWarps + 1) * 32;
__device__ __forceinline__ void bar_arrive(int id) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kBarThreads) : "memory");
}
__device__ __forceinline__ void bar_wait(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kBarThreads) : "memory");
}

constexpr uint64_t kDrainLimitNs = 2000000000ull;
constexpr uint64_t kTryNs = 10000;  // above a suspended try

struct Ctx {
    uint64_t limit;
    volatile int *abort_flag;
    unsigned int *err;
};

// A try may suspend the thread for some 4 us; under a limit near that warps 8 and 10, whose waits are the
// longest, test without being suspended (TEST).
template <bool TEST>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity, const Ctx &cx) {
    if (!TEST || cx.limit >= kTryNs) return mbar_try_wait(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
template <bool TEST = false>
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const Ctx &cx) {
    const uint32_t a = smem_u32(bar);
    if (try_wait<TEST>(a, parity, cx)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (try_wait<TEST>(a, parity, cx)) return true;
        if (*cx.abort_flag) return false;
        if (globaltimer_ns() - t0 > cx.limit) {
            *cx.abort_flag = 1;
            atomicOr(cx.err, ERR_BIT_TIMEOUT);
            return false;
        }
    }
}
// All lanes wait; the warp goes on only if every lane's wait succeeded.
template <bool TEST = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Ctx &cx) {
    return __all_sync(0xffffffffu, wait_bar<TEST>(bar, parity, cx));
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Two fp32 values in one 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2u(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// bf16 pairs of two values: hi = bf16(x), lo = bf16(x - hi), the first value in the low halves.
__device__ __forceinline__ void split2(uint64_t x, uint32_t &hi, uint32_t &lo) {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
    hi = pack_bf16x2(a, b);
    const uint64_t d = fma2(f2u(hi << 16, hi & 0xffff0000u), f2(-1.f, -1.f), x);
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
    lo = pack_bf16x2(a, b);
}
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    split2(f2(x0, x1), hi, lo);
}
// A 16 x 16 accumulator (two 16 x 8 fragments) as the bf16 pair of an A operand.
__device__ __forceinline__ void split_frag(const float (&c)[8], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(c[0], c[1], hi[0], lo[0]);
    split2(c[2], c[3], hi[1], lo[1]);
    split2(c[4], c[5], hi[2], lo[2]);
    split2(c[6], c[7], hi[3], lo[3]);
}

// acc + cross += A B with A and B bf16 pairs: two sums, so that fewer MMAs wait for one another.  The product of
// the two lo parts (2^-16 at most) is formed where LO says so.
template <bool LO>
__device__ __forceinline__ void prod16(float (&acc)[8], float (&cross)[8], const uint32_t (&ah)[4],
                                       const uint32_t (&al)[4], const uint32_t (&bh)[4],
                                       const uint32_t (&bl)[4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        mma_16816(acc + 4 * n, ah, bh[2 * n], bh[2 * n + 1]);
        if (LO) mma_16816(cross + 4 * n, al, bl[2 * n], bl[2 * n + 1]);
        mma_16816(cross + 4 * n, ah, bl[2 * n], bl[2 * n + 1]);
        mma_16816(cross + 4 * n, al, bh[2 * n], bh[2 * n + 1]);
    }
}

// ------------------------------------------------------------------------------------------------
// T warps

// A sum as hi + lo, lo the part that hi's rounding lost: sums of a chunk's gates keep about 2^-45.
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 add_sums(const Sum2 &a, const Sum2 &b) {
    const float s = a.hi + b.hi, bb = s - a.hi;
    const float lo = ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo);
    const float hi = s + lo;
    return {hi, lo - (hi - s)};
}
// log2(e) g, -1e4 standing for every g below (e^-1e4 is 0 in fp32, and the sums stay finite).
__device__ __forceinline__ Sum2 gate_log2(float g) {
    constexpr float kHi = 1.44269502162933349609f;     // log2(e) in fp32
    constexpr float kLo = 1.92596299112661746887e-8f;  // the rest
    g = g < -1e4f ? -1e4f : g;
    const float p = g * kHi;
    return {p, fmaf(g, kHi, -p) + g * kLo};
}

// The fragments of rows 16 blk .. + 15 of the [K; Q] tile (Q: blk + 4) at k-step ks, as an A operand; as a
// B operand the same registers are {0, 2} for columns 0-7 and {1, 3} for columns 8-15.  The tile starts on
// a 1024-byte boundary and row blocks on multiples of 16, so the swizzle is an exclusive or of the lane's
// address at = kq_lane() with the piece.
__device__ __forceinline__ uint32_t kq_lane(uint32_t tile, int lane) {
    const int mrow = lane & 7, midx = lane >> 3;  // matrices (k half, row half)
    return (tile + (uint32_t)((midx & 1) * 8 + mrow) * 128u) | (uint32_t)(((midx >> 1) ^ mrow) << 4);
}
__device__ __forceinline__ void kq_frag(uint32_t at, int blk, int ks, uint32_t (&f)[4]) {
    ldsm4((at ^ ((ks & 3) * 32u)) + (ks >> 2) * 16384u + blk * 2048u, f);
}
// acc (16 x 16) += A B^T of two such fragments.
__device__ __forceinline__ void dot_frag(float *acc, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
    mma_16816(acc, a, b[0], b[2]);
    mma_16816(acc + 4, a, b[1], b[3]);
}

// Address of a row's 16-byte piece kc (0, 1) in a part: row rho of T' (pt = 0) or P T (1), columns of step kk.
__device__ __forceinline__ uint32_t part_row(uint32_t part, int kk, int pt, int rho, int kc) {
    return part + part_ofs(kk) + (uint32_t)(rho + 16 * ((rho >> 4) + pt) - 32 * kk) * 32u +
           ((uint32_t)(kc ^ ((rho >> 2) & 1)) << 4);
}
// A fragment block (16 x 16) as a bf16 pair: rows rho0 .. + 15 of step kk.
__device__ __forceinline__ void put_block(uint8_t *parts, int kk, int pt, int rho0, int row, int cp,
                                          const float *x) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t h0, l0, h1, l1;
        split2(x[4 * hf], x[4 * hf + 1], h0, l0);
        split2(x[4 * hf + 2], x[4 * hf + 3], h1, l1);
        uint8_t *dst = parts + part_row(0, kk, pt, rho0 + row, hf) + cp * 2;
        *reinterpret_cast<uint32_t *>(dst) = h0;
        *reinterpret_cast<uint32_t *>(dst + 256) = h1;  // row + 8: the same swizzle
        *reinterpret_cast<uint32_t *>(dst + SZ_PART) = l0;
        *reinterpret_cast<uint32_t *>(dst + SZ_PART + 256) = l1;
    }
}
// The same into a scratch block (two panels of 8 columns; lo 512 bytes behind).
__device__ __forceinline__ void put_panel(uint8_t *blk, int row, int cp, const float *x) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t h0, l0, h1, l1;
        split2(x[4 * hf], x[4 * hf + 1], h0, l0);
        split2(x[4 * hf + 2], x[4 * hf + 3], h1, l1);
        uint8_t *dst = blk + hf * 256 + row * 16 + cp * 2;
        *reinterpret_cast<uint32_t *>(dst) = h0;
        *reinterpret_cast<uint32_t *>(dst + 128) = h1;
        *reinterpret_cast<uint32_t *>(dst + 512) = l0;
        *reinterpret_cast<uint32_t *>(dst + 640) = l1;
    }
}

// Per-token factors of the T kernel's blocks.
struct TokenFactors {
    const float *ghi, *glo, *rk, *brk, *qs;
};

// Block (a, b): kk and qk become A's and P's elements (above the diagonal zero, A's diagonal too).
__device__ __forceinline__ void scale_block(const TokenFactors &f, int a, int b, int row, int cp, float *kk,
                                            float *qk) {
    const int i0 = 16 * a + row, i1 = i0 + 8;
    const float gh0 = f.ghi[i0], gh1 = f.ghi[i1], gl0 = f.glo[i0], gl1 = f.glo[i1];
    const float ai0 = f.brk[i0], ai1 = f.brk[i1], qi0 = f.qs[i0], qi1 = f.qs[i1];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int j = 16 * b + 8 * hf + cp;
        const float2 gh = *reinterpret_cast<const float2 *>(f.ghi + j);
        const float2 gl = *reinterpret_cast<const float2 *>(f.glo + j);
        const float2 rj = *reinterpret_cast<const float2 *>(f.rk + j);
        const float e00 = ex2((gh0 - gh.x) + (gl0 - gl.x)) * rj.x;
        const float e01 = ex2((gh0 - gh.y) + (gl0 - gl.y)) * rj.y;
        const float e10 = ex2((gh1 - gh.x) + (gl1 - gl.x)) * rj.x;
        const float e11 = ex2((gh1 - gh.y) + (gl1 - gl.y)) * rj.y;
        float *k = kk + 4 * hf, *q = qk + 4 * hf;
        k[0] *= e00 * ai0;
        k[1] *= e01 * ai0;
        k[2] *= e10 * ai1;
        k[3] *= e11 * ai1;
        q[0] *= e00 * qi0;
        q[1] *= e01 * qi0;
        q[2] *= e10 * qi1;
        q[3] *= e11 * qi1;
        if (a == b) {
            if (j >= i0) k[0] = 0.f;
            if (j + 1 >= i0) k[1] = 0.f;
            if (j >= i1) k[2] = 0.f;
            if (j + 1 >= i1) k[3] = 0.f;
            if (j > i0) q[0] = 0.f;
            if (j + 1 > i0) q[1] = 0.f;
            if (j > i1) q[2] = 0.f;
            if (j + 1 > i1) q[3] = 0.f;
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Split of a long request.  With few (request, head) pairs the chain leaves SMs idle, and a segment of it
// can be run without its start state: its chunks take S to M S + N, N being the segment's result from
// S = 0 and M its result from the identity with V = 0, which are two more chains of the same kernel.  So the
// chain is cut into segs segments, the first ratio times as long as the others:
//   pass 1   segment 0 as usual; N and M of segments 1 .. segs - 2, side by side with it;
//   join     the segments' start states, S_1 from pass 1, S_{g+1} = M_g S_g + N_g in fp32;
//   pass 2   segments 1 .. segs - 1 from their start states, side by side.
// Rounding in a segment is amplified by the segments after it as the chain's own is.
// Measured whole / split, us, T kernel included, l2norm, one request: 8 heads: 1,280 tokens 57 / 50, 2,048:
// 84.6 / 60.5, 16,384: 626 / 190; 32 heads: 1,024: 52.7 / 61.9, 1,536: 75.3 / 73.7, 16,384: 703 / 445;
// 76 heads: 2,560: 145 / 149, 4,096: 222 / 212, 16,384: 836 / 720.
struct Split : Cut {
    int pass;       // 0: not split
    float *starts;  // [chains][segs - 1][D][D]: S_g at g - 1 (N_{g-1} before the join)
    float *trans;   // [chains][segs - 2][D][D]: M_g at g - 1
    const int32_t *plan;  // PLANNED: what follows; starts holds all of the plan's matrices
};
constexpr float kItemCost = 1.2f;  // of an item beside its chunks, in chunks
constexpr size_t kMat = (size_t)kHeadDim * kHeadDim;

// The job of a CTA (one item each): segment, whether it is a transition, whether outputs are written.
struct Job {
    int seg;
    bool transition, emit;
};
__device__ __forceinline__ Job split_job(const DeltaParams &p, const Split &s) {
    const int job = (int)blockIdx.x / (p.B * p.H);
    if (s.pass == 2) return {1 + job, false, true};
    return {(job + 1) >> 1, (job & 1) != 0, job == 0};
}

// Plan of a batch whose longest request is much longer than its share of the SMs (which the host judges by
// max_seqlen and T; the lengths are on the device).  The same two passes, but with one cut for all requests:
// segment 0 is a request's first a chunks, the next are b chunks each, so that short requests end in pass 1 as
// they are.  A CTA of the first kernel tries 128 pairs (a, b) and lists the segments of both passes longest
// first; an entry stands for its request's H heads.
constexpr int kPlanA = 0, kPlanB = 1, kPlanFirst = 2, kPlanSecond = 3, kPlanJoins = 4, kPlanStarts = 5;
constexpr int kPlanTaken1 = 6, kPlanTaken2 = 7;  // items taken in a pass, beyond each CTA's first
constexpr int kPlanList1 = 16;                                  // entries of pass 1
constexpr int kPlanList2 = kPlanList1 + kMaxPlanned + kPlanMats;  // of pass 2
constexpr int kPlanJoin = kPlanList2 + kPlanMats;               // requests with a join
constexpr int kPlanS = kPlanJoin + kMaxPlanned;                 // start states before a request's
constexpr int kPlanT = kPlanS + kMaxPlanned;                    // transitions before a request's
constexpr int kPlanInts = kPlanT + kMaxPlanned;
constexpr size_t kPlanBytes = kPlanInts * sizeof(int32_t);
static_assert(kPlanBytes % 16 == 0, "matrices are 16-byte aligned");
constexpr int kPlanTrans = 1 << 30;
__device__ __forceinline__ int plan_entry(int request, int seg) { return request | seg << 10; }
__host__ __device__ inline int segments_after(int nchunks, int a, int b) {
    return nchunks > a ? (nchunks - a + b - 1) / b : 0;
}
__device__ __forceinline__ bool request_ok(const DeltaParams &p, int t0, int t1) {
    return t0 >= 0 && t1 >= t0 && t1 <= p.T && t1 - t0 <= p.max_seqlen;
}
__device__ void plan_requests(const DeltaParams &p, int32_t *plan, int *sm) {
    int *len = sm, *last = sm + kMaxPlanned;
    __shared__ int most;
    __shared__ unsigned long long best;
    if (threadIdx.x == 0) {
        most = 0;
        best = ~0ull;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < p.B; r += kTThreads) {
        const int t0 = p.cu_seqlens[r], t1 = p.cu_seqlens[r + 1];
        len[r] = request_ok(p, t0, t1) ? (t1 - t0 + C - 1) / C : 0;
        atomicMax(&most, len[r]);
    }
    __syncthreads();
    auto cut_a = [&](int t) { return max(1, (most * ((t >> 3) + 1) + 15) / 16); };
    auto cut_b = [&](int t) { return max(1, (cut_a(t) * ((t & 7) + 1) + 7) / 8); };
    {
        const int a = cut_a(threadIdx.x), b = cut_b(threadIdx.x);
        int w1 = 0, w2 = 0, mats = 0, trans = 0, deepest = 0, tail = 0;
        for (int r = 0; r < p.B; ++r) {
            w1 += min(len[r], a);
            const int l = segments_after(len[r], a, b);
            if (l > 0) {
                w1 += 2 * (l - 1) * b;
                w2 += len[r] - a;
                mats += 2 * l - 1;
                trans += l - 1;
                deepest = max(deepest, l);
                tail = max(tail, min(b, len[r] - a));
            }
        }
        // the longest segment of a pass, or the SMs' share of all, items' own cost and uneven ends included
        const float share = 1.1f * (float)p.H / (float)kSplitSMs;
        float cost = fmaxf((float)min(a, most), share * ((float)w1 + kItemCost * (float)(p.B + 2 * trans)));
        if (deepest > 0) {
            cost += fmaxf((float)tail, share * ((float)w2 + kItemCost * (float)(mats - trans))) +
                    (float)kSplitCost + 2.f * (float)kJoinCost * (float)deepest;
            cost *= 1.f / (float)kSplitGain;
            if (mats > kPlanMats / p.H) cost = 3e38f;
        }
        atomicMin(&best, (unsigned long long)__float_as_uint(cost) << 32 | threadIdx.x);
    }
    __syncthreads();
    const int won = (int)(best & 0xffffffffu);
    const int a = cut_a(won), b = cut_b(won);
    for (int r = threadIdx.x; r < p.B; r += kTThreads) last[r] = segments_after(len[r], a, b);
    __syncthreads();
    for (int r = threadIdx.x; r < p.B; r += kTThreads) {
        const int first = min(len[r], a), mine = last[r];
        const int tail = len[r] - a - (mine - 1) * b;  // chunks of the last segment
        int rank1 = 0, rank2 = 0, whole = 0, starts = 0, trans = 0, joins = 0, all_trans = 0;
        for (int u = 0; u < p.B; ++u) {
            const int f = min(len[u], a), l = last[u], before = u < r;
            rank1 += f > first || (f == first && before);
            whole += f >= b;
            all_trans += max(l - 1, 0);
            if (before) {
                starts += l;
                trans += max(l - 1, 0);
                joins += l > 1;
            }
            const int x = len[u] - a - (l - 1) * b;
            rank2 += l > 0 && (x > tail || (x == tail && before));
        }
        plan[kPlanS + r] = starts;
        plan[kPlanT + r] = trans;
        if (mine > 1) plan[kPlanJoin + joins] = r;
        // N and M of a segment stand behind the first segments that are as long
        plan[kPlanList1 + rank1 + (first < b ? 2 * all_trans : 0)] = plan_entry(r, 0);
        for (int g = 1; g < mine; ++g) {
            plan[kPlanList1 + whole + 2 * (trans + g - 1)] = plan_entry(r, g);
            plan[kPlanList1 + whole + 2 * (trans + g - 1) + 1] = plan_entry(r, g) | kPlanTrans;
            plan[kPlanList2 + trans + g - 1] = plan_entry(r, g);
        }
        if (mine > 0) plan[kPlanList2 + all_trans + rank2] = plan_entry(r, mine);
        if (r == p.B - 1) {
            plan[kPlanTaken1] = plan[kPlanTaken2] = 0;
            plan[kPlanA] = a;
            plan[kPlanB] = b;
            plan[kPlanFirst] = p.B + 2 * all_trans;
            plan[kPlanSecond] = starts + mine;
            plan[kPlanJoins] = joins + (mine > 1);
            plan[kPlanStarts] = starts + mine;
        }
    }
}

// The order of a batch, and behind it a count.
__host__ __device__ inline int order_ints(int B) { return (B + 1 + 3) / 4 * 4; }
// Request of each rank in decreasing length order (ties by index), kTThreads requests per CTA.
__device__ void rank_requests(const DeltaParams &p, int block, int32_t *order, int *lens) {
    const int b = block * kTThreads + (int)threadIdx.x;
    const int mine = b < p.B ? p.cu_seqlens[b + 1] - p.cu_seqlens[b] : 0;
    int rank = 0;
    for (int u0 = 0; u0 < p.B; u0 += kTThreads) {
        __syncthreads();
        const int u = u0 + (int)threadIdx.x;
        lens[threadIdx.x] = u < p.B ? p.cu_seqlens[u + 1] - p.cu_seqlens[u] : 0;
        __syncthreads();
        const int m = min(kTThreads, p.B - u0);
        for (int x = 0; x < m; ++x) rank += (lens[x] > mine) || (lens[x] == mine && u0 + x < b);
    }
    if (b < p.B) order[rank] = b;
    if (b == 0) order[order_ints(p.B) - 1] = 0;  // items taken beyond each CTA's first
}

// Whether cu_seqlens decreases somewhere.  Chunk slots of different requests may then be the same, and a slot's
// request is not found by search, so that the chain kernel skips the whole batch.
__device__ void check_order(const DeltaParams &p, uint8_t *ws) {
    int less = 0;
    for (int r = threadIdx.x; r < p.B; r += kTThreads) less |= p.cu_seqlens[r + 1] < p.cu_seqlens[r];
    less = __syncthreads_or(less);
    if (threadIdx.x == 0) *reinterpret_cast<int *>(ws + OFF_DISORDER) = less;
}

// T', P T and the coefficients of one chunk and head (blockIdx.x = first_ctas + slot * H + head); of the
// first_ctas CTAs the first checks cu_seqlens, and they order the requests for the chain kernel, or plan its
// segments.  Warp w has the 16 rows 16 w ..
// of everything: the 16 x 16 blocks of K K^T and Q K^T (mma.sync: a block is too small for tcgen05), the inverse
// of its diagonal block of I + A by substitution, a lane per column, then the blocks below by T_ab = -T_aa
// sum A_am T_mb.
// Measured: 68 us on 8 requests of 512-4096 tokens x 16 heads, 260 us on 256 of 32-512; 40-50 % of DRAM and half
// of the issue slots.  Bound by the latency of the dependent small products and the barriers between them, at
// the 20 warps per SM that its 95 registers allow.  PLAN is a variant of its own, as its code slows the rest down
// by 4%.
template <bool PLAN>
__global__ void __launch_bounds__(kTThreads, 5)
    delta_t_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const DeltaParams p, uint8_t *ws, int32_t *order, int32_t *plan, int first_ctas) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t kq_full;
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int w = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // uniform, so its branches are too
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x < first_ctas) {
        if (blockIdx.x == 0) check_order(p, ws);
        if (PLAN)
            plan_requests(p, plan, reinterpret_cast<int *>(sm));
        else if (order)
            rank_requests(p, blockIdx.x, order, reinterpret_cast<int *>(sm));
        return;
    }
    const unsigned item = blockIdx.x - (unsigned)first_ctas;
    const int slot = (int)(item / (unsigned)p.H);
    const int h = (int)(item - (unsigned)slot * (unsigned)p.H);

    // The slot's request: the last b with floor(cu_seqlens[b] / C) + b <= slot, 32 candidates at a time.
    // (A batch that is out of order and requests that are too long are skipped by the chain kernel; whatever is
    // found for them is checked before it is used.)
    int b = 0;
    {
        int step = 1;
        while (step * 32 < p.B) step *= 32;
        int lo = 0;
        for (; step > 0; step /= 32) {
            const int cand = lo + lane * step;
            const bool in = cand < p.B && (p.cu_seqlens[cand] >> 6) + cand <= slot;
            const uint32_t m = __ballot_sync(0xffffffffu, in);
            if (m == 0) return;
            lo += (31 - __clz(m)) * step;
        }
        b = lo;
    }
    const int t_req0 = p.cu_seqlens[b], t_req1 = p.cu_seqlens[b + 1];
    if (t_req0 < 0 || t_req1 < t_req0 || t_req1 > p.T) return;
    const int c = slot - (t_req0 >> 6) - b;
    const int r = t_req1 - t_req0 - c * C;  // tokens from this chunk on
    if (c < 0 || r <= 0) return;
    const size_t t0 = (size_t)t_req0 + (size_t)c * C;

    float *tok = reinterpret_cast<float *>(sm + TK_TOK);
    float *ghi = tok, *glo = tok + 64, *rk = tok + 128, *brk = tok + 192, *qs = tok + 256;
    uint8_t *abp = sm + TK_AB, *tdp = sm + TK_TD;
    const uint32_t ab = smem_u32(abp), td = smem_u32(tdp), kq = smem_u32(sm + TK_KQ), parts = smem_u32(sm);
    float *ad = reinterpret_cast<float *>(tdp + w * 1024);
    uint8_t *slot_out = ws + (size_t)item * SZ_SLOT;
    float *cf = reinterpret_cast<float *>(slot_out + 2 * SZ_PART);
    const int row = lane >> 2, cp = (lane & 3) * 2;  // fragment row, column pair
    const int mrow = lane & 7, midx = lane >> 3;     // ldmatrix: row, matrix
    const uint32_t off_p = (uint32_t)((midx & 1) * 256 + (midx >> 1) * 128 + mrow * 16);
    const int i16 = 16 * w + (lane & 15);            // this warp's tokens, twice

    // K and Q into swizzled tiles
    if (threadIdx.x == 0) {
        mbar_init(&kq_full, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&kq_full, SZ_KQ);
        const int x = (h / p.group) * kHeadDim;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            tma_load_2d(sm + y * 16384, &tk, &kq_full, x + 64 * y, (int)t0);
            tma_load_2d(sm + y * 16384 + 8192, &tq, &kq_full, x + 64 * y, (int)t0);
        }
    }
    const float beta = i16 < r ? p.beta[(t0 + i16) * p.H + h] : 0.f;
    // running sums of the gates, by warp 0
    if (w == 0) {
        const float *gp = p.g + (t0 * p.H + h);
        Sum2 x0 = gate_log2(lane < r ? gp[(size_t)lane * p.H] : 0.f);
        Sum2 x1 = gate_log2(lane + 32 < r ? gp[(size_t)(lane + 32) * p.H] : 0.f);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum2 y0{__shfl_up_sync(0xffffffffu, x0.hi, d), __shfl_up_sync(0xffffffffu, x0.lo, d)};
            const Sum2 y1{__shfl_up_sync(0xffffffffu, x1.hi, d), __shfl_up_sync(0xffffffffu, x1.lo, d)};
            if (lane >= d) {
                x0 = add_sums(x0, y0);
                x1 = add_sums(x1, y1);
            }
        }
        x1 = add_sums(x1, {__shfl_sync(0xffffffffu, x0.hi, 31), __shfl_sync(0xffffffffu, x0.lo, 31)});
        ghi[lane] = x0.hi;
        glo[lane] = x0.lo;
        ghi[lane + 32] = x1.hi;
        glo[lane + 32] = x1.lo;
    }
    __syncthreads();
    // the CTA goes on only if every thread's wait succeeded
    if (!__syncthreads_and(mbar_wait(&kq_full, 0, p.wait_limit_ns))) {
        // the copies are waited for once more before the CTA's shared memory goes away
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_TIMEOUT);
        mbar_wait(&kq_full, 0, kDrainLimitNs);
        return;
    }
    if (r < C) {
        // rows past the end hold the next request's tokens, and 0 x NaN is NaN: zero them
        for (int x = r * 32 + (int)threadIdx.x; x < C * 32; x += kTThreads)  // (token, K or Q, block, piece)
            *reinterpret_cast<uint4 *>(sm + ((x >> 3) & 1) * 16384 + ((x >> 5) + ((x >> 4) & 1) * 64) * 128 +
                                       (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }

    // ---- K K^T and Q K^T of the warp's blocks (a, b): the diagonal one (w, w), then (3,0) | (1,0) |
    // (2,0) (2,1) | (3,1) (3,2), rows of the warp's own fragments but for (3,0), which has its columns;
    // Q Q^T for the norms
    const int a1 = w == 0 ? 3 : w, b1 = w == 3 ? 1 : 0, b2 = w - 1;
    float kk[3][8] = {}, qk[3][8] = {}, qq[8] = {};
    {
        const uint32_t at = kq_lane(kq, lane);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t fk[4], fq[4], f[4];
            kq_frag(at, w, ks, fk);
            kq_frag(at, 4 + w, ks, fq);
            dot_frag(kk[0], fk, fk);
            dot_frag(qk[0], fq, fk);
            if (p.l2norm) dot_frag(qq, fq, fq);
            if (w == 0) {
                kq_frag(at, 3, ks, f);
                dot_frag(kk[1], f, fk);
                kq_frag(at, 7, ks, f);
                dot_frag(qk[1], f, fk);
            } else {
                kq_frag(at, b1, ks, f);
                dot_frag(kk[1], fk, f);
                dot_frag(qk[1], fq, f);
            }
            if (w >= 2) {
                kq_frag(at, b2, ks, f);
                dot_frag(kk[2], fk, f);
                dot_frag(qk[2], fq, f);
            }
        }
    }
    float nk = 1.f, nq = 1.f;  // squared norms of token i16
    if (p.l2norm) {
        // element (i, i) of a fragment block: rows 0-7 in lane 4 i + i / 2, rows 8-15 likewise
        const int src = 4 * (lane & 7) + ((lane & 7) >> 1);
        const float k0 = __shfl_sync(0xffffffffu, row & 1 ? kk[0][1] : kk[0][0], src);
        const float k1 = __shfl_sync(0xffffffffu, row & 1 ? kk[0][7] : kk[0][6], src);
        const float q0 = __shfl_sync(0xffffffffu, row & 1 ? qq[1] : qq[0], src);
        const float q1 = __shfl_sync(0xffffffffu, row & 1 ? qq[7] : qq[6], src);
        nk = (lane & 8 ? k1 : k0) + kDeltaEps;
        nq = (lane & 8 ? q1 : q0) + kDeltaEps;
    }
    {
        const float inv = p.l2norm ? rsqrtf(lane < 16 ? nk : nq) : 1.f;
        const float gh = ghi[i16], gl = glo[i16];
        const float gam = ex2(gh + gl);
        if (lane < 16) {
            rk[i16] = inv;
            brk[i16] = beta * inv;
            cf[i16] = beta;
            cf[64 + i16] = -beta * gam * inv;
            cf[128 + i16] = ex2((ghi[C - 1] - gh) + (glo[C - 1] - gl)) * inv;
        } else {
            qs[i16] = kScale * inv;
            cf[192 + i16] = kScale * gam * inv;
        }
        if (w == 0 && lane == 0) cf[256] = ex2(ghi[C - 1] + glo[C - 1]);
    }
    __syncthreads();  // K and Q are read: P and T' take their place

    // ---- scaled blocks: A to scratch, P to its place
    {
        const TokenFactors f{ghi, glo, rk, brk, qs};
        scale_block(f, w, w, row, cp, kk[0], qk[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e)  // transposed: column m of A's block at ad + 16 m
            ad[(8 * (e >> 2) + cp + (e & 1)) * 16 + row + 8 * ((e >> 1) & 1)] = kk[0][e];
        put_block(sm, w, 1, 16 * w, row, cp, qk[0]);
        scale_block(f, a1, b1, row, cp, kk[1], qk[1]);
        put_panel(abp + (a1 * (a1 - 1) / 2 + b1) * 1024, row, cp, kk[1]);
        put_block(sm, b1, 1, 16 * a1, row, cp, qk[1]);
        if (w >= 2) {
            scale_block(f, w, b2, row, cp, kk[2], qk[2]);
            put_panel(abp + (w * (w - 1) / 2 + b2) * 1024, row, cp, kk[2]);
            put_block(sm, b2, 1, 16 * w, row, cp, qk[2]);
        }
    }
    __syncwarp();

    // ---- the diagonal block of T: column j = lane % 16 by substitution
    {
        float x[16];
        const int j = lane & 15;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 15; ++m) {
#pragma unroll
            for (int v4 = (m + 1) / 4; v4 < 4; ++v4) {
                const float4 f = *reinterpret_cast<const float4 *>(ad + m * 16 + 4 * v4);
                if (4 * v4 > m) x[4 * v4] = fmaf(-f.x, x[m], x[4 * v4]);
                if (4 * v4 + 1 > m) x[4 * v4 + 1] = fmaf(-f.y, x[m], x[4 * v4 + 1]);
                if (4 * v4 + 2 > m) x[4 * v4 + 2] = fmaf(-f.z, x[m], x[4 * v4 + 2]);
                if (4 * v4 + 3 > m) x[4 * v4 + 3] = fmaf(-f.w, x[m], x[4 * v4 + 3]);
            }
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) ad[i * 16 + j] = x[i];
        }
        __syncwarp();
        float t[8];  // the block in fragment layout
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 f = *reinterpret_cast<const float2 *>(ad + (row + 8 * ((e >> 1) & 1)) * 16 +
                                                               8 * (e >> 2) + cp);
            t[e] = f.x;
            t[e + 1] = f.y;
        }
        __syncwarp();
        put_panel(tdp + w * 1024, row, cp, t);
        // the operand tile holds T' = T - I
        if (row == cp) t[0] = t[6] = 0.f;
        if (row == cp + 1) t[1] = t[7] = 0.f;
        put_block(sm, w, 0, 16 * w, row, cp, t);
    }
    __syncthreads();  // all blocks of A, all diagonal blocks of T

    // ---- column block b = w of T below the diagonal, as its transpose:
    // T_rb^T = -(sum_{b <= m < r} T_mb^T A_rm^T) T_rr^T.
    // With the products of the lo parts: where keys are nearly the same those do not average out, and T multiplies
    // A's error from both sides.  At beta near 2 and keys within 8 degrees the state's error is 1.2e-4 of its norm
    // with them and 6.1e-4 without, at beta near 1 1.8e-5 and 2.1e-5 (256 requests of 32-512 tokens: 640.7 us with,
    // 637.9 without).  P T goes without them, as its errors reach one output and no state.
    {
        const int b = w;
        uint32_t yh[3][4], yl[3][4];
        ldsm4_t(td + b * 1024 + off_p, yh[0]);
        ldsm4_t(td + b * 1024 + 512 + off_p, yl[0]);
#pragma unroll
        for (int dr = 1; dr < 4; ++dr) {
            const int rr = b + dr;
            if (rr > 3) break;
            float acc[8] = {}, cross[8] = {};
            uint32_t bh[4], bl[4];
#pragma unroll
            for (int dm = 0; dm < dr; ++dm) {
                const uint32_t blk = ab + (rr * (rr - 1) / 2 + b + dm) * 1024 + off_p;
                ldsm4(blk, bh);
                ldsm4(blk + 512, bl);
                prod16<true>(acc, cross, yh[dm], yl[dm], bh, bl);
            }
            uint32_t zh[4], zl[4];
            float t[8] = {}, tc[8] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += cross[e];
            split_frag(acc, zh, zl);
            ldsm4(td + rr * 1024 + off_p, bh);
            ldsm4(td + rr * 1024 + 512 + off_p, bl);
            prod16<true>(t, tc, zh, zl, bh, bl);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = -t[e] - tc[e];
            split_frag(t, zh, zl);
            // matrices (j half, i half) -> rows i of the tile, columns 16 b + j
            const uint32_t at = part_row(parts, b, 0, 16 * rr + 8 * (midx >> 1) + mrow, midx & 1);
            stsm4_t(at, zh);
            stsm4_t(at + SZ_PART, zl);
            if (dr < 3) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    yh[dr][e] = zh[e];
                    yl[dr][e] = zl[e];
                }
            }
        }
    }
    // ---- P T over P, five products a warp: blocks (3,0) (0,0) | (3,1) (1,0) | (2,0) (2,1) | (3,2) (1,1)
    // (2,2) (3,3).  Every block of P is in its readers' registers before one is overwritten.
    {
        const int k = (midx & 1) * 8 + mrow, nh = midx >> 1;
        const uint32_t pa_off = (uint32_t)((midx & 1) * 8 + mrow), kc = (uint32_t)(midx >> 1);
        uint32_t fh[5][4], fl[5][4];
        // the i-th product of the warp: P block (a, m) times T block (m, b)
        auto which = [&](int i, int &a, int &m, int &b) {
            if (w == 0) {
                a = i < 4 ? 3 : 0, m = i < 4 ? i : 0, b = 0;
            } else if (w == 1) {
                a = i < 3 ? 3 : 1, m = i < 3 ? 1 + i : i - 3, b = i < 3 ? 1 : 0;
            } else if (w == 2) {
                a = 2, m = i < 3 ? i : i - 2, b = i < 3 ? 0 : 1;
            } else {
                a = i < 2 ? 3 : i - 1, m = i < 2 ? 2 + i : i - 1, b = i < 2 ? 2 : i - 1;
            }
        };
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            int a, m, b;
            which(i, a, m, b);
            const uint32_t pa = part_row(parts, m, 1, 16 * a + pa_off, kc);
            ldsm4(pa, fh[i]);
            ldsm4(pa + SZ_PART, fl[i]);
        }
        __syncthreads();  // T' is written, P is read
        float acc[8] = {}, cross[8] = {};
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            int a, m, b;
            which(i, a, m, b);
            uint32_t bh[4], bl[4];
            const uint32_t at = m == b ? td + b * 1024 + nh * 256 + k * 16 : part_row(parts, b, 0, 16 * m + k, nh);
            ldsm4_t(at, bh);
            ldsm4_t(at + (m == b ? 512 : SZ_PART), bl);
            prod16<false>(acc, cross, fh[i], fl[i], bh, bl);
            if (m == a) {  // the block's last product
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += cross[e];
                put_block(sm, b, 1, 16 * a, row, cp, acc);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = cross[e] = 0.f;
            }
        }
    }

    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
        bulk_store(slot_out, sm, 2 * SZ_PART);
        bulk_commit_group();
        bulk_wait_group0();
    }
}

// ------------------------------------------------------------------------------------------------
// E warps: lanes are value columns v = 32 q + lane; half hf of the chunk's tokens and of the k columns.

// Eight pairs (one k-step of an operand) as 8 columns of hi parts and 8 of lo parts; the MMA issuer may
// use them once every E warp has arrived.
__device__ __forceinline__ void put_step(uint32_t t, const uint64_t *x, int bar) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split2(x[e], hi[e], lo[e]);
    tmem_st8(t, hi);
    tmem_st8(t + 8u, lo);
    tmem_st_wait();
    tc_fence_before();
    bar_arrive(bar);
}

// 32 per-token coefficients (the same for all lanes).
__device__ __forceinline__ void load_pairs(const float *src, uint64_t (&x)[16]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(src + 4 * e);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
}

template <Kind KIND>
__device__ void e_role(const DeltaParams &p, uint8_t *sm, Bars *bars, const Ctx &cx, uint32_t tbase, int q,
                       int hf, int lane, int items, const Split &split) {
    constexpr bool SPLIT = KIND == SEGMENT;
    const int v = 32 * q + lane;
    const int tok0 = 32 * hf;  // tokens tok0 .. + 31 of the chunk
    const uint32_t lanes = tbase + ((uint32_t)(32 * q) << 16);
    const uint32_t ts = lanes + TM_S + 64u * hf;
    const uint32_t tx = lanes + TM_X + 32u * hf, ty = lanes + TM_Y + 64u * hf, td = lanes + TM_D + 64u * hf;
    const int at = 64 * hf * kHeadDim + v;
    bool ok = true;
    int cc = 0;  // chunks of the items before
    for (int k = 0; k < (KIND == MANY || KIND == PLANNED ? items : 1); ++k) {
        bar_wait(kBarItem);
        if (!*(volatile int *)&bars->go[k & 1]) break;
        const Item item = bars->items[k % kItems];
        warp_arrive(&bars->item_empty[k % kItems], lane);
        const int n = item.n, h = item.h, nchunks = (n + C - 1) / C;
        const size_t t0 = (size_t)item.t0;
        const bool transition =
            KIND == PLANNED ? item.transition != 0 : SPLIT && split_job(p, split).transition;
        const bool emit = KIND == PLANNED ? item.emit != 0 : !SPLIT || split_job(p, split).emit;
        // a transition's V as zero (a choice between values makes its loads wait behind a branch: 975 us in
        // place of 840 for 32,768 tokens)
        const uint32_t vmask = transition ? 0u : 0xffffffffu;

        uint64_t S[32];  // S[64 hf + 2 x, 64 hf + 2 x + 1][v]
        if (item.from) {
            const float *gs = item.from + at;
#pragma unroll
            for (int x = 0; x < 32; ++x) S[x] = f2(gs[2 * x * kHeadDim], gs[(2 * x + 1) * kHeadDim]);
        } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const int d = transition ? v - 64 * hf - 2 * x : -1;
                S[x] = f2(d == 0 ? 1.f : 0.f, d == 1 ? 1.f : 0.f);
            }
        }
        if (nchunks > 0) {
#pragma unroll
            for (int x = 0; x < 4; ++x) put_step(ts + 16u * x, S + 8 * x, kBarS + x);
        }

        // a wait gave up: the named barriers that are left of this chunk, from R's, U's or S's on (waited for,
        // so that no warp runs a chunk ahead of the others)
        auto give_up = [&](int from, int c) {
            ok = false;
            for (int x = from; x < kBarU + 2; ++x) bar_wait(x);
            if (c + 1 < nchunks)
                for (int x = kBarS; x < kBarR; ++x) bar_wait(x);
        };
        for (int c = 0; c < nchunks; ++c) {
            if (!ok) {
                give_up(kBarR, c);
                continue;
            }
            const uint32_t par = (cc + c) & 1, ph = ((cc + c) >> 1) & 1;
            const int r = n - c * C;  // tokens from this chunk on
            const float *cf = reinterpret_cast<const float *>(sm + OFF_COEF + par * SZ_T) + tok0;
            // ---- R = beta V - (beta gamma rk) X^K; what needs no X is formed while its product runs
            if (!warp_wait(&bars->t_full[par], ph, cx)) {
                give_up(kBarR, c);
                continue;
            }
            if (!warp_wait(&bars->v_full[par], ph, cx)) {
                give_up(kBarR, c);
                continue;
            }
            uint64_t R[16], f[16];
            {
                const uint8_t *vp = sm + OFF_V + par * 16384 + tok0 * 256 + v * 2;
                load_pairs(cf, R);
                load_pairs(cf + 64, f);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const uint32_t v0 = *reinterpret_cast<const uint16_t *>(vp + (2 * x) * 256);
                    const uint32_t v1 = *reinterpret_cast<const uint16_t *>(vp + (2 * x + 1) * 256);
                    R[x] = mul2(R[x], f2u((v0 << 16) & vmask, (v1 << 16) & vmask));
                }
            }
            if (!warp_wait(&bars->x_full, par, cx)) {
                give_up(kBarR, c);
                continue;
            }
            tc_fence_after();
            {
                uint32_t w[2][16];
                tmem_ld16(tx, w[0]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    tmem_ld_wait_regs(w[y]);
                    if (y == 0) tmem_ld16(tx + 16u, w[1]);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        R[8 * y + x] = fma2(f[8 * y + x], f2u(w[y][2 * x], w[y][2 * x + 1]), R[8 * y + x]);
                    if (r < C) {  // rows past the end hold other requests' values
#pragma unroll
                        for (int x = 8 * y; x < 8 * y + 8; ++x) {
                            if (tok0 + 2 * x >= r) R[x] = 0ull;
                            else if (tok0 + 2 * x + 1 >= r) R[x] &= 0xffffffffull;
                        }
                    }
                    put_step(tx + 16u * y, R + 8 * y, kBarR + y);
                }
            }

            // ---- U = R + T' R, scaled for the state update
            load_pairs(cf + 128, f);
            if (!warp_wait(&bars->y_full, par, cx)) {
                give_up(kBarU, c);
                continue;
            }
            tc_fence_after();
            {
                uint32_t w[2][16];
                tmem_ld16(ty, w[0]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    tmem_ld_wait_regs(w[y]);
                    if (y == 0) tmem_ld16(ty + 32u, w[1]);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        R[8 * y + x] =
                            mul2(f[8 * y + x], add2(R[8 * y + x], f2u(w[y][2 * x], w[y][2 * x + 1])));
                    put_step(ty + 32u * y, R + 8 * y, kBarU + y);
                }
            }

            // ---- o = (scale gamma rq) X^Q + P T R; neighbouring lanes exchange halves, so that each
            // stores two value columns of one token
            if (!emit) {
                warp_arrive(&bars->o_free, lane);
            } else {
                const size_t tok = t0 + (size_t)c * C + tok0 + (lane & 1);
                __nv_bfloat16 *op = p.out + (tok * p.H + h) * kHeadDim + (v & ~1);
                const size_t two = (size_t)p.H * kHeadDim * 2;
                const int left = r - tok0 - (lane & 1);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t w[16], y[16];
                    tmem_ld16(tx + 64u + 16u * z, w);
                    tmem_ld16(ty + 16u + 32u * z, y);
                    tmem_ld_wait_regs(w);
                    tmem_ld_wait_regs(y);
                    if (z == 1) {
                        tc_fence_before();
                        warp_arrive(&bars->o_free, lane);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 o = *reinterpret_cast<const float4 *>(cf + 192 + 16 * z + 4 * x);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int at = 4 * x + 2 * e;
                            float za, zb;
                            asm("mov.b64 {%0, %1}, %2;"
                                : "=f"(za), "=f"(zb)
                                : "l"(fma2(e ? f2(o.z, o.w) : f2(o.x, o.y), f2u(w[at], w[at + 1]),
                                           f2u(y[at], y[at + 1]))));
                            const uint32_t mine = pack_bf16x2(za, zb);  // tokens at, at + 1
                            const uint32_t theirs = __shfl_xor_sync(0xffffffffu, mine, 1);
                            // even lanes: the first token of (v, v + 1); odd lanes: the second of (v - 1, v)
                            const uint32_t word = (lane & 1) ? __byte_perm(theirs, mine, 0x7632)
                                                             : __byte_perm(mine, theirs, 0x5410);
                            if (16 * z + at < left)
                                *reinterpret_cast<uint32_t *>(op + (8 * z + (at >> 1)) * two) = word;
                        }
                    }
                }
            }

            // ---- S = gamma_C S + K^T U
            const float ge = cf[256 - tok0];
            warp_arrive(&bars->c_free[par], lane);
            if (!warp_wait(&bars->d_full, par, cx)) {
                give_up(kBarU + 2, c);
                continue;
            }
            tc_fence_after();
            {
                const uint64_t ge2 = f2(ge, ge);
                uint32_t w[2][16];
                tmem_ld16(td, w[0]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t(&d)[16] = w[x & 1];
                    tmem_ld_wait_regs(d);
                    if (x < 3) tmem_ld16(td + 16u * (x + 1), w[(x + 1) & 1]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        S[8 * x + e] = fma2(ge2, S[8 * x + e], f2u(d[2 * e], d[2 * e + 1]));
                    if (c + 1 < nchunks) put_step(ts + 16u * x, S + 8 * x, kBarS + x);
                }
            }
        }
        cc += nchunks;
        if (ok && item.to) {
            float *gs = item.to + at;
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                float a, b;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(S[x]));
                gs[2 * x * kHeadDim] = a;
                gs[(2 * x + 1) * kHeadDim] = b;
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// MMA issuer: one warp, of which lane 0 issues.  The warp stays together and only the instruction itself is
// predicated, so that its operands are formed by the uniform datapath: with a branch around them each MMA
// took some 110 cycles to issue, longer than to run.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ void mma_role(Bars *bars, uint32_t tbase, uint32_t s_base, int items, int lane, Ctx cx) {
    const uint32_t id = idesc_bf16_f32(128, 128, false, false);
    const uint32_t idD = idesc_bf16_f32(128, 128, false, true);
    // B operands of one swizzle have the same high descriptor word (8-row groups 1024 bytes apart, 128-byte
    // swizzle); the low word holds the start address and the leading-dimension offset.
    const uint64_t high = sdesc_sw128(0, 0, 1024);
    const uint64_t high32 = sdesc_sw32(0, 0, 256);  // T's tile: rows of 32 bytes
    uint32_t lead = lane == 0;  // 0 in every lane once a wait gave up
    auto mma = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint64_t hw) {
        mma_ts(lead, tbase + d, tbase + a, hw | b, idesc, acc);
    };
    bool ok = true;
    int st = 0, cc = 0;  // cc: chunks of the items before
    uint32_t stp = 0;
    for (int k = 0; k < items; ++k) {
        ok = ok && warp_wait(&bars->item_full[k % kItems], (k / kItems) & 1, cx);
        const bool go =
            __shfl_sync(0xffffffffu, (int)(ok && !*cx.abort_flag && bars->items[k % kItems].n >= 0), 0);
        if (lane == 0) bars->go[k & 1] = go;
        __syncwarp();
        bar_wait(kBarItem);
        if (!go) break;
        const int n = bars->items[k % kItems].n, nchunks = (n + C - 1) / C;
        warp_arrive(&bars->item_empty[k % kItems], lane);
        for (int c = 0; c < nchunks; ++c) {
            const uint32_t par = (cc + c) & 1, ph = ((cc + c) >> 1) & 1;
            // once a wait gave up nothing more is issued, but every named barrier is waited for
            ok = ok && warp_wait(&bars->kq_full[st], stp, cx) &&
                 (cc + c == 0 || warp_wait(&bars->o_free, (cc + c - 1) & 1, cx));
            if (!ok) lead = 0;
            const uint32_t kq = (s_base + OFF_KQ + st * SZ_KQ) >> 4;
            // a k-step starts as soon as the E warps have put it in place
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                bar_wait(kBarS + y);
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int kk = y + 4 * (x >> 1);  // hi, lo of k-steps y and 4 + y
                    mma(TM_X, TM_S + 16u * kk + 8u * (x & 1),
                        kq + ((kk >> 2) * 1024 + (kk & 3) * 2) + (1u << 16), id, y + x > 0, high);
                }
                if (y == 3) commit_if(lead, &bars->x_full);
            }
            ok = ok && warp_wait(&bars->t_full[par], ph, cx);
            if (!ok) lead = 0;
            const uint32_t tt = (s_base + OFF_T + par * SZ_T) >> 4;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                bar_wait(kBarR + y);
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 6; ++x) {  // R_hi T_hi, R_lo T_hi, R_hi T_lo of k-steps y and 2 + y,
                                               // for the rows that are not zero
                    const int kk = y + 2 * (x / 3), term = x % 3;
                    mma(TM_Y + 32u * kk, TM_X + 16u * kk + (term == 1 ? 8u : 0u),
                        tt + (term == 2 ? SZ_PART >> 4 : 0u) + (part_ofs(kk) >> 4) + (1u << 16),
                        idesc_bf16_f32(128, 128 - 32 * kk, false, false), y + x > 0, high32);
                }
                if (y == 1) {
                    commit_if(lead, &bars->y_full);
                    commit_if(lead, &bars->y_done[par]);
                }
            }
            if (n - c * C < C) {
                ok = ok && warp_wait(&bars->kq_ready[st], stp, cx);
                if (!ok) lead = 0;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                bar_wait(kBarU + y);
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int kk = y + 2 * (x >> 1);
                    mma(TM_D, TM_Y + 32u * kk + 8u * (x & 1), kq + kk * 128 + ((16384u >> 4) << 16), idD,
                        y + x > 0, high);
                }
                if (y == 1) {
                    commit_if(lead, &bars->d_full);
                    commit_if(lead, &bars->kq_empty[st]);
                }
            }
            if (++st == kStages) {
                st = 0;
                stp ^= 1;
            }
        }
        cc += nchunks;
    }
    // every issued MMA must finish before tensor memory is freed
    if (lane == 0) {
        mma_commit(&bars->drain);
        int dummy = 0;
        cx.abort_flag = &dummy;
        cx.limit = kDrainLimitNs;
        wait_bar(&bars->drain, 0, cx);
    }
}

// Item k of a CTA where none are counted out: rows of gridDim.x items, taken from the left and the right in
// turn.
__device__ __forceinline__ int item_at(int k) {
    return k * (int)gridDim.x + (int)((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
__device__ __forceinline__ int item_count(int all) {
    const int rows = all / (int)gridDim.x;
    return rows + (item_at(rows) < all);
}

template <Kind KIND>
__device__ __forceinline__ Item find_item(const DeltaParams &p, const uint8_t *ws, const int32_t *order,
                                          const Split &split, int which, int &slot0) {
    constexpr bool SPLIT = KIND == SEGMENT;
    Item item{nullptr, nullptr, 0, 0, 0, 0, 1};
    const int chains = p.B * p.H;
    const int chain = SPLIT ? which % chains : which;
    const int h = chain % p.H, want = chain / p.H;
    const int32_t *plan = split.plan;
    const int entry = KIND == PLANNED ? plan[(split.pass == 2 ? kPlanList2 : kPlanList1) + want] : 0;
    // Longest request first where there is more than one row of items.
    const int b = KIND == PLANNED ? entry & 1023 : !SPLIT && order ? order[want] : want;
    item.h = h;
    const int slot = p.state_idx[b];
    const int t_req0 = p.cu_seqlens[b], t_req1 = p.cu_seqlens[b + 1];
    const bool prefix = p.prefix_mask[b];
    const bool disorder = *reinterpret_cast<const int *>(ws + OFF_DISORDER) != 0;
    if (slot < 0 || slot >= p.num_slots) {
        atomicOr(p.err, ERR_BIT_SLOT_RANGE);
        return item;
    }
    if (disorder || !request_ok(p, t_req0, t_req1)) {
        atomicOr(p.err, ERR_BIT_SEQLENS);
        return item;
    }
    int n = t_req1 - t_req0, c0 = 0;  // tokens, first chunk
    float *state = p.pool + ((size_t)slot * p.H + h) * kMat;
    if (prefix) item.from = state;
    if (!prefix || n > 0) item.to = state;
    if (SPLIT) {
        const int nchunks = (n + C - 1) / C;
        const int base = split_base(split, nchunks), last = split_last(split, nchunks);
        float *starts = split.starts + (size_t)chain * (split.segs - 1) * kMat;
        const Job job = split_job(p, split);
        const int seg = job.seg;
        // no such segment, or one whose end state nothing needs
        if (seg > last || (seg == last && !job.emit)) return Item{nullptr, nullptr, 0, 0, 0, 0, 0};
        if (seg > 0) item.from = split.pass == 2 ? starts + (seg - 1) * kMat : nullptr;
        if (job.transition)
            item.to = split.trans + ((size_t)chain * (split.segs - 2) + seg - 1) * kMat;
        else if (seg < last)
            item.to = split.pass == 2 ? nullptr : starts + seg * kMat;
        c0 = seg ? (split.ratio + seg - 1) * base : 0;
        n = seg < last ? (seg ? base : split.ratio * base) * C : n - c0 * C;
    }
    if (KIND == PLANNED) {
        const int nchunks = (n + C - 1) / C, a = plan[kPlanA], len = plan[kPlanB];
        const int seg = (entry >> 10) & 1023, last = segments_after(nchunks, a, len);
        // start state g of head h; the transitions stand behind all start states
        auto mat = [&](int x) { return split.starts + ((size_t)x * p.H + h) * kMat; };
        auto start = [&](int g) { return mat(plan[kPlanS + b] + g - 1); };
        const bool second = split.pass == 2;
        item.transition = (entry & kPlanTrans) != 0;
        item.emit = second || seg == 0;
        if (seg > 0) item.from = second ? start(seg) : nullptr;
        if (item.transition)
            item.to = mat(plan[kPlanStarts] + plan[kPlanT + b] + seg - 1);
        else if (seg < last)
            item.to = second ? nullptr : start(seg + 1);
        c0 = seg ? a + (seg - 1) * len : 0;
        n = seg < last ? (seg ? len : a) * C : n - c0 * C;
    }
    item.t0 = t_req0 + c0 * C;
    item.n = n;
    slot0 = (t_req0 >> 6) + b + c0;
    return item;
}

template <Kind KIND>
__device__ void producer_role(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, Bars *bars,
                              uint8_t *sm, const DeltaParams &p, const uint8_t *ws, const int32_t *order,
                              const Split &split, int32_t *taken, int all, int items, Item item, int slot0,
                              Ctx cx) {
    int kq = 0, vv = 0;  // chunks whose K and Q, whose T and V are on the way
    const size_t slot_step = (size_t)p.H * SZ_SLOT;
    bool ok = true;
    for (int k = 0; ok && k < items; ++k) {
        if (k > 0) {
            // items come longest first, and the next one goes to the CTA that is ready for it first
            const int which = taken ? (int)gridDim.x + atomicAdd(taken, 1) : item_at(k);
            if (which >= all) {
                item.n = -1;  // no more
                item.from = nullptr;
                items = k;
            } else {
                item = find_item<KIND>(p, ws, order, split, which, slot0);
            }
            if (item.from && item.n > 0) bulk_prefetch(item.from, kMat * sizeof(float));
            if (k >= kItems && !wait_bar<true>(&bars->item_empty[k % kItems], (k / kItems - 1) & 1, cx)) break;
        }
        bars->items[k % kItems] = item;
        mbar_arrive(&bars->item_full[k % kItems]);
        const int nchunks = item.n > 0 ? (item.n + C - 1) / C : 0;
        const uint8_t *slots = ws + ((size_t)slot0 * p.H + item.h) * SZ_SLOT;
        const int xq = (item.h / p.group) * kHeadDim, xv = item.h * kHeadDim;
        for (int c = 0; c < nchunks; ++c) {
            const int st = kq % kStages, g = kq & 1;
            if (kq >= kStages && !(ok = wait_bar<true>(&bars->kq_empty[st], (kq / kStages - 1) & 1, cx))) break;
            uint8_t *dst = sm + OFF_KQ + st * SZ_KQ;
            const int y = item.t0 + c * C;
            mbar_arrive_expect_tx(&bars->kq_full[st], SZ_KQ);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                tma_load_2d(dst + x * 16384, &tk, &bars->kq_full[st], xq + 64 * x, y);
                tma_load_2d(dst + x * 16384 + 8192, &tq, &bars->kq_full[st], xq + 64 * x, y);
            }
            ++kq;
            if (vv >= 2 && !(ok = wait_bar<true>(&bars->y_done[g], ((vv >> 1) - 1) & 1, cx) &&
                                  wait_bar<true>(&bars->c_free[g], ((vv >> 1) - 1) & 1, cx)))
                break;
            mbar_arrive_expect_tx(&bars->t_full[g], SZ_SLOT);
            bulk_load(sm + OFF_T + g * SZ_T, slots + c * slot_step, SZ_SLOT, &bars->t_full[g]);
            mbar_arrive_expect_tx(&bars->v_full[g], 16384);
            tma_load_2d(sm + OFF_V + g * 16384, &tv, &bars->v_full[g], xv, y);
            ++vv;
        }
    }
    // copies still in flight must land before the shared memory goes away
    int dummy = 0;
    cx.abort_flag = &dummy;
    cx.limit = kDrainLimitNs;
    for (int c = kq >= kStages ? kq - kStages : 0; c < kq; ++c)
        wait_bar(&bars->kq_full[c % kStages], (c / kStages) & 1, cx);
    for (int c = vv >= 2 ? vv - 2 : 0; c < vv; ++c) {
        wait_bar(&bars->t_full[c & 1], (c >> 1) & 1, cx);
        wait_bar(&bars->v_full[c & 1], (c >> 1) & 1, cx);
    }
}

// Warp 10: rows of the request's last K tile past its end are zeroed.
__device__ void fix_role(Bars *bars, uint8_t *sm, int items, int lane, const Ctx &cx) {
    int st = 0;
    uint32_t stp = 0;
    for (int k = 0; k < items; ++k) {
        if (!warp_wait<true>(&bars->item_full[k % kItems], (k / kItems) & 1, cx)) return;
        const int n = bars->items[k % kItems].n;
        if (n < 0) return;
        warp_arrive(&bars->item_empty[k % kItems], lane);
        for (int left = n; left > 0; left -= C) {
            if (!warp_wait<true>(&bars->kq_full[st], stp, cx)) return;
            if (left < C) {
                uint8_t *tile = sm + OFF_KQ + st * SZ_KQ;
                for (int x = left * 16 + lane; x < C * 16; x += 32)  // (token, column block, piece)
                    *reinterpret_cast<uint4 *>(tile + ((x >> 3) & 1) * 16384 + (x >> 4) * 128 +
                                               (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            warp_arrive(&bars->kq_ready[st], lane);
            warp_arrive(&bars->kq_empty[st], lane);
            if (++st == kStages) {
                st = 0;
                stp ^= 1;
            }
        }
    }
}

// Items: the chains (SEGMENT: the jobs of a pass), one CTA each, or a CTA per SM that takes several in turn,
// its loads running ahead into the next item.
template <Kind KIND>
__global__ void __launch_bounds__(kThreads, 1)
    delta_extend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const DeltaParams p, const uint8_t *ws,
                        const int32_t *order, const Split split, int32_t *taken, int all_items) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars *bars = reinterpret_cast<Bars *>(sm + OFF_BAR);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->kq_full[s], 1);
            mbar_init(&bars->kq_empty[s], 2);
            mbar_init(&bars->kq_ready[s], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bars->v_full[g], 1);
            mbar_init(&bars->t_full[g], 1);
            mbar_init(&bars->y_done[g], 1);
            mbar_init(&bars->c_free[g], kEWarps);
        }
        for (int k = 0; k < kItems; ++k) {
            mbar_init(&bars->item_full[k], 1);
            mbar_init(&bars->item_empty[k], kEWarps + 2);
        }
        mbar_init(&bars->x_full, 1);
        mbar_init(&bars->y_full, 1);
        mbar_init(&bars->d_full, 1);
        mbar_init(&bars->o_free, kEWarps);
        mbar_init(&bars->drain, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    if (KIND == PLANNED) all_items = split.plan[split.pass == 2 ? kPlanSecond : kPlanFirst] * p.H;
    if (KIND == PLANNED && (int)blockIdx.x >= all_items) return;
    const int items = taken ? 0x7fffffff : item_count(all_items);
    Item first{};
    int slot0 = 0;
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    } else if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        first = find_item<KIND>(p, ws, order, split, item_at(0), slot0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the same in every lane, for the uniform datapath
    const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const Ctx cx{p.wait_limit_ns, &bars->abort_flag, p.err};

    if (warp < kEWarps)
        reg_inc<kRegsE>();
    else
        reg_dec<kRegsRest>();
    if (warp < kEWarps) {
        e_role<KIND>(p, sm, bars, cx, tbase, warp & 3, warp >> 2, lane, items, split);
    } else if (warp == kProducerWarp) {
        if (lane == 0)
            producer_role<KIND>(tq, tk, tv, bars, sm, p, ws, order, split, taken, all_items, items, first,
                                slot0, cx);
    } else if (warp == kMmaWarp) {
        mma_role(bars, tbase, smem_u32(sm), items, lane, cx);
    } else if (warp == kFixWarp) {
        fix_role(bars, sm, items, lane, cx);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, kTmemCols);
    }
}

// The join: a CTA takes COLS columns of one chain's states through all segments, 128 x 128 x COLS fp32 products
// a segment, 4 x 4 of them a thread (8 COLS threads); M is fetched one segment ahead (64 KB, from L2).  Bound by
// the latency of its shared-memory loads, so with few chains the columns go to more CTAs, of which an SM holds
// one: one request of 16,384 tokens with 32 / 16 columns, 8 heads 202 / 190 us, 16 heads 285 / 273, 32 heads
// (more CTAs than SMs at 16 columns) 445 / 449.
constexpr int kJoinPitch = kHeadDim + 4;
constexpr uint32_t join_smem_bytes(int cols) {
    return (2 * kHeadDim * kJoinPitch + 2 * kHeadDim * cols) * sizeof(float);
}
template <int COLS>
__device__ __forceinline__ void fetch_mat(float *dst, const float *src) {
    for (int x = threadIdx.x; x < (int)kMat / 4; x += 8 * COLS)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         smem_u32(dst + (x >> 5) * kJoinPitch + (x & 31) * 4)),
                     "l"(src + 4 * x)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// starts: S_1, N_1, .. of one chain, trans: M_1, .., step values apart.
template <int COLS>
__device__ __forceinline__ void join_chain(float *starts, const float *trans, size_t step, int last, float *ms,
                                           float *ss) {
    if (last < 2) return;
    fetch_mat<COLS>(ms, trans);
    // rows k0 + 32 i and columns v .. v + 3 of a thread
    const int v = threadIdx.x % (COLS / 4) * 4, k0 = threadIdx.x / (COLS / 4);
    starts += v;
    ss += v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(ss + (k0 + 32 * i) * COLS) =
            *reinterpret_cast<const float4 *>(starts + (k0 + 32 * i) * kHeadDim);
    for (int g = 1; g < last; ++g) {
        const float *m = ms + ((g - 1) & 1) * kHeadDim * kJoinPitch + k0 * kJoinPitch;
        const float *s = ss + ((g - 1) & 1) * kHeadDim * COLS;
        float *next = starts + g * step;
        float4 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum[i] = *reinterpret_cast<const float4 *>(next + (k0 + 32 * i) * kHeadDim);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // M_g and S_g are there, and all are done with the other buffers
        if (g + 1 < last) fetch_mat<COLS>(ms + (g & 1) * kHeadDim * kJoinPitch, trans + g * step);
#pragma unroll 4
        for (int j = 0; j < kHeadDim; j += 4) {
            float4 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = *reinterpret_cast<const float4 *>(m + 32 * i * kJoinPitch + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 x = *reinterpret_cast<const float4 *>(s + (j + e) * COLS);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = e == 0 ? f[i].x : e == 1 ? f[i].y : e == 2 ? f[i].z : f[i].w;
                    sum[i].x = fmaf(y, x.x, sum[i].x);
                    sum[i].y = fmaf(y, x.y, sum[i].y);
                    sum[i].z = fmaf(y, x.z, sum[i].z);
                    sum[i].w = fmaf(y, x.w, sum[i].w);
                }
            }
        }
        float *keep = ss + (g & 1) * kHeadDim * COLS;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<float4 *>(keep + (k0 + 32 * i) * COLS) = sum[i];
            *reinterpret_cast<float4 *>(next + (k0 + 32 * i) * kHeadDim) = sum[i];
        }
    }
}

template <int COLS>
__global__ void __launch_bounds__(8 * COLS)
    delta_join_kernel(const DeltaParams p, const Split split) {
    extern __shared__ __align__(16) float join_smem[];
    float *ms = join_smem, *ss = join_smem + 2 * kHeadDim * kJoinPitch;
    pdl_wait();
    pdl_trigger();
    constexpr int kParts = kHeadDim / COLS;
    const int32_t *plan = split.plan;
    const int all = (plan ? plan[kPlanJoins] : p.B) * p.H * kParts;
    for (int x = blockIdx.x; x < all; x += gridDim.x) {
        const int chain = x / kParts, v0 = x % kParts * COLS;
        const int h = chain % p.H, b = plan ? plan[kPlanJoin + chain / p.H] : chain / p.H;
        const int t0 = p.cu_seqlens[b], t1 = p.cu_seqlens[b + 1];
        if (!request_ok(p, t0, t1)) continue;
        const int nchunks = (t1 - t0 + C - 1) / C;
        if (plan) {
            join_chain<COLS>(split.starts + ((size_t)plan[kPlanS + b] * p.H + h) * kMat + v0,
                       split.starts + ((size_t)(plan[kPlanStarts] + plan[kPlanT + b]) * p.H + h) * kMat,
                       p.H * kMat, segments_after(nchunks, plan[kPlanA], plan[kPlanB]), ms, ss);
        } else {
            join_chain<COLS>(split.starts + (size_t)chain * (split.segs - 1) * kMat + v0,
                       split.trans + (size_t)chain * (split.segs - 2) * kMat, kMat, split_last(split, nchunks),
                       ms, ss);
        }
        __syncthreads();  // the buffers are free
    }
}

using JoinKernel = void (*)(const DeltaParams, const Split);
JoinKernel join_kernel(int cols) {
    return cols == 8 ? delta_join_kernel<8> : cols == 16 ? delta_join_kernel<16> : delta_join_kernel<32>;
}
// Bytes of the slots, of the order, of a split's matrices.
unsigned long long slots_bytes(long long B, long long T, long long H) {
    return ((unsigned long long)chunk_slots(T, B) * (unsigned long long)H * SZ_SLOT);
}
unsigned long long order_bytes(long long B) {
    return (unsigned long long)order_ints((int)B) * sizeof(int32_t);
}

}  // namespace

unsigned long long delta_scratch_bytes(long long B, long long T, long long H) {
    if (T <= 0 || B <= 0) return 0ull;
    const long long chunks = (T + C - 1) / C;
    const unsigned long long mat = kMat * sizeof(float);
    return slots_bytes(B, T, H) + order_bytes(B) + split_mats(B * H, chunks) * mat +
           (planned(B, H, chunks, chunks) ? kPlanBytes + kPlanMats * mat : 0ull);
}

cudaError_t launch_delta_extend(const DeltaParams &p, void *ws, int num_sms, cudaStream_t stream) {
    const long long ctas = (long long)p.B * p.H;
    const long long t_ctas = chunk_slots(p.T, p.B) * p.H;
    CUtensorMap tq, tk, tv;
    if (!make_rows_map(&tq, p.q, p.T, (long long)p.Hk * kHeadDim, p.q_rs, 64, C, true) ||
        !make_rows_map(&tk, p.k, p.T, (long long)p.Hk * kHeadDim, p.k_rs, 64, C, true) ||
        !make_rows_map(&tv, p.v, p.T, (long long)p.H * kHeadDim, p.v_rs, kHeadDim, C, false))
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
            for (auto *kernel : {delta_extend_kernel<MANY>, delta_extend_kernel<ONE>,
                                 delta_extend_kernel<SEGMENT>, delta_extend_kernel<PLANNED>}) {
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
                if (e != cudaSuccess) return e;
            }
            for (auto *kernel : {delta_t_kernel<false>, delta_t_kernel<true>}) {
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTSmemBytes);
                if (e != cudaSuccess) return e;
            }
            for (const int cols : {8, 16, 32}) {
                e = cudaFuncSetAttribute(join_kernel(cols), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)join_smem_bytes(cols));
                if (e != cudaSuccess) return e;
            }
            configured[dev] = true;
        }
    }
    uint8_t *w = static_cast<uint8_t *>(ws);
    int32_t *order = nullptr, *plan = nullptr;
    int first_ctas = 1;
    const Schedule how = make_schedule(p.B, p.T, p.H, p.max_seqlen, num_sms);
    if (how.planned) {
        plan = reinterpret_cast<int32_t *>(w + slots_bytes(p.B, p.T, p.H) + order_bytes(p.B));
    } else if (how.ranked) {
        order = reinterpret_cast<int32_t *>(w + slots_bytes(p.B, p.T, p.H));
        first_ctas = (p.B + kTThreads - 1) / kTThreads;
    }
    e = launch_pdl(plan ? delta_t_kernel<true> : delta_t_kernel<false>, dim3((unsigned)(first_ctas + t_ctas)),
                   dim3(kTThreads), kTSmemBytes, stream, tq, tk, p, w, order, plan, first_ctas);
    if (e != cudaSuccess) return e;
    Split split{how.cut, 0, nullptr, nullptr, nullptr};
    if (plan) {
        split.plan = plan;
        split.starts = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(plan) + kPlanBytes);
        for (split.pass = 1; split.pass <= 2; ++split.pass) {
            if (split.pass == 2) {
                e = launch_pdl(join_kernel(16), dim3((unsigned)num_sms), dim3(8 * 16), join_smem_bytes(16),
                               stream, p, split);
                if (e != cudaSuccess) return e;
            }
            e = launch_pdl(delta_extend_kernel<PLANNED>, dim3((unsigned)num_sms), dim3(kThreads), kSmemBytes,
                           stream, tq, tk, tv, p, (const uint8_t *)w, (const int32_t *)nullptr, split,
                           plan + (split.pass == 2 ? kPlanTaken2 : kPlanTaken1), 0);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    if (split.segs == 1)
        return launch_pdl(ctas > num_sms ? delta_extend_kernel<MANY> : delta_extend_kernel<ONE>,
                          dim3((unsigned)(ctas < num_sms ? ctas : num_sms)), dim3(kThreads), kSmemBytes,
                          stream, tq, tk, tv, p, (const uint8_t *)w, (const int32_t *)order, split,
                          order ? order + order_ints(p.B) - 1 : (int32_t *)nullptr, (int)ctas);
    split.starts = reinterpret_cast<float *>(w + slots_bytes(p.B, p.T, p.H) + order_bytes(p.B));
    split.trans = split.starts + (size_t)ctas * (split.segs - 1) * kMat;
    split.pass = 1;
    e = launch_pdl(delta_extend_kernel<SEGMENT>, dim3((unsigned)(ctas * (2 * split.segs - 3))), dim3(kThreads),
                   kSmemBytes, stream, tq, tk, tv, p, (const uint8_t *)w, (const int32_t *)nullptr, split,
                   (int32_t *)nullptr, (int)(ctas * (2 * split.segs - 3)));
    if (e != cudaSuccess) return e;
    int cols = 32;
    while (cols > 8 && ctas * (kHeadDim / cols) * 2 <= num_sms) cols /= 2;
    e = launch_pdl(join_kernel(cols), dim3((unsigned)(ctas * (kHeadDim / cols))), dim3(8 * cols),
                   join_smem_bytes(cols), stream, p, split);
    if (e != cudaSuccess) return e;
    split.pass = 2;
    return launch_pdl(delta_extend_kernel<SEGMENT>, dim3((unsigned)(ctas * (split.segs - 1))), dim3(kThreads),
                      kSmemBytes, stream, tq, tk, tv, p, (const uint8_t *)w, (const int32_t *)nullptr, split,
                      (int32_t *)nullptr, (int)(ctas * (split.segs - 1)));
}

}  // namespace la
