// la_delta_extend.cu -- chunked gated delta rule on the 5th-generation tensor cores, one CTA per
// (request, value head) or per half of its value columns.
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
// Every exponent is formed as a difference of sums that are exact in fixed point, so that steep
// decays lose nothing; factors are at most 1.
//
// Stacked operands.  K and Q of a chunk share one [128][128] tile, interleaved by 16 rows (rows 32 a ..
// + 15: tokens 16 a .. of K, the next 16 the same tokens of Q), so that every product has M = 128: an
// M = 64 or N = 64 tcgen05.mma costs about what the full one does.  One product of the tile with its own
// transpose gives K K^T, Q K^T and, on its diagonal, the squared norms; [T'; P T] is stacked the same
// way, so that T' R and P T R are one product, and the output needs no product after U.
//
// Precision.  Products run in bf16 with fp32 accumulation.  K, Q are used as loaded; the operands that
// are computed (S, R, T', P T, U) are bf16 pairs hi + lo, off by at most 2^-16 and about a sixth of that
// in the mean; U takes R itself in fp32 and only T' R through pairs; the state stays in fp32
// registers and is never accumulated in tensor memory.
//
// Roles (512 threads, one CTA per SM):
//   warps 0-3   T: per chunk the gate sums and norms, A and P from tensor memory, T by blocks of 16
//               (diagonal blocks by substitution in fp32, the others with warp-level MMAs from bf16
//               pairs), P T; a chunk ahead of the rest.
//   warps 4-11  E: the state (32 k rows x 64 v columns a warp) and the passes R, U, O and S.
//   warp 12     TMA producer; warp 13 tensor-memory owner and MMA issuer;
//   warp 14     zeroes the tile rows past the end of the request's last chunk (they hold the next
//               request's tokens, and 0 x NaN is NaN).
// Per chunk the chain is X -> R -> T' R -> U -> K^T U -> S; the product for the next chunk's T runs under
// R, the output pass under K^T U.
//
// Every wait is an mbarrier wait with a deadline; one that runs out sets the error word and an abort flag
// that ends every role, then the CTA waits for its copies and MMAs, frees tensor memory and exits.
#include <cuda.h>
#include <string.h>

#include <mutex>

#include "la_delta.h"
#include "la_sm100.cuh"

namespace la {

namespace {

using namespace sm100;

constexpr int C = 64;  // tokens of a chunk
constexpr int kTWarps = 4, kEWarps = 8;
constexpr int kProducerWarp = 12, kMmaWarp = 13, kFixWarp = 14;
constexpr int kThreads = 512;
// registers per thread of the roles: 64 + 128 + 2 x 160 = 4 x 128, the launch's share
constexpr int kRegsT = 128, kRegsE = 160, kRegsRest = 64;
static_assert(kRegsT + 2 * kRegsE + kRegsRest <= 512, "register split");
constexpr float kScale = 0.08838834764831845f;  // 128^-0.5

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_X = 0, TM_Y = 128, TM_A = 256, TM_D = 384;

// Shared memory, from a 1024-byte aligned base.  Operand tiles are 128-byte-swizzled blocks of 64
// columns; the blocks of [128]-row tiles lie 16 KiB apart, those of [64]-row tiles 8 KiB.
constexpr uint32_t OFF_KQ = 0;                     // 2 stages x [128][128]
constexpr uint32_t OFF_V = OFF_KQ + 2 * 32768;     // [64][128]
constexpr uint32_t OFF_SHI = OFF_V + 16384;        // [128][128] hi, lo
constexpr uint32_t OFF_SLO = OFF_SHI + 32768;
constexpr uint32_t OFF_RHI = OFF_SLO + 32768;      // [64][128] hi, lo: R, then U
constexpr uint32_t OFF_RLO = OFF_RHI + 16384;
constexpr uint32_t OFF_THI = OFF_RLO + 16384;      // [128][64] hi, lo: T' and P T, interleaved
constexpr uint32_t OFF_TLO = OFF_THI + 16384;
// 16 x 16 blocks of the inversion, as two panels of 8 columns x 16 rows x 16 bytes: the blocks of A
// below the diagonal (hi, lo), the diagonal blocks of T (hi, lo), and A's diagonal blocks in fp32,
// transposed
constexpr uint32_t OFF_AB = OFF_TLO + 16384;       // 6 x (512 hi + 512 lo)
constexpr uint32_t OFF_TD = OFF_AB + 6 * 1024;     // 4 x (512 hi + 512 lo)
constexpr uint32_t OFF_AD = OFF_TD + 4 * 1024;     // 4 x 1024
constexpr uint32_t OFF_TOK = OFF_AD + 4 * 1024;    // per token: ghi, glo, rk, beta rk, scale rq
constexpr uint32_t OFF_COEF = OFF_TOK + 5 * 256;   // 2 x per token: beta, beta gamma rk, lam rk, out
constexpr uint32_t OFF_BAR = OFF_COEF + 2 * 1024;
constexpr uint32_t SZ_BAR = 320;
constexpr uint32_t kSmemBytes = OFF_BAR + SZ_BAR + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Bars {
    uint64_t kq_full[2], kq_empty[2];
    uint64_t v_full;
    uint64_t kq_last;      // producer: the last chunk's loads are issued
    uint64_t kq_fixed;     // warp 14: rows past the end of the last chunk zeroed
    uint64_t a_full;       // A = [K; Q] [K; Q]^T done
    uint64_t a_free;       // T warps: A read (4)
    uint64_t t_sync[3];    // among the T warps (4)
    uint64_t coef[2];      // T warps: the chunk's coefficients written (4); two, as the T warps may
                           // be a chunk ahead of a reader
    uint64_t t_ready;      // T warps: T', P T written (4)
    uint64_t x_full, y_full, d_full;
    uint64_t r_ready, u_ready, s_ready, o_free;  // E warps (8)
    uint64_t drain;
    float gend[2];         // e^{G_C} of the chunk
    uint32_t tmem_base;
    int abort_flag;
    int request;
};
static_assert(sizeof(Bars) <= SZ_BAR, "barrier block");

constexpr uint64_t kDrainLimitNs = 2000000000ull;

struct Ctx {
    uint64_t limit;
    volatile int *abort_flag;
    unsigned int *err;
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const Ctx &cx) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(a, parity)) return true;
        if (*cx.abort_flag) return false;
        if (globaltimer_ns() - t0 > cx.limit) {
            *cx.abort_flag = 1;
            atomicOr(cx.err, ERR_BIT_TIMEOUT);
            return false;
        }
    }
}
// All lanes wait; the warp goes on only if every lane's wait succeeded.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Ctx &cx) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, cx));
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(x0, x1);
    lo = pack_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
}

// A 16 x 16 accumulator (two 16 x 8 fragments) as the bf16 pair of an A operand.
__device__ __forceinline__ void split_frag(const float (&c)[8], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(c[0], c[1], hi[0], lo[0]);
    split2(c[2], c[3], hi[1], lo[1]);
    split2(c[4], c[5], hi[2], lo[2]);
    split2(c[6], c[7], hi[3], lo[3]);
}

// acc += A B with A and B bf16 pairs (the product of the two lo parts, 2^-16, is left out).
__device__ __forceinline__ void prod16(float (&acc)[8], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                       const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        mma_16816(acc + 4 * n, ah, bh[2 * n], bh[2 * n + 1]);
        mma_16816(acc + 4 * n, ah, bl[2 * n], bl[2 * n + 1]);
        mma_16816(acc + 4 * n, al, bh[2 * n], bh[2 * n + 1]);
    }
}

// ------------------------------------------------------------------------------------------------
// T warps

// 2^40 log2(e) g as a fixed-point number, -1e4 standing for everything below (e^-1e4 is 0 in fp32,
// and the sums of a chunk stay finite), 1e4 for everything above.
__device__ __forceinline__ long long gate_fixed(float g) {
    constexpr float kHi = 1.44269502162933349609f;   // log2(e) in fp32
    constexpr float kLo = 1.92596299112661746887e-8f;  // the rest
    g = g < -1e4f ? -1e4f : g > 1e4f ? 1e4f : g;
    const float p = g * kHi;
    const float e = fmaf(g, kHi, -p) + g * kLo;
    return __float2ll_rn(p * 1099511627776.f) + __float2ll_rn(e * 1099511627776.f);
}
constexpr float kFixedStep = 9.094947017729282379e-13f;  // 2^-40

__device__ void t_role(const DeltaParams &p, uint8_t *sm, Bars *bars, const Ctx &cx, uint32_t tbase,
                       int a, int lane, size_t t0, int n, int h, int nchunks) {
    float *tok = reinterpret_cast<float *>(sm + OFF_TOK);
    float *ghi = tok, *glo = tok + 64, *rk = tok + 128, *brk = tok + 192, *qs = tok + 256;
    const uint32_t ab = smem_u32(sm + OFF_AB), td = smem_u32(sm + OFF_TD);
    const uint32_t thi = smem_u32(sm + OFF_THI);
    float *ad = reinterpret_cast<float *>(sm + OFF_AD) + a * 256;
    const int row = lane >> 2, cp = (lane & 3) * 2;  // fragment row, column pair
    const int mrow = lane & 7, midx = lane >> 3;     // ldmatrix: row, matrix
    // operand blocks: matrices (panel, row half); the same for transposed A and for [n][k] B
    const uint32_t off_p = (uint32_t)((midx & 1) * 256 + (midx >> 1) * 128 + mrow * 16);
    const uint32_t lane_k = tbase + TM_A + ((uint32_t)(a * 32) << 16);

    const float *gp = p.g + (t0 * p.H + h), *bp = p.beta + (t0 * p.H + h);
    float gn0 = 0.f, gn1 = 0.f, bn = 0.f;
    auto fetch = [&](int c) {  // gates of tokens lane and lane + 32, beta of this warp's token
        const int r = n - c * C;
        const size_t at = (size_t)c * C;
        gn0 = lane < r ? gp[(at + lane) * p.H] : 0.f;
        gn1 = lane + 32 < r ? gp[(at + lane + 32) * p.H] : 0.f;
        const int i = 16 * a + (lane & 15);
        bn = i < r ? bp[(at + i) * p.H] : 0.f;
    };
    if (nchunks > 0) fetch(0);

    for (int c = 0; c < nchunks; ++c) {
        const uint32_t par = c & 1;
        // running sums of the gates: every warp forms all 64
        long long x0 = gate_fixed(gn0), x1 = gate_fixed(gn1);
        // a NaN has no fixed-point form: it is passed on through beta
        const uint32_t bad = a < 2 ? __ballot_sync(0xffffffffu, gn0 != gn0)
                                   : __ballot_sync(0xffffffffu, gn1 != gn1);
        const float beta =
            (bad >> (16 * (a & 1) + (lane & 15))) & 1u ? __uint_as_float(0x7fffffffu) : bn;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y0 = __shfl_up_sync(0xffffffffu, x0, d);
            const long long y1 = __shfl_up_sync(0xffffffffu, x1, d);
            if (lane >= d) {
                x0 += y0;
                x1 += y1;
            }
        }
        x1 += __shfl_sync(0xffffffffu, x0, 31);
        const long long xend = __shfl_sync(0xffffffffu, x1, 31);
        // this warp's tokens 16 a + (lane % 16)
        const long long xi =
            __shfl_sync(0xffffffffu, a < 2 ? x0 : x1, 16 * (a & 1) + (lane & 15));
        if (c + 1 < nchunks) fetch(c + 1);

        if (!warp_wait(&bars->a_full, par, cx)) return;
        tc_fence_after();
        {
            // squared norms: K's in lanes 0-15, Q's in lanes 16-31, of tokens 16 a + lane % 16
            uint32_t dg[32];
            tmem_ld32(lane_k + (uint32_t)(a * 32), dg);
            tmem_ld_wait_regs(dg);
            float nn = 0.f;
#pragma unroll
            for (int x = 0; x < 32; ++x) nn = lane == x ? __uint_as_float(dg[x]) : nn;
            const float inv = p.l2norm ? 1.f / sqrtf(nn + kDeltaEps) : 1.f;
            const int i = 16 * a + (lane & 15);
            const float gam = ex2((float)xi * kFixedStep);
            float *cf = reinterpret_cast<float *>(sm + OFF_COEF + par * 1024);
            if (lane < 16) {
                const float hi = (float)xi;
                ghi[i] = hi * kFixedStep;
                glo[i] = (float)(xi - __float2ll_rn(hi)) * kFixedStep;
                rk[i] = inv;
                brk[i] = beta * inv;
                cf[i] = beta;
                cf[64 + i] = beta * gam * inv;
                cf[128 + i] = ex2((float)(xend - xi) * kFixedStep) * inv;
            } else {
                qs[i] = kScale * inv;
                cf[192 + i] = kScale * gam * inv;
            }
            if (a == 0 && lane == 0) bars->gend[par] = ex2((float)xend * kFixedStep);
        }
        warp_arrive(&bars->t_sync[0], lane);
        if (!warp_wait(&bars->t_sync[0], par, cx)) return;
        if (lane == 0) mbar_arrive(&bars->coef[par]);

        // ---- A and P of row block a
        uint32_t ph[4][4], pl[4][4];
        {
            const int i0 = 16 * a + row, i1 = i0 + 8;
            const float gh0 = ghi[i0], gh1 = ghi[i1], gl0 = glo[i0], gl1 = glo[i1];
            const float ai0 = brk[i0], ai1 = brk[i1], qi0 = qs[i0], qi1 = qs[i1];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b > a) break;
                uint32_t kk[8], qk[8];
                tmem_ld16x256_pair_wait(lane_k + (uint32_t)(b * 32),
                                        lane_k + (16u << 16) + (uint32_t)(b * 32), kk, qk);
                float pv[8];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int j = 16 * b + 8 * hf + cp;
                    const float2 gh = *reinterpret_cast<const float2 *>(ghi + j);
                    const float2 gl = *reinterpret_cast<const float2 *>(glo + j);
                    const float2 rj = *reinterpret_cast<const float2 *>(rk + j);
                    const float e00 = ex2((gh0 - gh.x) + (gl0 - gl.x)) * rj.x;
                    const float e01 = ex2((gh0 - gh.y) + (gl0 - gl.y)) * rj.y;
                    const float e10 = ex2((gh1 - gh.x) + (gl1 - gl.x)) * rj.x;
                    const float e11 = ex2((gh1 - gh.y) + (gl1 - gl.y)) * rj.y;
                    float a00 = __uint_as_float(kk[4 * hf]) * (e00 * ai0);
                    float a01 = __uint_as_float(kk[4 * hf + 1]) * (e01 * ai0);
                    float a10 = __uint_as_float(kk[4 * hf + 2]) * (e10 * ai1);
                    float a11 = __uint_as_float(kk[4 * hf + 3]) * (e11 * ai1);
                    pv[4 * hf] = __uint_as_float(qk[4 * hf]) * (e00 * qi0);
                    pv[4 * hf + 1] = __uint_as_float(qk[4 * hf + 1]) * (e01 * qi0);
                    pv[4 * hf + 2] = __uint_as_float(qk[4 * hf + 2]) * (e10 * qi1);
                    pv[4 * hf + 3] = __uint_as_float(qk[4 * hf + 3]) * (e11 * qi1);
                    if (b == a) {
                        if (j > i0) pv[4 * hf] = 0.f;
                        if (j + 1 > i0) pv[4 * hf + 1] = 0.f;
                        if (j > i1) pv[4 * hf + 2] = 0.f;
                        if (j + 1 > i1) pv[4 * hf + 3] = 0.f;
                        const int m = 8 * hf + cp;
                        ad[m * 16 + row] = j < i0 ? a00 : 0.f;
                        ad[(m + 1) * 16 + row] = j + 1 < i0 ? a01 : 0.f;
                        ad[m * 16 + row + 8] = j < i1 ? a10 : 0.f;
                        ad[(m + 1) * 16 + row + 8] = j + 1 < i1 ? a11 : 0.f;
                    } else {
                        uint32_t h0, l0, h1, l1;
                        split2(a00, a01, h0, l0);
                        split2(a10, a11, h1, l1);
                        uint8_t *blk = sm + OFF_AB + (a * (a - 1) / 2 + b) * 1024 + hf * 256 +
                                       row * 16 + cp * 2;
                        *reinterpret_cast<uint32_t *>(blk) = h0;
                        *reinterpret_cast<uint32_t *>(blk + 128) = h1;
                        *reinterpret_cast<uint32_t *>(blk + 512) = l0;
                        *reinterpret_cast<uint32_t *>(blk + 640) = l1;
                    }
                }
                split_frag(pv, ph[b], pl[b]);
            }
        }
        tc_fence_before();
        warp_arrive(&bars->a_free, lane);

        // ---- the diagonal block of T: column j = lane % 16 by substitution
        float x[16];
        {
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
            // lanes 0-15 keep the hi parts, lanes 16-31 the lo parts
            uint8_t *dst = sm + OFF_TD + a * 1024 + (lane >> 4) * 512 + (j >> 3) * 256 + (j & 7) * 2;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
                const __nv_bfloat16 lo = __float2bfloat16_rn(x[i] - __bfloat162float(hi));
                *reinterpret_cast<__nv_bfloat16 *>(dst + i * 16) = lane < 16 ? hi : lo;
            }
        }
        warp_arrive(&bars->t_sync[1], lane);
        // the previous chunk's product with [T'; P T] is done with the tile
        if (c > 0 && !warp_wait(&bars->y_full, (c - 1) & 1, cx)) return;
        {
            const int j = lane & 15;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int rho = 32 * a + i;
                const float v = i > j ? x[i] : 0.f;
                const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                const __nv_bfloat16 lo = __float2bfloat16_rn(v - __bfloat162float(hi));
                *reinterpret_cast<__nv_bfloat16 *>(sm + (lane < 16 ? OFF_THI : OFF_TLO) + rho * 128 +
                                                   (((2 * a + (j >> 3)) ^ (rho & 7)) << 4) +
                                                   (j & 7) * 2) = lane < 16 ? hi : lo;
            }
        }
        if (!warp_wait(&bars->t_sync[1], par, cx)) return;

        // ---- column block b = a of T below the diagonal, as its transpose:
        // T_rb^T = -(sum_{b <= m < r} T_mb^T A_rm^T) T_rr^T
        {
            const int b = a;
            uint32_t yh[3][4], yl[3][4];
            ldsm4_t(td + b * 1024 + off_p, yh[0]);
            ldsm4_t(td + b * 1024 + 512 + off_p, yl[0]);
#pragma unroll
            for (int dr = 1; dr < 4; ++dr) {
                const int r = b + dr;
                if (r > 3) break;
                float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int dm = 0; dm < dr; ++dm) {
                    uint32_t bh[4], bl[4];
                    const uint32_t blk = ab + (r * (r - 1) / 2 + b + dm) * 1024 + off_p;
                    ldsm4(blk, bh);
                    ldsm4(blk + 512, bl);
                    prod16(acc, yh[dm], yl[dm], bh, bl);
                }
                uint32_t zh[4], zl[4], bh[4], bl[4];
                split_frag(acc, zh, zl);
                float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                ldsm4(td + r * 1024 + off_p, bh);
                ldsm4(td + r * 1024 + 512 + off_p, bl);
                prod16(t, zh, zl, bh, bl);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = -t[e];
                split_frag(t, zh, zl);
                // matrices (j half, i half) -> rows i of the tile, columns 16 b + j
                const int rho = 32 * r + 8 * (midx >> 1) + mrow;
                const uint32_t at = thi + rho * 128 + (((2 * b + (midx & 1)) ^ (rho & 7)) << 4);
                stsm4_t(at, zh);
                stsm4_t(at + (OFF_TLO - OFF_THI), zl);
                if (dr < 3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        yh[dr][e] = zh[e];
                        yl[dr][e] = zl[e];
                    }
                }
            }
        }
        warp_arrive(&bars->t_sync[2], lane);
        if (!warp_wait(&bars->t_sync[2], par, cx)) return;

        // ---- row block a of P T
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (b > a) break;
            float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = b; m < 4; ++m) {
                if (m > a) break;
                uint32_t bh[4], bl[4];
                const int k = (midx & 1) * 8 + mrow, nh = midx >> 1;
                if (m == b) {
                    const uint32_t at = td + b * 1024 + nh * 256 + k * 16;
                    ldsm4_t(at, bh);
                    ldsm4_t(at + 512, bl);
                } else {
                    const int rho = 32 * m + k;
                    const uint32_t at = thi + rho * 128 + (((2 * b + nh) ^ (rho & 7)) << 4);
                    ldsm4_t(at, bh);
                    ldsm4_t(at + (OFF_TLO - OFF_THI), bl);
                }
                prod16(acc, ph[m], pl[m], bh, bl);
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t h0, l0, h1, l1;
                split2(acc[4 * hf], acc[4 * hf + 1], h0, l0);
                split2(acc[4 * hf + 2], acc[4 * hf + 3], h1, l1);
                const int rho = 32 * a + 16 + row;  // and rho + 8: the same rho % 8
                uint8_t *dst =
                    sm + OFF_THI + rho * 128 + (((2 * b + hf) ^ (rho & 7)) << 4) + cp * 2;
                *reinterpret_cast<uint32_t *>(dst) = h0;
                *reinterpret_cast<uint32_t *>(dst + 1024) = h1;
                *reinterpret_cast<uint32_t *>(dst + (OFF_TLO - OFF_THI)) = l0;
                *reinterpret_cast<uint32_t *>(dst + (OFF_TLO - OFF_THI) + 1024) = l1;
            }
        }
        fence_proxy_async_smem();
        warp_arrive(&bars->t_ready, lane);
    }
}

// ------------------------------------------------------------------------------------------------
// E warps: quarter q of the lanes, half hf of the CTA's NV value columns.

// A thread's fragment rows (tokens 16 q + lane / 4 and + 8) of its CW columns into the [64][NV] tiles.
template <int CW>
__device__ __forceinline__ void store_rows_split(uint8_t *sm, int i0, int sw, int col0, int cp,
                                                 const float (&x)[CW / 2]) {
#pragma unroll
    for (int j = 0; j < CW / 8; ++j) {
        const int col = col0 + 8 * j;
        const uint32_t off = (uint32_t)(col >> 6) * 8192u + (uint32_t)i0 * 128u +
                             (((uint32_t)((col & 63) >> 3) ^ (uint32_t)sw) << 4) + (uint32_t)cp * 2u;
        uint32_t h0, l0, h1, l1;
        split2(x[4 * j], x[4 * j + 1], h0, l0);
        split2(x[4 * j + 2], x[4 * j + 3], h1, l1);
        *reinterpret_cast<uint32_t *>(sm + OFF_RHI + off) = h0;
        *reinterpret_cast<uint32_t *>(sm + OFF_RLO + off) = l0;
        *reinterpret_cast<uint32_t *>(sm + OFF_RHI + off + 1024) = h1;
        *reinterpret_cast<uint32_t *>(sm + OFF_RLO + off + 1024) = l1;
    }
}

// The thread's row of the state (CW columns from col0) as a bf16 pair into the operand tiles.
template <int CW>
__device__ __forceinline__ void store_state_split(uint8_t *sm, int row, int col0, const float (&S)[CW]) {
#pragma unroll
    for (int k = 0; k < CW / 8; ++k) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(S[8 * k + 2 * e], S[8 * k + 2 * e + 1], hi[e], lo[e]);
        const int col = col0 + 8 * k;
        const uint32_t off = (uint32_t)(col >> 6) * 16384u + (uint32_t)row * 128u +
                             ((uint32_t)(((col & 63) >> 3) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4 *>(sm + OFF_SHI + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(sm + OFF_SLO + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

template <int NV>
__device__ void e_role(const DeltaParams &p, uint8_t *sm, Bars *bars, const Ctx &cx, uint32_t tbase, int q,
                       int hf, int lane, size_t t0, int n, int h, int c0, int slot, bool prefix,
                       int nchunks) {
    constexpr int CW = NV / 2;
    const int col0 = hf * CW;                // of the CTA's NV columns
    const int srow = 32 * q + lane;          // state row
    const int sw = lane >> 2;                // token row % 8 of both fragment rows
    const int i0 = 16 * q + sw, i1 = i0 + 8; // tokens of the chunk
    const int cp = (lane & 3) * 2;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    float *gs = p.pool + (((size_t)slot * p.H + h) * kHeadDim + srow) * kHeadDim + c0 + col0;

    float S[CW];
    if (prefix) {
#pragma unroll
        for (int x = 0; x < CW / 4; ++x) {
            const float4 f = reinterpret_cast<const float4 *>(gs)[x];
            S[4 * x] = f.x;
            S[4 * x + 1] = f.y;
            S[4 * x + 2] = f.z;
            S[4 * x + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int x = 0; x < CW; ++x) S[x] = 0.f;
    }
    if (nchunks > 0) {
        store_state_split<CW>(sm, srow, col0, S);
        fence_proxy_async_smem();
        warp_arrive(&bars->s_ready, lane);
    }

    bool ok = true;
    for (int c = 0; c < nchunks; ++c) {
        const uint32_t par = c & 1;
        const int r = n - c * C;  // tokens from this chunk on
        const float *cf = reinterpret_cast<const float *>(sm + OFF_COEF + par * 1024);
        // ---- R = beta V - (beta gamma rk) X^K
        if (!(ok = warp_wait(&bars->coef[par], (c >> 1) & 1, cx))) break;
        const float b0 = cf[i0], b1 = cf[i1], bx0 = cf[64 + i0], bx1 = cf[64 + i1];
        if (!(ok = warp_wait(&bars->v_full, par, cx))) break;
        if (!(ok = warp_wait(&bars->x_full, par, cx))) break;
        tc_fence_after();
        float R[CW / 2];
        {
            uint32_t w[CW / 2];
            tmem_ld16x256_wait(tbase + lanes + TM_X + (uint32_t)col0, w);
#pragma unroll
            for (int j = 0; j < CW / 8; ++j) {
                const int col = col0 + 8 * j;
                const uint8_t *v = sm + OFF_V + (col >> 6) * 8192 + i0 * 128 +
                                   ((((col & 63) >> 3) ^ sw) << 4) + cp * 2;
                const uint32_t v0 = *reinterpret_cast<const uint32_t *>(v);
                const uint32_t v1 = *reinterpret_cast<const uint32_t *>(v + 1024);
                R[4 * j] = fmaf(-bx0, __uint_as_float(w[4 * j]), b0 * __uint_as_float(v0 << 16));
                R[4 * j + 1] =
                    fmaf(-bx0, __uint_as_float(w[4 * j + 1]), b0 * __uint_as_float(v0 & 0xffff0000u));
                R[4 * j + 2] = fmaf(-bx1, __uint_as_float(w[4 * j + 2]), b1 * __uint_as_float(v1 << 16));
                R[4 * j + 3] =
                    fmaf(-bx1, __uint_as_float(w[4 * j + 3]), b1 * __uint_as_float(v1 & 0xffff0000u));
            }
        }
        if (r < C) {  // rows past the end hold other requests' values
#pragma unroll
            for (int j = 0; j < CW / 8; ++j) {
                if (i0 >= r) R[4 * j] = R[4 * j + 1] = 0.f;
                if (i1 >= r) R[4 * j + 2] = R[4 * j + 3] = 0.f;
            }
        }
        store_rows_split<CW>(sm, i0, sw, col0, cp, R);
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&bars->r_ready, lane);

        // ---- U = R + T' R, scaled for the state update
        const float u0 = cf[128 + i0], u1 = cf[128 + i1];
        if (!(ok = warp_wait(&bars->y_full, par, cx))) break;
        tc_fence_after();
        {
            uint32_t w[CW / 2];
            tmem_ld16x256_wait(tbase + lanes + TM_Y + (uint32_t)col0, w);
#pragma unroll
            for (int j = 0; j < CW / 8; ++j) {
                R[4 * j] = (R[4 * j] + __uint_as_float(w[4 * j])) * u0;
                R[4 * j + 1] = (R[4 * j + 1] + __uint_as_float(w[4 * j + 1])) * u0;
                R[4 * j + 2] = (R[4 * j + 2] + __uint_as_float(w[4 * j + 2])) * u1;
                R[4 * j + 3] = (R[4 * j + 3] + __uint_as_float(w[4 * j + 3])) * u1;
            }
        }
        store_rows_split<CW>(sm, i0, sw, col0, cp, R);
        fence_proxy_async_smem();
        warp_arrive(&bars->u_ready, lane);

        // ---- o = (scale gamma rq) X^Q + P T R
        {
            const float co0 = cf[192 + i0], co1 = cf[192 + i1];
            uint32_t w[CW / 2], y[CW / 2];
            tmem_ld16x256_wait(tbase + lanes + (16u << 16) + TM_X + (uint32_t)col0, w);
            tmem_ld16x256_wait(tbase + lanes + (16u << 16) + TM_Y + (uint32_t)col0, y);
            tc_fence_before();
            warp_arrive(&bars->o_free, lane);
            const size_t tok = t0 + (size_t)c * C;
            __nv_bfloat16 *o0 = p.out + ((tok + i0) * p.H + h) * kHeadDim + c0 + col0;
            __nv_bfloat16 *o1 = p.out + ((tok + i1) * p.H + h) * kHeadDim + c0 + col0;
            const int t4 = lane & 3;
#pragma unroll
            for (int j4 = 0; j4 < CW / 32; ++j4) {
                // the thread's column pairs of four 8-column fragments, for its two rows; a 4 x 4
                // transpose among the row's four lanes leaves lane t4 with fragment t4's 8 columns
                uint32_t o[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 16 * j4 + 4 * e;
                    o[0][e] = pack_bf16x2(fmaf(co0, __uint_as_float(w[at]), __uint_as_float(y[at])),
                                          fmaf(co0, __uint_as_float(w[at + 1]), __uint_as_float(y[at + 1])));
                    o[1][e] =
                        pack_bf16x2(fmaf(co1, __uint_as_float(w[at + 2]), __uint_as_float(y[at + 2])),
                                    fmaf(co1, __uint_as_float(w[at + 3]), __uint_as_float(y[at + 3])));
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t(&v)[4] = o[x];
                    const bool lo2 = t4 < 2;
                    const uint32_t ra = __shfl_xor_sync(0xffffffffu, lo2 ? v[2] : v[0], 2);
                    const uint32_t rb = __shfl_xor_sync(0xffffffffu, lo2 ? v[3] : v[1], 2);
                    if (lo2) { v[2] = ra; v[3] = rb; } else { v[0] = ra; v[1] = rb; }
                    const bool even = (t4 & 1) == 0;
                    const uint32_t rc = __shfl_xor_sync(0xffffffffu, even ? v[1] : v[0], 1);
                    const uint32_t rd = __shfl_xor_sync(0xffffffffu, even ? v[3] : v[2], 1);
                    if (even) { v[1] = rc; v[3] = rd; } else { v[0] = rc; v[2] = rd; }
                    const int i = x ? i1 : i0;
                    if (i < r)
                        *reinterpret_cast<uint4 *>((x ? o1 : o0) + 32 * j4 + 8 * t4) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }

        // ---- S = gamma_C S + K^T U
        const float ge = bars->gend[par];
        if (!(ok = warp_wait(&bars->d_full, par, cx))) break;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < CW / 32; ++x) {
            uint32_t w[32];
            tmem_ld32(tbase + lanes + TM_D + (uint32_t)(col0 + 32 * x), w);
            tmem_ld_wait_regs(w);
#pragma unroll
            for (int y = 0; y < 32; ++y) S[32 * x + y] = fmaf(ge, S[32 * x + y], __uint_as_float(w[y]));
        }
        if (c + 1 < nchunks) {
            store_state_split<CW>(sm, srow, col0, S);
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&bars->s_ready, lane);
        }
    }
    if (ok && !(prefix && nchunks == 0)) {
#pragma unroll
        for (int x = 0; x < CW / 4; ++x)
            reinterpret_cast<float4 *>(gs)[x] =
                make_float4(S[4 * x], S[4 * x + 1], S[4 * x + 2], S[4 * x + 3]);
    }
}

// ------------------------------------------------------------------------------------------------
// MMA issuer (one thread)
template <int NV>
__device__ void mma_role(Bars *bars, uint32_t tbase, uint32_t s_base, int nchunks, bool ragged, Ctx cx) {
    const uint32_t idA = idesc_bf16_f32(128, 128, false, false);
    const uint32_t idX = idesc_bf16_f32(128, NV, false, true);
    const uint32_t idD = idesc_bf16_f32(128, NV, true, true);
    // All operands have the same high descriptor word (8-row groups 1024 bytes apart, 128-byte
    // swizzle), so only low words are kept: start address and leading-dimension offset.
    const uint64_t high = sdesc_sw128(0, 0, 1024);
    auto low = [&](uint32_t off, uint32_t lbo) { return ((s_base + off) >> 4) | ((lbo >> 4) << 16); };
    auto mma = [&](uint32_t d, uint32_t da, uint32_t db, uint32_t id, uint32_t acc) {
        mma_bf16(tbase + d, high | da, high | db, id, acc);
    };
    const uint32_t dKQ = low(OFF_KQ, 16);      // K-major
    const uint32_t dKt = low(OFF_KQ, 16384);   // M-major (k dimensions)
    const uint32_t dSh = low(OFF_SHI, 16384), dSl = low(OFF_SLO, 16384);
    const uint32_t dTh = low(OFF_THI, 16), dTl = low(OFF_TLO, 16);
    const uint32_t dRh = low(OFF_RHI, 8192), dRl = low(OFF_RLO, 8192);
    constexpr uint32_t stage = 32768 >> 4;
    auto kofs = [](int kk) { return (uint32_t)((kk >> 2) * 1024 + (kk & 3) * 2); };

    auto issue_a = [&](int c) -> bool {
        const int st = c & 1;
        if (!wait_bar(&bars->kq_full[st], (c >> 1) & 1, cx)) return false;
        if (ragged && c == nchunks - 1 && !wait_bar(&bars->kq_fixed, 0, cx)) return false;
        if (c > 0 && !wait_bar(&bars->a_free, (c - 1) & 1, cx)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma(TM_A, dKQ + st * stage + kofs(kk), dKQ + st * stage + kofs(kk), idA, kk > 0);
        mma_commit(&bars->a_full);
        return true;
    };
    bool ok = nchunks > 0 ? issue_a(0) : true;
    for (int c = 0; c < nchunks && ok; ++c) {
        const int st = c & 1;
        const uint32_t par = c & 1;
        ok = wait_bar(&bars->s_ready, par, cx) && (c == 0 || wait_bar(&bars->o_free, (c - 1) & 1, cx));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma(TM_X, dKQ + st * stage + kofs(kk), dSh + kk * 128, idX, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma(TM_X, dKQ + st * stage + kofs(kk), dSl + kk * 128, idX, 1);
        mma_commit(&bars->x_full);
        if (c + 1 < nchunks && !(ok = issue_a(c + 1))) break;
        if (!(ok = wait_bar(&bars->t_ready, par, cx) && wait_bar(&bars->r_ready, par, cx))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma(TM_Y, dTh + kk * 2, dRh + kk * 128, idX, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma(TM_Y, dTh + kk * 2, dRl + kk * 128, idX, 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma(TM_Y, dTl + kk * 2, dRh + kk * 128, idX, 1);
        mma_commit(&bars->y_full);
        if (!(ok = wait_bar(&bars->u_ready, par, cx))) break;
        tc_fence_after();
        // 16 tokens of K a step: rows 32 kk .. 32 kk + 15 of the interleaved tile
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma(TM_D, dKt + st * stage + kk * 256, dRh + kk * 128, idD, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma(TM_D, dKt + st * stage + kk * 256, dRl + kk * 128, idD, 1);
        mma_commit(&bars->d_full);
        mma_commit(&bars->kq_empty[st]);
    }
    // every issued MMA must finish before tensor memory is freed
    mma_commit(&bars->drain);
    int dummy = 0;
    cx.abort_flag = &dummy;
    cx.limit = kDrainLimitNs;
    wait_bar(&bars->drain, 0, cx);
}

template <int NV>
__device__ void producer_role(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, Bars *bars,
                              uint8_t *sm, int t0, int nchunks, int xq, int xv, Ctx cx) {
    int kq = 0, vv = 0;
    for (int c = 0; c < nchunks; ++c) {
        const int st = c & 1;
        if (c >= 2 && !wait_bar(&bars->kq_empty[st], ((c >> 1) - 1) & 1, cx)) break;
        uint8_t *dst = sm + OFF_KQ + st * 32768;
        mbar_arrive_expect_tx(&bars->kq_full[st], 32768);
        const int y = t0 + c * C;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                tma_load_2d(dst + x * 16384 + a * 4096, &tk, &bars->kq_full[st], xq + 64 * x, y + 16 * a);
                tma_load_2d(dst + x * 16384 + a * 4096 + 2048, &tq, &bars->kq_full[st], xq + 64 * x,
                            y + 16 * a);
            }
        }
        kq = c + 1;
        if (kq == nchunks) mbar_arrive(&bars->kq_last);
        if (c >= 1 && !wait_bar(&bars->r_ready, (c - 1) & 1, cx)) break;
        mbar_arrive_expect_tx(&bars->v_full, NV * C * 2);
#pragma unroll
        for (int x = 0; x < NV / 64; ++x)
            tma_load_2d(sm + OFF_V + x * 8192, &tv, &bars->v_full, xv + 64 * x, y);
        vv = c + 1;
    }
    // copies still in flight must land before the shared memory goes away
    int dummy = 0;
    cx.abort_flag = &dummy;
    cx.limit = kDrainLimitNs;
    for (int c = kq >= 2 ? kq - 2 : 0; c < kq; ++c) wait_bar(&bars->kq_full[c & 1], (c >> 1) & 1, cx);
    if (vv > 0) wait_bar(&bars->v_full, (vv - 1) & 1, cx);
}

template <int NV>
__global__ void __launch_bounds__(kThreads, 1)
    delta_extend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const DeltaParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars *bars = reinterpret_cast<Bars *>(sm + OFF_BAR);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    constexpr int kParts = kHeadDim / NV;
    const int part = (int)blockIdx.x % kParts;
    const int h = ((int)blockIdx.x / kParts) % p.H;
    const int want = (int)blockIdx.x / kParts / p.H;

    // Longest request first for batches that the CTA can rank itself: CTAs are issued in index
    // order, so long requests do not finish last.
    int b = want;
    if (p.B > 1 && p.B <= kThreads) {
        int *lens = reinterpret_cast<int *>(sm);
        const int t = threadIdx.x;
        const int mine = t < p.B ? p.cu_seqlens[t + 1] - p.cu_seqlens[t] : 0;
        lens[t] = mine;
        __syncthreads();
        if (t < p.B) {
            int rank = 0;
            for (int u = 0; u < p.B; ++u) {
                const int lu = lens[u];
                rank += (lu > mine) || (lu == mine && u < t);
            }
            if (rank == want) bars->request = t;
        }
        __syncthreads();
        b = bars->request;
    }

    const int slot = p.state_idx[b];
    const int t_req0 = p.cu_seqlens[b], t_req1 = p.cu_seqlens[b + 1];
    if (slot < 0 || slot >= p.num_slots) {
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SLOT_RANGE);
        return;
    }
    if (t_req0 < 0 || t_req1 < t_req0 || t_req1 > p.T || t_req1 - t_req0 > p.max_seqlen) {
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SEQLENS);
        return;
    }
    const int n = t_req1 - t_req0;
    const int nchunks = (n + C - 1) / C;
    const bool ragged = n % C != 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->kq_full[s], 1);
            mbar_init(&bars->kq_empty[s], 1);
            mbar_init(&bars->coef[s], kTWarps);
        }
        mbar_init(&bars->v_full, 1);
        mbar_init(&bars->kq_last, 1);
        mbar_init(&bars->kq_fixed, 1);
        mbar_init(&bars->a_full, 1);
        mbar_init(&bars->a_free, kTWarps);
        for (int s = 0; s < 3; ++s) mbar_init(&bars->t_sync[s], kTWarps);
        mbar_init(&bars->t_ready, kTWarps);
        mbar_init(&bars->x_full, 1);
        mbar_init(&bars->y_full, 1);
        mbar_init(&bars->d_full, 1);
        mbar_init(&bars->r_ready, kEWarps);
        mbar_init(&bars->u_ready, kEWarps);
        mbar_init(&bars->s_ready, kEWarps);
        mbar_init(&bars->o_free, kEWarps);
        mbar_init(&bars->drain, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    if (warp == kProducerWarp && lane == 0 && nchunks > 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    // the blocks of [T'; P T] above the diagonal stay zero
    for (int x = threadIdx.x; x < 32768 / 16; x += kThreads)
        reinterpret_cast<uint4 *>(sm + OFF_THI)[x] = make_uint4(0u, 0u, 0u, 0u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = bars->tmem_base;
    const Ctx cx{p.wait_limit_ns, &bars->abort_flag, p.err};
    const int c0 = part * NV;

    if (warp < kTWarps) {
        reg_dec<kRegsT>();
        t_role(p, sm, bars, cx, tbase, warp, lane, (size_t)t_req0, n, h, nchunks);
    } else if (warp < kTWarps + kEWarps) {
        reg_inc<kRegsE>();
        e_role<NV>(p, sm, bars, cx, tbase, warp & 3, (warp - kTWarps) >> 2, lane, (size_t)t_req0, n, h, c0,
                   slot, p.prefix_mask[b] != 0, nchunks);
    } else {
        reg_dec<kRegsRest>();
        if (warp == kProducerWarp) {
            if (lane == 0)
                producer_role<NV>(tq, tk, tv, bars, sm, t_req0, nchunks, (h / p.group) * kHeadDim,
                                  h * kHeadDim + c0, cx);
        } else if (warp == kMmaWarp) {
            if (lane == 0) mma_role<NV>(bars, tbase, smem_u32(sm), nchunks, ragged, cx);
        } else if (warp == kFixWarp && ragged) {
            const int c = nchunks - 1;
            if (warp_wait(&bars->kq_last, 0, cx) &&
                warp_wait(&bars->kq_full[c & 1], (c >> 1) & 1, cx)) {
                uint8_t *tile = sm + OFF_KQ + (c & 1) * 32768;
                // (token, K or Q, column block, 16-byte piece)
                for (int x = (n - c * C) * 32 + lane; x < C * 32; x += 32) {
                    const int i = x >> 5;
                    const int rho = 32 * (i >> 4) + (i & 15) + ((x >> 4) & 1) * 16;
                    *reinterpret_cast<uint4 *>(tile + ((x >> 3) & 1) * 16384 + rho * 128 + (x & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                warp_arrive(&bars->kq_fixed, lane);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, kTmemCols);
    }
}

template <int NV>
cudaError_t launch_nv(const DeltaParams &p, cudaStream_t stream) {
    const long long ctas = (long long)p.B * p.H * (kHeadDim / NV);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    CUtensorMap tq, tk, tv;
    memset(&tq, 0, sizeof(tq));
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    if (p.T > 0 &&
        (!make_rows_map(&tq, p.q, p.T, (long long)p.Hk * kHeadDim, p.q_rs, 16) ||
         !make_rows_map(&tk, p.k, p.T, (long long)p.Hk * kHeadDim, p.k_rs, 16) ||
         !make_rows_map(&tv, p.v, p.T, (long long)p.H * kHeadDim, p.v_rs, C)))
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
            e = cudaFuncSetAttribute(delta_extend_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSmemBytes);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    return launch_pdl(delta_extend_kernel<NV>, dim3((unsigned)ctas), dim3(kThreads), kSmemBytes, stream, tq,
                      tk, tv, p);
}

}  // namespace

cudaError_t launch_delta_extend(const DeltaParams &p, int num_sms, cudaStream_t stream) {
    if (p.B <= 0) return cudaSuccess;
    // two CTAs per head while that still is one wave
    if ((long long)p.B * p.H * 2 <= num_sms) return launch_nv<64>(p, stream);
    return launch_nv<128>(p, stream);
}

}  // namespace la
