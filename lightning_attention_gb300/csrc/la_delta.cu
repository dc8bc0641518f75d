// la_delta.cu -- token-serial gated delta rule: one-token decode, chain verify.
//
// Per request and value head h, with key head h / (H / Hk), from the state S (rows: k, columns: v):
//   S <- e^{g} S;  u = beta (v - S^T k);  S <- S + k u^T;  o = D^-0.5 S^T q.
// Both readouts are taken from the state before the token, so that one reduction over the rows
// serves them:  x = e^g S^T k,  u = beta (v - x),  S^T q after the update = e^g S^T q + (k.q) u.
// (The update then needs u in every thread, the output only in the threads that store it.)
//
// Columns of S never meet, so a CTA takes COLS of the 128 value columns of one (request, head):
// all of them when there are enough (request, head) pairs to fill the GPU, a quarter otherwise.
// HBM-bound: a state is read once and written once (verify: written once per draft token).
// Every access is a 16-byte vector of a row, all of a thread's loads are issued before any
// arithmetic (64 KiB in flight per CTA, 16 KiB at a quarter), one barrier per token.
#include "la_delta.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// head_dim^-0.5 for head_dim = 128, i.e. 2^-3.5
constexpr float kScale = 0.08838834764831845f;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <int MODE, int COLS>
__global__ void __launch_bounds__(kThreads) delta_recurrent_kernel(const DeltaParams p) {
    constexpr int kParts = kHeadDim / COLS;
    constexpr int kLanesPerRow = COLS / 4;              // a lane owns 4 columns
    constexpr int kRowGroups = kWarps * (32 / kLanesPerRow);
    constexpr int kRows = kHeadDim / kRowGroups;        // rows of a thread
    pdl_wait();
    pdl_trigger();
    const int H = p.H;
    const int part = kParts == 1 ? 0 : (int)(blockIdx.x % kParts);
    const int pair = (int)(blockIdx.x / kParts);
    const int b = pair / H;
    const int h = pair - b * H;
    const int hk = h / p.group;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int row_group = threadIdx.x / kLanesPerRow;   // rows row_group + kRowGroups r
    const int c4 = (lane % kLanesPerRow) * 4;           // column of the CTA's COLS
    const int col = part * COLS + c4;                   // value column

    __shared__ __align__(16) float red_x[2][kWarps][COLS];
    __shared__ __align__(16) float red_o[2][kWarps][COLS];
    __shared__ __align__(16) float sk[2][kHeadDim], sq[2][kHeadDim];

    const int slot = p.state_idx[b];
    if (slot < 0 || slot >= p.num_slots) {
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SLOT_RANGE);
        return;
    }
    constexpr size_t kMat = (size_t)kHeadDim * kHeadDim;
    float *state = p.pool + ((size_t)slot * H + h) * kMat + col;

    size_t t_begin;
    int n;
    bool zero = false;
    if constexpr (MODE == DELTA_EXTEND) {
        const int t0 = p.cu_seqlens[b], t1 = p.cu_seqlens[b + 1];
        if (t0 < 0 || t1 < t0 || t1 > p.T || t1 - t0 > p.max_seqlen) {
            if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SEQLENS);
            return;
        }
        t_begin = (size_t)t0;
        n = t1 - t0;
        zero = p.prefix_mask[b] == 0;
    } else {
        t_begin = (size_t)b * p.N;
        n = p.N;
    }

    float4 s[kRows];
    if (zero) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            s[r] = __ldcs(reinterpret_cast<const float4 *>(
                state + (size_t)(row_group + r * kRowGroups) * kHeadDim));
    }

    for (int t = 0; t < n; ++t) {
        const size_t tok = t_begin + t;
        // Every warp forms the token's three inner products from its own copy of the rows.
        const uint2 kw = *reinterpret_cast<const uint2 *>(p.k + tok * p.k_rs + hk * kHeadDim + lane * 4);
        const uint2 qw = *reinterpret_cast<const uint2 *>(p.q + tok * p.q_rs + hk * kHeadDim + lane * 4);
        const uint2 vv = *reinterpret_cast<const uint2 *>(p.v + tok * p.v_rs + h * kHeadDim + col);
        const float decay = expf(p.g[tok * H + h]);
        const float beta = p.beta[tok * H + h];
        const float k0 = bf_lo(kw.x), k1 = bf_hi(kw.x), k2 = bf_lo(kw.y), k3 = bf_hi(kw.y);
        const float q0 = bf_lo(qw.x), q1 = bf_hi(qw.x), q2 = bf_lo(qw.y), q3 = bf_hi(qw.y);
        const int buf = t & 1;
        if (warp == 0) {
            *reinterpret_cast<float4 *>(&sk[buf][lane * 4]) = make_float4(k0, k1, k2, k3);
            *reinterpret_cast<float4 *>(&sq[buf][lane * 4]) = make_float4(q0, q1, q2, q3);
        }
        float kq = warp_sum(fmaf(k0, q0, fmaf(k1, q1, fmaf(k2, q2, k3 * q3))));
        float rk = 1.f, rq = 1.f;
        if (p.l2norm) {
            rk = 1.f / sqrtf(warp_sum(fmaf(k0, k0, fmaf(k1, k1, fmaf(k2, k2, k3 * k3)))) + kDeltaEps);
            rq = 1.f / sqrtf(warp_sum(fmaf(q0, q0, fmaf(q1, q1, fmaf(q2, q2, q3 * q3)))) + kDeltaEps);
            kq *= rk * rq;
        }
        __syncthreads();  // k and q staged; the partials of token t - 1 are read

        float kf[kRows];
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), o = x;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            kf[r] = sk[buf][row_group + r * kRowGroups];
            const float qf = sq[buf][row_group + r * kRowGroups];
            x.x = fmaf(kf[r], s[r].x, x.x);
            x.y = fmaf(kf[r], s[r].y, x.y);
            x.z = fmaf(kf[r], s[r].z, x.z);
            x.w = fmaf(kf[r], s[r].w, x.w);
            o.x = fmaf(qf, s[r].x, o.x);
            o.y = fmaf(qf, s[r].y, o.y);
            o.z = fmaf(qf, s[r].z, o.z);
            o.w = fmaf(qf, s[r].w, o.w);
        }
#pragma unroll
        for (int d = kLanesPerRow; d < 32; d <<= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, d);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, d);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, d);
            x.w += __shfl_xor_sync(0xffffffffu, x.w, d);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
        }
        if (lane < kLanesPerRow) {
            *reinterpret_cast<float4 *>(&red_x[buf][warp][c4]) = x;
            *reinterpret_cast<float4 *>(&red_o[buf][warp][c4]) = o;
        }
        __syncthreads();
        float4 sx = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 f = *reinterpret_cast<const float4 *>(&red_x[buf][w][c4]);
            sx.x += f.x;
            sx.y += f.y;
            sx.z += f.z;
            sx.w += f.w;
        }
        const float xs = decay * rk;
        float4 u;
        u.x = beta * (bf_lo(vv.x) - xs * sx.x);
        u.y = beta * (bf_hi(vv.x) - xs * sx.y);
        u.z = beta * (bf_lo(vv.y) - xs * sx.z);
        u.w = beta * (bf_hi(vv.y) - xs * sx.w);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float kr = kf[r] * rk;
            s[r].x = fmaf(kr, u.x, s[r].x * decay);
            s[r].y = fmaf(kr, u.y, s[r].y * decay);
            s[r].z = fmaf(kr, u.z, s[r].z * decay);
            s[r].w = fmaf(kr, u.w, s[r].w * decay);
        }
        if constexpr (MODE == DELTA_VERIFY) {
            float *dst = p.inter + (((size_t)b * p.N + t) * H + h) * kMat + col;
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                __stcs(reinterpret_cast<float4 *>(
                           dst + (size_t)(row_group + r * kRowGroups) * kHeadDim),
                       s[r]);
        }
        if (threadIdx.x < kLanesPerRow) {
            float4 so = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 f = *reinterpret_cast<const float4 *>(&red_o[buf][w][c4]);
                so.x += f.x;
                so.y += f.y;
                so.z += f.z;
                so.w += f.w;
            }
            const float os = decay * rq;
            const __nv_bfloat162 a =
                __floats2bfloat162_rn(fmaf(kq, u.x, os * so.x) * kScale, fmaf(kq, u.y, os * so.y) * kScale);
            const __nv_bfloat162 c =
                __floats2bfloat162_rn(fmaf(kq, u.z, os * so.z) * kScale, fmaf(kq, u.w, os * so.w) * kScale);
            uint2 w2;
            w2.x = *reinterpret_cast<const uint32_t *>(&a);
            w2.y = *reinterpret_cast<const uint32_t *>(&c);
            *reinterpret_cast<uint2 *>(p.out + (tok * H + h) * kHeadDim + col) = w2;
        }
    }

    if constexpr (MODE != DELTA_VERIFY) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            __stcs(reinterpret_cast<float4 *>(state + (size_t)(row_group + r * kRowGroups) * kHeadDim),
                   s[r]);
    }
}

template <int MODE>
cudaError_t launch_mode(const DeltaParams &p, int num_sms, cudaStream_t stream) {
    const long long pairs = (long long)p.B * p.H;
    if (pairs <= 0) return cudaSuccess;
    if (pairs * 4 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // a quarter of the columns per CTA while that leaves at most two CTAs per SM
    if (pairs * 4 <= 2ll * num_sms)
        return launch_pdl(delta_recurrent_kernel<MODE, 32>, dim3((unsigned)(pairs * 4)),
                          dim3(kThreads), 0, stream, p);
    return launch_pdl(delta_recurrent_kernel<MODE, 128>, dim3((unsigned)pairs), dim3(kThreads), 0,
                      stream, p);
}

}  // namespace

cudaError_t launch_delta_recurrent(DeltaMode mode, const DeltaParams &p, int num_sms,
                                   cudaStream_t stream) {
    switch (mode) {
        case DELTA_DECODE: return launch_mode<DELTA_DECODE>(p, num_sms, stream);
        case DELTA_VERIFY: return launch_mode<DELTA_VERIFY>(p, num_sms, stream);
        case DELTA_EXTEND: return launch_mode<DELTA_EXTEND>(p, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace la
