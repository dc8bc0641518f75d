// la_delta.cu -- token-serial gated delta rule: one-token decode, chain verify, extend of a few tokens.
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
// arithmetic (64 KiB in flight per CTA, 16 KiB at a quarter).  A thread's rows are contiguous, so its
// k and q entries are one or two broadcast vector loads, and the sums that the whole rows need (|k|^2,
// |q|^2, k.q) are formed over the same rows and meet in the same reduction: one barrier per token.  The
// next token's entries are loaded before the barrier.
//
// Measured: decode of 256 requests x 16 heads 82.4 us, 0.97 of the copy bandwidth; chain verify of
// 128 x 5 tokens x 64 heads 493 us, 0.97 likewise.  Both need the two CTAs per SM that 128 registers a
// thread allow.  A single request is bound by latency (2.2 us of kernel at 8 heads).
#include "la_delta.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// head_dim^-0.5 for head_dim = 128, i.e. 2^-3.5
constexpr float kScale = 0.08838834764831845f;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// n consecutive bf16 values (4 or 16) of a row.
template <int n>
struct RowVec {
    uint32_t w[n / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if constexpr (n == 4) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x;
            w[1] = u.y;
        } else {
#pragma unroll
            for (int x = 0; x < n / 8; ++x) {
                const uint4 u = reinterpret_cast<const uint4 *>(p)[x];
                w[4 * x] = u.x;
                w[4 * x + 1] = u.y;
                w[4 * x + 2] = u.z;
                w[4 * x + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        return i & 1 ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
    }
};

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 shfl4(const float4 &a, int d) {
    return make_float4(__shfl_xor_sync(0xffffffffu, a.x, d), __shfl_xor_sync(0xffffffffu, a.y, d),
                       __shfl_xor_sync(0xffffffffu, a.z, d), __shfl_xor_sync(0xffffffffu, a.w, d));
}

template <int MODE, int COLS>
__global__ void __launch_bounds__(kThreads, 2) delta_recurrent_kernel(const DeltaParams p) {
    constexpr int kParts = kHeadDim / COLS;
    constexpr int kLanesPerRow = COLS / 4;                             // a lane owns 4 columns
    constexpr int kRows = kHeadDim / (kThreads / kLanesPerRow);        // rows of a thread
    static_assert(kRows == 16 || kRows == 4, "a thread's rows are whole vectors");
    pdl_wait();
    pdl_trigger();
    const int H = p.H;
    const int part = kParts == 1 ? 0 : (int)(blockIdx.x % kParts);
    const int pair = (int)(blockIdx.x / kParts);
    const int b = pair / H;
    const int h = pair - b * H;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int row0 = (int)(threadIdx.x / kLanesPerRow) * kRows;
    const int c4 = (lane % kLanesPerRow) * 4;           // column of the CTA's COLS
    const int col = part * COLS + c4;                   // value column

    __shared__ __align__(16) float red_x[2][kWarps][COLS];
    __shared__ __align__(16) float red_o[2][kWarps][COLS];
    __shared__ __align__(16) float4 red_s[2][kWarps];   // sums of k k, q q, k q

    const int slot = p.state_idx[b];
    if (slot < 0 || slot >= p.num_slots) {
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SLOT_RANGE);
        return;
    }
    constexpr size_t kMat = (size_t)kHeadDim * kHeadDim;
    float *state = p.pool + ((size_t)slot * H + h) * kMat + (size_t)row0 * kHeadDim + col;
    int n = MODE == DELTA_DECODE ? 1 : p.N;
    size_t t_begin = (size_t)b * n;
    bool prefix = true;
    if (MODE == DELTA_SERIAL) {
        const int t0 = p.cu_seqlens[b], t1 = p.cu_seqlens[b + 1];
        if (t0 < 0 || t1 < t0 || t1 > p.T || t1 - t0 > p.max_seqlen) {
            if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SEQLENS);
            return;
        }
        n = t1 - t0;
        t_begin = (size_t)t0;
        prefix = p.prefix_mask[b] != 0;
        if (n == 0 && prefix) return;
    }
    float4 s[kRows];
    if (prefix) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            s[r] = __ldcs(reinterpret_cast<const float4 *>(state + (size_t)r * kHeadDim));
    } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (MODE == DELTA_SERIAL && n == 0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) __stcs(reinterpret_cast<float4 *>(state + (size_t)r * kHeadDim), s[r]);
        return;
    }
    const __nv_bfloat16 *kp = p.k + t_begin * p.k_rs + (size_t)(h / p.group) * kHeadDim + row0;
    const __nv_bfloat16 *qp = p.q + t_begin * p.q_rs + (size_t)(h / p.group) * kHeadDim + row0;
    const __nv_bfloat16 *vp = p.v + t_begin * p.v_rs + (size_t)h * kHeadDim + col;
    const float *gp = p.g + t_begin * H + h, *bp = p.beta + t_begin * H + h;
    RowVec<kRows> kf, qf;
    RowVec<4> vf;
    kf.load(kp);
    qf.load(qp);
    vf.load(vp);
    float g = *gp, beta = *bp;

    for (int t = 0; t < n; ++t) {
        const int buf = t & 1;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), o = x, sum = x;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float k = kf[r], q = qf[r];
            x.x = fmaf(k, s[r].x, x.x);
            x.y = fmaf(k, s[r].y, x.y);
            x.z = fmaf(k, s[r].z, x.z);
            x.w = fmaf(k, s[r].w, x.w);
            o.x = fmaf(q, s[r].x, o.x);
            o.y = fmaf(q, s[r].y, o.y);
            o.z = fmaf(q, s[r].z, o.z);
            o.w = fmaf(q, s[r].w, o.w);
            sum.x = fmaf(k, k, sum.x);
            sum.y = fmaf(q, q, sum.y);
            sum.z = fmaf(k, q, sum.z);
        }
#pragma unroll
        for (int d = kLanesPerRow; d < 32; d <<= 1) {
            x = add4(x, shfl4(x, d));
            o = add4(o, shfl4(o, d));
            sum = add4(sum, shfl4(sum, d));
        }
        if (lane < kLanesPerRow) {
            *reinterpret_cast<float4 *>(&red_x[buf][warp][c4]) = x;
            *reinterpret_cast<float4 *>(&red_o[buf][warp][c4]) = o;
        }
        if (lane == 0) red_s[buf][warp] = sum;
        RowVec<kRows> kn, qn;
        RowVec<4> vn;
        float gn = 0.f, bn = 0.f;
        if (MODE != DELTA_DECODE && t + 1 < n) {
            const size_t next = (size_t)(t + 1);
            kn.load(kp + next * p.k_rs);
            qn.load(qp + next * p.q_rs);
            vn.load(vp + next * p.v_rs);
            gn = gp[next * H];
            bn = bp[next * H];
        }
        __syncthreads();  // one per token: buffer t & 1 is rewritten after the barrier of token t + 1
        float4 sx = make_float4(0.f, 0.f, 0.f, 0.f), ss = sx;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            sx = add4(sx, *reinterpret_cast<const float4 *>(&red_x[buf][w][c4]));
            ss = add4(ss, red_s[buf][w]);
        }
        const float decay = expf(g);
        const float rk = p.l2norm ? 1.f / sqrtf(ss.x + kDeltaEps) : 1.f;
        const float rq = p.l2norm ? 1.f / sqrtf(ss.y + kDeltaEps) : 1.f;
        const float xs = decay * rk;
        float4 u;
        u.x = beta * (vf[0] - xs * sx.x);
        u.y = beta * (vf[1] - xs * sx.y);
        u.z = beta * (vf[2] - xs * sx.z);
        u.w = beta * (vf[3] - xs * sx.w);
        float *dst = MODE == DELTA_VERIFY
                         ? p.inter + (((size_t)b * n + t) * H + h) * kMat + (size_t)row0 * kHeadDim + col
                         : state;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float kr = kf[r] * rk;
            s[r].x = fmaf(kr, u.x, s[r].x * decay);
            s[r].y = fmaf(kr, u.y, s[r].y * decay);
            s[r].z = fmaf(kr, u.z, s[r].z * decay);
            s[r].w = fmaf(kr, u.w, s[r].w * decay);
            if (MODE != DELTA_SERIAL || t + 1 == n)
                __stcs(reinterpret_cast<float4 *>(dst + (size_t)r * kHeadDim), s[r]);
        }
        if (threadIdx.x < kLanesPerRow) {
            float4 so = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                so = add4(so, *reinterpret_cast<const float4 *>(&red_o[buf][w][c4]));
            const float os = decay * rq, kq = ss.z * rk * rq;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(fmaf(kq, u.x, os * so.x) * kScale,
                                                            fmaf(kq, u.y, os * so.y) * kScale);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(fmaf(kq, u.z, os * so.z) * kScale,
                                                            fmaf(kq, u.w, os * so.w) * kScale);
            uint2 w2;
            w2.x = *reinterpret_cast<const uint32_t *>(&lo);
            w2.y = *reinterpret_cast<const uint32_t *>(&hi);
            *reinterpret_cast<uint2 *>(p.out + ((t_begin + t) * H + h) * kHeadDim + col) = w2;
        }
        if (MODE != DELTA_DECODE) {
            kf = kn;
            qf = qn;
            vf = vn;
            g = gn;
            beta = bn;
        }
    }
}

template <int MODE>
cudaError_t launch_mode(const DeltaParams &p, int num_sms, cudaStream_t stream) {
    const long long pairs = (long long)p.B * p.H;
    // A quarter of the columns per CTA while all of those CTAs are on the SMs at once (two each).  Quarters /
    // whole rows, us: decode of 8 pairs 2.2 / 3.5, 64: 4.1 / 4.6, 76: 4.2 / 4.7, 96: 6.1 / 5.1, 304:
    // 13.2 / 8.7; verify of 5 tokens 6.3 / 11.1, 9.1 / 12.1, 9.3 / 12.2, 14.5 / 12.6, 32.9 / 22.1.
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
        case DELTA_SERIAL: return launch_mode<DELTA_SERIAL>(p, num_sms, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace la
