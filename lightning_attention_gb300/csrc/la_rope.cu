// la_rope.cu -- rotary positions, alone or with the rotated keys and the values stored into the pages
// of a key/value cache.
//
// A pair (x, y) of a head at position p becomes m (x cos a - y sin a, x sin a + y cos a), a = p f.  The
// angle in turns is p (f / 2 pi) modulo 1, so f / 2 pi is taken as a 64-bit binary fraction and
// multiplied by p in integers: the overflow drops whole turns, and what is left is off by
// p 2^-53 f / 2 pi turns (the rounding of f to 64 bits), some 1e-10 at a million positions, where a
// product in 32 bits would be off by whole radians.  sincospif takes the upper 32 bits of it.
//
// The kernel is a copy bound by HBM.  A CTA has a run of head rows, of a part of a token's heads or of several tokens,
// 8 threads a row, each with two 16-byte pieces that hold both halves of its pairs (columns c and c + rot / 2 in the half
// layout, neighbours in the interleaved one), four rows of a thread in flight; its tokens' angles are formed once, under
// the loads.  Measured: 16,384 tokens x 64 heads 79 us (the copy bandwidth), x 40 heads into pages 57 us (0.87), 32,768
// tokens x 9 heads 32 us (0.70; a CTA per token, 64 us).  128 threads and four rows each: with 256 threads 91, 66
// and 36 us, with two rows 87, 68 and 33; without the streaming hints on loads and stores 83, 64 and 33.
#include "la_attn.h"

#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = kThreads / 8;  // head rows of a pass

struct Pieces {
    uint4 a, b;
};

__device__ __forceinline__ void unpack8(const uint4 x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(sm100::pack_bf16x2(f[0], f[1]), sm100::pack_bf16x2(f[2], f[3]),
                      sm100::pack_bf16x2(f[4], f[5]), sm100::pack_bf16x2(f[6], f[7]));
}

// kUnroll: rows of a thread.  rows: heads of a token, at least 2.
template <int kUnroll>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int rows) {
    constexpr int kTokens = kRows * kUnroll / 2 + 1;  // that a CTA's rows may belong to
    __shared__ alignas(16) float cs[kTokens][64], sn[kTokens][64];
    __shared__ unsigned long long turn[64];  // turns per position, a binary fraction
    __shared__ long long place[kTokens];     // where a token's keys and values go, -1: nowhere
    pdl_wait();
    pdl_trigger();
    const int c = threadIdx.x & 7;  // piece of the row; pairs 8 c .. 8 c + 7 where it is rotated
    const bool turned = 16 * c < p.rot, store = p.loc != nullptr;
    const int col_a = p.interleaved || !turned ? 16 * c : 8 * c;
    const int col_b = p.interleaved || !turned ? 16 * c + 8 : 8 * c + p.rot / 2;
    const long long first = (long long)blockIdx.x * (kRows * kUnroll), all = (long long)p.T * rows;
    const int t0 = (int)(first / rows), skip = (int)(first - (long long)t0 * rows);
    const int mine = (int)min((long long)(kRows * kUnroll), all - first), tokens = (skip + mine - 1) / rows + 1;

    Pieces x[kUnroll];
    int tok[kUnroll], row[kUnroll];  // token from t0 on; -1: no row
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int at = skip + (threadIdx.x >> 3) + u * kRows;
        tok[u] = at < skip + mine ? at / rows : -1;
        if (tok[u] < 0) continue;
        const int r = row[u] = at - tok[u] * rows;
        const long long t = t0 + tok[u];
        const __nv_bfloat16 *src;
        if (r < p.H)
            src = p.q + t * p.q_rs + (long long)r * kHeadDim;
        else if (r < p.H + p.Hkv)
            src = p.k + t * p.k_rs + (long long)(r - p.H) * kHeadDim;
        else
            src = p.v + t * p.v_rs + (long long)(r - p.H - p.Hkv) * kHeadDim;
        x[u].a = __ldcs(reinterpret_cast<const uint4 *>(src + col_a));
        x[u].b = __ldcs(reinterpret_cast<const uint4 *>(src + col_b));
    }
    const int half = p.rot / 2;
    if (threadIdx.x < half) {
        double f = p.inv_freq[threadIdx.x] * 0.15915494309189533577;  // turns per position
        f -= floor(f);
        turn[threadIdx.x] = __double2ull_rz(f * 18446744073709551616.0);
    }
    if (store) {
        for (int i = threadIdx.x; i < tokens; i += kThreads) {
            const int loc = p.loc[t0 + i];
            long long at = -1;  // row loc % page_size of page loc / page_size
            if (loc >= 0 && loc < (long long)p.cache.num_pages * p.cache.page_size) {
                const int page = loc / p.cache.page_size;
                at = (long long)page * p.cache.page_stride + (long long)(loc - page * p.cache.page_size) * kHeadDim;
            } else if (loc != -1) {
                atomicOr(p.err, ERR_BIT_PAGE);
            }
            place[i] = at;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const unsigned long long angle = (unsigned long long)(long long)p.positions[t0 + t] * turn[f];
        float s, co;
        sincospif((float)(int)(angle >> 32) * 4.656612873077392578125e-10f, &s, &co);  // 2^-31: half turns
        cs[t][f] = co * p.mscale;
        sn[t][f] = s * p.mscale;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (tok[u] < 0) continue;
        const int r = row[u];
        const long long t = t0 + tok[u];
        const bool is_v = r >= p.H + p.Hkv;
        __nv_bfloat16 *dst;
        if (r < p.H) {
            dst = p.q_out + t * p.qo_rs + (long long)r * kHeadDim;
        } else if (!store) {
            dst = p.k_out + t * p.ko_rs + (long long)(r - p.H) * kHeadDim;
        } else {
            if (place[tok[u]] < 0) continue;
            const long long head = (long long)(r - p.H - (is_v ? p.Hkv : 0)) * p.cache.page_size * kHeadDim;
            dst = (is_v ? p.cache.v : p.cache.k) + place[tok[u]] + head;
        }
        if (turned && !is_v) {
            float a[8], b[8], y[8], z[8];
            unpack8(x[u].a, a);
            unpack8(x[u].b, b);
            const float4 c0 = reinterpret_cast<const float4 *>(cs[tok[u]])[2 * c];
            const float4 c1 = reinterpret_cast<const float4 *>(cs[tok[u]])[2 * c + 1];
            const float4 s0 = reinterpret_cast<const float4 *>(sn[tok[u]])[2 * c];
            const float4 s1 = reinterpret_cast<const float4 *>(sn[tok[u]])[2 * c + 1];
            const float co[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float si[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[2 * i] = a[2 * i] * co[i] - a[2 * i + 1] * si[i];
                    y[2 * i + 1] = a[2 * i] * si[i] + a[2 * i + 1] * co[i];
                    z[2 * i] = b[2 * i] * co[4 + i] - b[2 * i + 1] * si[4 + i];
                    z[2 * i + 1] = b[2 * i] * si[4 + i] + b[2 * i + 1] * co[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = a[i] * co[i] - b[i] * si[i];
                    z[i] = a[i] * si[i] + b[i] * co[i];
                }
            }
            x[u].a = pack8(y);
            x[u].b = pack8(z);
        }
        __stcs(reinterpret_cast<uint4 *>(dst + col_a), x[u].a);
        __stcs(reinterpret_cast<uint4 *>(dst + col_b), x[u].b);
    }
}

}  // namespace

// Few rows go to as many CTAs as there are, one row a thread.
cudaError_t launch_rope(const RopeParams &p, cudaStream_t stream) {
    const int rows = p.H + p.Hkv * (p.loc ? 2 : 1);
    const long long all = (long long)p.T * rows;
    if (all <= 4ll * kAttnCtas * kRows)
        return launch_pdl(rope_kernel<1>, dim3((unsigned)((all + kRows - 1) / kRows)), dim3(kThreads), 0, stream, p, rows);
    return launch_pdl(rope_kernel<4>, dim3((unsigned)((all + 4 * kRows - 1) / (4 * kRows))), dim3(kThreads), 0, stream, p,
                      rows);
}

}  // namespace la
