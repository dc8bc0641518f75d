// la_rope.cu -- rotary positions, alone or with the rotated keys and the values stored into the pages
// of a key/value cache.
//
// A pair (x, y) of a head at position p becomes m (x cos a - y sin a, x sin a + y cos a), a = p f.  The
// angle in turns is p (f / 2 pi) modulo 1, so f / 2 pi is taken as a 64-bit binary fraction and
// multiplied by p in integers: the overflow drops whole turns, and what is left is off by
// p 2^-53 f / 2 pi turns (the rounding of f to 64 bits), some 1e-10 at a million positions, where a
// product in 32 bits would be off by whole radians.  sincospif takes the upper 32 bits of it.
//
// The kernel is a copy bound by HBM: a CTA per token, 8 threads per head row, each with two 16-byte
// pieces that hold both halves of its pairs (columns c and c + rot / 2 in the half layout, neighbours
// in the interleaved one), four rows of a thread in flight.  64 threads form the token's angles once
// for all heads.
#include "la_attn.h"

#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = kThreads / 8;  // head rows of a pass
constexpr int kUnroll = 4;           // passes in flight

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

__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    __shared__ alignas(16) float cs[64], sn[64];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const int c = threadIdx.x & 7;  // piece of the row; pairs 8 c .. 8 c + 7 where it is rotated
    const int r0 = threadIdx.x >> 3;
    const bool turned = 16 * c < p.rot;
    const int col_a = p.interleaved || !turned ? 16 * c : 8 * c;
    const int col_b = p.interleaved || !turned ? 16 * c + 8 : 8 * c + p.rot / 2;
    const bool store = p.loc != nullptr;
    const int rows = p.H + p.Hkv * (store ? 2 : 1);

    // where the token's keys and values go: row `at` of page `page`, or nowhere
    long long base = -1;
    if (store) {
        const int loc = p.loc[t];
        if (loc >= 0 && loc < (long long)p.cache.num_pages * p.cache.page_size) {
            const int page = loc / p.cache.page_size;
            base = (long long)page * p.cache.page_stride +
                   (long long)(loc - page * p.cache.page_size) * kHeadDim;
        } else if (loc != -1 && threadIdx.x == 0) {
            atomicOr(p.err, ERR_BIT_PAGE);
        }
    }
    if (threadIdx.x < p.rot / 2) {
        double f = p.inv_freq[threadIdx.x] * 0.15915494309189533577;  // turns per position
        f -= floor(f);
        const unsigned long long turn =
            (unsigned long long)(long long)p.positions[t] * __double2ull_rz(f * 18446744073709551616.0);
        float s, co;
        sincospif((float)(int)(turn >> 32) * 4.656612873077392578125e-10f, &s, &co);  // 2^-31: half turns
        cs[threadIdx.x] = co * p.mscale;
        sn[threadIdx.x] = s * p.mscale;
    }

    for (int row0 = 0; row0 < rows; row0 += kRows * kUnroll) {
        const int first = row0 + r0;
        Pieces x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = first + u * kRows;
            if (r >= rows) break;
            const __nv_bfloat16 *src;
            if (r < p.H)
                src = p.q + t * p.q_rs + (long long)r * kHeadDim;
            else if (r < p.H + p.Hkv)
                src = p.k + t * p.k_rs + (long long)(r - p.H) * kHeadDim;
            else
                src = p.v + t * p.v_rs + (long long)(r - p.H - p.Hkv) * kHeadDim;
            x[u].a = *reinterpret_cast<const uint4 *>(src + col_a);
            x[u].b = *reinterpret_cast<const uint4 *>(src + col_b);
        }
        if (row0 == 0) __syncthreads();  // the angles
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = first + u * kRows;
            if (r >= rows) break;
            const bool is_v = r >= p.H + p.Hkv;
            __nv_bfloat16 *dst;
            if (r < p.H) {
                dst = p.q_out + t * p.qo_rs + (long long)r * kHeadDim;
            } else if (!store) {
                dst = p.k_out + t * p.ko_rs + (long long)(r - p.H) * kHeadDim;
            } else {
                if (base < 0) continue;
                const long long head = (long long)(r - p.H - (is_v ? p.Hkv : 0)) * p.cache.page_size * kHeadDim;
                dst = (is_v ? p.cache.v : p.cache.k) + base + head;
            }
            if (turned && !is_v) {
                float a[8], b[8], y[8], z[8];
                unpack8(x[u].a, a);
                unpack8(x[u].b, b);
                const float4 c0 = reinterpret_cast<const float4 *>(cs)[2 * c];
                const float4 c1 = reinterpret_cast<const float4 *>(cs)[2 * c + 1];
                const float4 s0 = reinterpret_cast<const float4 *>(sn)[2 * c];
                const float4 s1 = reinterpret_cast<const float4 *>(sn)[2 * c + 1];
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
            *reinterpret_cast<uint4 *>(dst + col_a) = x[u].a;
            *reinterpret_cast<uint4 *>(dst + col_b) = x[u].b;
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t stream) {
    return launch_pdl(rope_kernel, dim3((unsigned)p.T), dim3(kThreads), 0, stream, p);
}

}  // namespace la
