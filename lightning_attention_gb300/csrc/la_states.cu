// la_states.cu -- the packed state store: pool slots (fp32) to 8-bit entries and back.
//
// A state row of 128 values is four blocks of 32 along v.  A block is kept as int8 codes in
// [-127, 127] and one scale 2^(s - 127), s an unsigned byte: the smallest power of two, at least
// 2^-127, for which the block's largest code stays at 127 or less.  Scaling by a power of two is
// exact, so a code is the value divided by the scale, rounded once to the nearest integer (ties to
// even): a restored value is off by at most half a scale, at most 1/127 of the block's largest
// magnitude where s > 0; where s = 0 that half is 2^-128, whatever the magnitudes.  (Only magnitudes above
// 127.5 * 2^121 are held at 127 of the largest scale instead.)
// s = 255 marks a block that held an infinity or a NaN; it is restored as NaN.
//
// Both directions are copies bound by HBM (64 KiB of fp32 against 16.5 KiB packed): one CTA of 256
// threads per (request, head), a warp per row of 128 values with 16-byte fp32 accesses, all of a
// thread's loads in flight before the first is used.  Measured: 128 slots x 32 heads there and back
// 101.7 us (0.97 of the copy bandwidth), 96 entries x 32 heads restored 40.1 us (0.93).
#include "la_delta.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = kHeadDim / kWarps;  // 16
constexpr size_t kMat = (size_t)kHeadDim * kHeadDim;

__device__ __forceinline__ bool pair_ok(const PackParams &p, int slot, int entry) {
    if (slot >= 0 && slot < p.num_slots && entry >= 0 && entry < p.entries) return true;
    if (threadIdx.x == 0) atomicOr(p.err, ERR_BIT_SLOT_RANGE);
    return false;
}

// The largest scale, 2^121: at the next one code 64 would stand for 2^128, beyond fp32.  Magnitudes
// above 127.5 * 2^121 keep it and are held at code 127.
constexpr int kMaxScale = 248;

__device__ __forceinline__ uint32_t code(float scaled) {
    return (uint32_t)max(min(__float2int_rn(scaled), 127), -127) & 255u;
}

__global__ void __launch_bounds__(kThreads) pack_states_kernel(const PackParams p) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x / p.H;
    const int h = blockIdx.x - b * p.H;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int slot = p.state_idx[b], entry = p.store_idx[b];
    if (!pair_ok(p, slot, entry)) return;
    const int row0 = warp * kRowsPerWarp;
    const float *src = p.pool + ((size_t)slot * p.H + h) * kMat + (size_t)row0 * kHeadDim + lane * 4;
    float4 x[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r)
        x[r] = __ldcs(reinterpret_cast<const float4 *>(src + (size_t)r * kHeadDim));
    const size_t at = ((size_t)entry * p.H + h) * kHeadDim + row0;  // row of the entry
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.codes + at * kHeadDim) + lane;
    uint32_t my_scales = 0;  // lane r (r < 16): the four scales of row row0 + r
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        // magnitudes compare as their bit patterns, with infinities and NaN on top
        const uint32_t m = 0x7fffffffu;
        uint32_t top = max(max(__float_as_uint(x[r].x) & m, __float_as_uint(x[r].y) & m),
                           max(__float_as_uint(x[r].z) & m, __float_as_uint(x[r].w) & m));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = (int)(top >> 23);
        int s = max(e - 6, 0);
        // 2^(127 - s) for s in [0, 248]
        if (s < kMaxScale &&
            __float2int_rn(__uint_as_float(top) * __uint_as_float((uint32_t)(254 - s) << 23)) > 127)
            ++s;
        uint32_t w = 0;
        if (e == 255) {
            s = 255;
        } else {
            const float f = __uint_as_float((uint32_t)(254 - s) << 23);
            w = code(x[r].x * f) | (code(x[r].y * f) << 8) | (code(x[r].z * f) << 16) |
                (code(x[r].w * f) << 24);
        }
        dst[r * (kHeadDim / 4)] = w;
        const uint32_t s0 = __shfl_sync(0xffffffffu, (uint32_t)s, 0);
        const uint32_t s1 = __shfl_sync(0xffffffffu, (uint32_t)s, 8);
        const uint32_t s2 = __shfl_sync(0xffffffffu, (uint32_t)s, 16);
        const uint32_t s3 = __shfl_sync(0xffffffffu, (uint32_t)s, 24);
        if (lane == r) my_scales = s0 | (s1 << 8) | (s2 << 16) | (s3 << 24);
    }
    if (lane < kRowsPerWarp)
        reinterpret_cast<uint32_t *>(p.scales + at * (kHeadDim / 32))[lane] = my_scales;
}

__global__ void __launch_bounds__(kThreads) unpack_states_kernel(const PackParams p) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x / p.H;
    const int h = blockIdx.x - b * p.H;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int slot = p.state_idx[b], entry = p.store_idx[b];
    if (!pair_ok(p, slot, entry)) return;
    const int row0 = warp * kRowsPerWarp;
    const size_t at = ((size_t)entry * p.H + h) * kHeadDim + row0;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(p.codes + at * kHeadDim) + lane;
    const uint8_t *sc = p.scales + at * (kHeadDim / 32) + (lane >> 3);
    float *dst = p.pool + ((size_t)slot * p.H + h) * kMat + (size_t)row0 * kHeadDim + lane * 4;
    uint32_t w[kRowsPerWarp];
    uint32_t s[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        w[r] = __ldcs(src + r * (kHeadDim / 4));
        s[r] = sc[r * (kHeadDim / 32)];
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        // 2^(s - 127): s = 0 is the subnormal 2^-127, s = 255 the mark of a block without values
        const float f = s[r] == 255u ? __uint_as_float(0x7fffffffu)
                                     : __uint_as_float(s[r] == 0u ? 0x00400000u : s[r] << 23);
        float4 x;
        x.x = (float)(int8_t)(w[r] & 255u) * f;
        x.y = (float)(int8_t)((w[r] >> 8) & 255u) * f;
        x.z = (float)(int8_t)((w[r] >> 16) & 255u) * f;
        x.w = (float)(int8_t)(w[r] >> 24) * f;
        __stcs(reinterpret_cast<float4 *>(dst + (size_t)r * kHeadDim), x);
    }
}

}  // namespace

cudaError_t launch_pack_states(const PackParams &p, cudaStream_t stream) {
    const long long blocks = (long long)p.B * p.H;
    return launch_pdl(pack_states_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_unpack_states(const PackParams &p, cudaStream_t stream) {
    const long long blocks = (long long)p.B * p.H;
    return launch_pdl(unpack_states_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
}

}  // namespace la
