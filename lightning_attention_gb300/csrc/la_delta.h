// la_delta.h -- the gated delta rule's launchers and their parameters (not part of the ABI).
#pragma once

#include "la_internal.h"

// The entry points have checked all sizes: B and H are at least 1, and the grids fit.
namespace la {

// Per request and value head h, with key head h / group:
//   S <- e^{g_t} S;  u_t = beta_t (v_t - S^T k_t);  S <- S + k_t u_t^T;  o_t = D^-0.5 S^T q_t.
struct DeltaParams {
    const __nv_bfloat16 *q, *k, *v;  // rows of Hk (q, k) and H (v) heads
    long long q_rs, k_rs, v_rs;      // elements from one token's row to the next
    const float *g, *beta;           // [tokens][H]
    float *pool;                     // [num_slots][H][D][D]
    const int32_t *state_idx;        // [B]
    const int32_t *cu_seqlens;       // [B + 1] (extend)
    const uint8_t *prefix_mask;      // [B] (extend)
    float *inter;                    // [B][N][H][D][D] (verify)
    __nv_bfloat16 *out;              // [tokens][H * D]
    unsigned int *err;
    int B, T, H, Hk, N, num_slots, max_seqlen;
    int group;                       // H / Hk
    int l2norm;                      // q and k are divided by sqrt(sum x^2 + kDeltaEps) first
    unsigned long long wait_limit_ns;
};
constexpr float kDeltaEps = 1e-6f;

enum DeltaMode : int { DELTA_DECODE = 0, DELTA_VERIFY = 1, DELTA_SERIAL = 2 };
// Token-serial kernels: the state stays in registers from the first token to the last.  DELTA_SERIAL: an
// extend of at most kSerialTokens tokens a request.  Token by token / by chunks, us, every request of n tokens
// with a prefix state: 8 (request, head) pairs n = 1: 2.8 / 12.9, 4: 4.9 / 12.8, 8: 7.9 / 12.8, 12: 10.9 /
// 12.9, 16: 13.8 / 12.8; 256 pairs n = 8: 20 / 26, 12: 27 / 26; 4,096 pairs n = 1: 86 / 198, 4: 150 / 199,
// 8: 242 / 201.
constexpr int kSerialTokens = 6;
cudaError_t launch_delta_recurrent(DeltaMode mode, const DeltaParams &p, int num_sms,
                                   cudaStream_t stream);

// Chunked extend on the tensor cores (la_delta_extend.cu), of B > 0 requests and T > kSerialTokens tokens; ws:
// delta_scratch_bytes() bytes.
unsigned long long delta_scratch_bytes(long long B, long long T, long long H);
cudaError_t launch_delta_extend(const DeltaParams &p, void *ws, int num_sms, cudaStream_t stream);

// Packed state store: slot state_idx[b] of the pool <-> entry store_idx[b] of codes and scales.
struct PackParams {
    float *pool;               // [num_slots][H][D][D]
    const int32_t *state_idx;  // [B]
    int8_t *codes;             // [entries][H][D][D]
    uint8_t *scales;           // [entries][H][D][D / 32]
    const int32_t *store_idx;  // [B]
    unsigned int *err;
    int B, H, num_slots, entries;
};
cudaError_t launch_pack_states(const PackParams &p, cudaStream_t stream);
cudaError_t launch_unpack_states(const PackParams &p, cudaStream_t stream);

}  // namespace la
