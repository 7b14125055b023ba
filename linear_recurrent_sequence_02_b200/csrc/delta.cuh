// Shared by the gated delta rule's kernels (internal header).
//
// Per (sequence, value head), row vectors q_t, k_t (dk), v_t (dv), a log
// decay g_t and a write strength b_t, state S [dk, dv] in float32:
//   S <- e^{g_t} S;  x_t = b_t (v_t - k_t S);  S <- S + k_t^T x_t;  o_t = scale q_t S.
// q and k have key_heads heads, each shared by heads / key_heads value heads.
#pragma once

#include "kernels.h"

namespace retnet {

// Tokens of sequence b that belong to it.
__device__ __forceinline__ int delta_tokens_of(const int *lengths, int b, int seqlen) {
    return lengths ? min(max(lengths[b], 0), seqlen) : seqlen;
}

// x is linear in b, and dbeta is (gradient of x) . x / b.  Where b is 0 the
// backward takes a b of this size instead: x keeps all its digits, the
// quotient is the limit, and what it writes to the state is nothing beside it.
__device__ __forceinline__ float nonzero_beta(float b) { return fabsf(b) < 1e-15f ? 1e-15f : b; }

// g where sums of it are formed: e^g is 0 in float32 far above this bound,
// and differences of sums stay finite when g is -inf.
__device__ __forceinline__ float log_decay(float g) { return g < -1000.f ? -1000.f : g; }

}  // namespace retnet
