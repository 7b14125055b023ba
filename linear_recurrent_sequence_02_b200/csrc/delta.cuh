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

// Tokens that write nothing: b of 0, or too small for quotients by it.  dbeta
// is (gradient of x) . (v - k S), which for the others is taken from x as
// (gradient of x) . x / b; for these x is 0, whatever v and k hold, and the
// backward forms v - k S beside it.
__device__ __forceinline__ bool writes_nothing(float b) { return fabsf(b) < 1e-15f; }

// g where sums of it are formed: e^g is 0 in float32 from here on, and
// differences of sums stay finite when g is -inf.
__device__ __forceinline__ float log_decay(float g) { return g < -105.f ? -105.f : g; }

// Sums of a chunk's log decays, so that a difference of two keeps float32
// accuracy behind any decays before it: each is an unevaluated sum of two
// floats (the second what the first rounded away, by Knuth's two-sum), and
// they start anew every 16 tokens.
struct DecaySums {
    float2 in[64];                         // from the 16-token block's start, inclusive
    float total[4];                        // of a block
    // G_i - G_j for tokens of one block
    __device__ __forceinline__ float within(int i, int j) const {
        const float2 a = in[i], b = in[j];
        return (a.x - b.x) + (a.y - b.y);
    }
    __device__ __forceinline__ float since_start(int i) const {            // G_i
        float s = 0.f;
        for (int b = 0; b < i / 16; ++b) s += total[b];
        return s + (in[i].x + in[i].y);
    }
    // from token j to the end of block `last` (not before j's own)
    __device__ __forceinline__ float until(int j, int last) const {
        const float2 e = in[j | 15], a = in[j];
        float s = (e.x - a.x) + (e.y - a.y);
        for (int b = j / 16 + 1; b <= last; ++b) s += total[b];
        return s;
    }
};
// By one warp; lo, hi: log decays of tokens lane and lane + 32.
__device__ __forceinline__ void sum_decays(DecaySums &d, int lane, float lo, float hi) {
    float2 a = make_float2(lo, 0.f), b = make_float2(hi, 0.f);
    auto add = [](float2 &x, float h, float l) {           // x + (h + l)
        const float s = x.x + h, v = s - x.x;
        x.y += l + ((x.x - (s - v)) + (h - v));
        x.x = s;
    };
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const float ah = __shfl_up_sync(0xffffffffu, a.x, o), al = __shfl_up_sync(0xffffffffu, a.y, o);
        const float bh = __shfl_up_sync(0xffffffffu, b.x, o), bl = __shfl_up_sync(0xffffffffu, b.y, o);
        if ((lane & 15) >= o) {
            add(a, ah, al);
            add(b, bh, bl);
        }
    }
    d.in[lane] = a;
    d.in[lane + 32] = b;
    if ((lane & 15) == 15) {
        d.total[lane / 16] = a.x + a.y;
        d.total[2 + lane / 16] = b.x + b.y;
    }
}

}  // namespace retnet
