// Gated delta rule, token by token in float32, and its gradient.
//
//   forward   y = k S, z = q S of the state before the token;
//             x = b (v - a y);  S <- a S + k^T x;  o = scale (a z + (q.k) x)
//             with a = e^g.  Both products read the same state, so a token
//             costs one reduction.
//   reverse   D is the gradient of the state behind a token:
//             r = k D + scale (k.q) do;  D <- a (D + scale q^T do - b k^T r).
//             r is the gradient of x; dv = b r.
// Two kernels hold S in registers in float32:
//   delta_step_kernel    one token (decode): an HBM stream of 8 dk dv bytes a
//     head.  A CTA takes 32 columns as the retention step does: 8 float4
//     column groups by 32 row lanes, a column's row lanes reduced by shuffles
//     and then over the eight warps in shared memory.
//   delta_walk_kernel    more tokens (multi-token decode, the float32 prefill,
//     short bf16 ones, and the two sweeps of the float32 backward), bound by
//     the latency of the chain product -> reduction -> update from token to
//     token: a warp owns 4 columns and all rows, so that the chain is nine
//     shuffles and no barrier (1000 tokens of 128 x 64: 650 us in slabs of 32
//     columns, 265 us so, 129 in segments; four tokens a turn by the triangle between them
//     gained a tenth forward and lost it back: one warp a scheduler is then
//     bound by its instructions).
#include "delta.cuh"
#include "pairs.cuh"

namespace retnet {

constexpr int kDeltaThreads = 256;
constexpr int kDeltaCols = 32;                 // state columns per CTA
constexpr int kDeltaGroups = kDeltaCols / 4;   // float4 column groups
constexpr int kDeltaLanes = kDeltaThreads / kDeltaGroups;   // 32 row lanes

// What a walk is for: outputs; x and the states, kept for the gradients; r and
// D, kept, from the last token on; and the state alone, either way.
enum DeltaSweep { kSweepForward, kSweepSave, kSweepReverse, kSweepCarry, kSweepCarryBack };

template <typename T>
__device__ __forceinline__ float4 load_f4(const T *p);
template <>
__device__ __forceinline__ float4 load_f4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load_f4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    uint2 u = *reinterpret_cast<const uint2 *>(p);
    float2 a = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&u.x));
    float2 b = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_f4(float *p, float4 v) {
    *reinterpret_cast<float4 *>(p) = v;
}
__device__ __forceinline__ void store_f4(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}
__device__ __forceinline__ void fma4(float4 &a, float s, float4 v) {
    a.x = fmaf(s, v.x, a.x); a.y = fmaf(s, v.y, a.y);
    a.z = fmaf(s, v.z, a.z); a.w = fmaf(s, v.w, a.w);
}
__device__ __forceinline__ float4 scale4(float s, float4 v) {
    return make_float4(s * v.x, s * v.y, s * v.z, s * v.w);
}
__device__ __forceinline__ void add4(float4 &a, float4 v) {
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
}
__device__ __forceinline__ void reduce_row_lanes(float4 &a) {
#pragma unroll
    for (int m = kDeltaGroups; m < 32; m <<= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, m);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, m);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, m);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, m);
    }
}

// ---- one token in slabs of 32 columns

// q.k by one warp.
template <int DK, typename R>
__device__ __forceinline__ float token_dot(const R *q, const R *k, int lane) {
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < DK / 32; ++j) dot = fmaf(to_f32(q[lane + 32 * j]), to_f32(k[lane + 32 * j]), dot);
#pragma unroll
    for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
    return dot;
}
// This warp's part of y = k S and z = q S.
template <int RPL, typename R>
__device__ __forceinline__ void token_products(const float4 (&s)[RPL], const R *qs, const R *ks,
                                               int rl, int lane, float4 *ry, float4 *rz) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        fma4(y, to_f32(ks[rl + i * kDeltaLanes]), s[i]);
        fma4(z, to_f32(qs[rl + i * kDeltaLanes]), s[i]);
    }
    reduce_row_lanes(y);
    reduce_row_lanes(z);
    if (lane < kDeltaGroups) {
        ry[lane] = y;
        rz[lane] = z;
    }
}
// x, and S <- a S + k^T x.
template <int RPL, typename R>
__device__ __forceinline__ float4 token_update(float4 (&s)[RPL], const R *ks, int rl,
                                               const float4 (*red)[kDeltaGroups], int cg, float4 v,
                                               float a, float b) {
    float4 y = red[0][cg];
#pragma unroll
    for (int w = 1; w < kDeltaThreads / 32; ++w) add4(y, red[w][cg]);
    float4 x = v;
    fma4(x, -a, y);
    x = scale4(b, x);
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        s[i] = scale4(a, s[i]);
        fma4(s[i], to_f32(ks[rl + i * kDeltaLanes]), x);
    }
    return x;
}
__device__ __forceinline__ float4 token_output(const float4 (*red)[kDeltaGroups], int cg, float4 x,
                                               float a, float qk, float scale) {
    float4 z = red[0][cg];
#pragma unroll
    for (int w = 1; w < kDeltaThreads / 32; ++w) add4(z, red[w][cg]);
    float4 o = scale4(a, z);
    fma4(o, qk, x);
    return scale4(scale, o);
}

// One token; q, k [batch, key_heads, DK], v, out [batch, heads, dv].
// Persistent: a CTA takes every gridDim.x-th (sequence, head, 32 columns) and
// copies the states, q, k and v of the next ones to shared memory while it
// works on this one (a CTA for each, its loads waited for, spent two thirds
// of its time at barriers behind them: 128 sequences, 16 heads of 256, 258 us
// against 196 us so).  The state's slots are a thread's own.
template <typename T, int DK>
struct DeltaStepSmem {
    static constexpr int RPL = DK / kDeltaLanes;
    struct Stage {
        float4 s[RPL][kDeltaThreads];
        T q[DK], k[DK], v[kDeltaCols];
    };
    static constexpr int kStages = DK == 256 ? 2 : 4;                // three CTAs share an SM's 227 KB
    Stage stage[kStages];
    float4 red[2][kDeltaThreads / 32][kDeltaGroups];
    float qk;
};
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
template <typename T, int DK>
__global__ void __launch_bounds__(kDeltaThreads, 3)
delta_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                  const T *__restrict__ g, const T *__restrict__ beta,
                  const int *__restrict__ lengths, float *state, T *__restrict__ out, float scale,
                  int heads, int key_heads, int dv, int items) {
    using Smem = DeltaStepSmem<T, DK>;
    constexpr int RPL = Smem::RPL, S = Smem::kStages;
    constexpr int kRowCopies = DK * (int)sizeof(T) / 16;             // of a q or k row
    constexpr int kVCopies = kDeltaCols * (int)sizeof(T) / 16;
    static_assert(128 + kRowCopies + kVCopies <= kDeltaThreads, "threads for the copies");
    extern __shared__ __align__(16) char raw[];
    Smem &m = *reinterpret_cast<Smem *>(raw);
    const int slabs = dv / kDeltaCols, group = heads / key_heads;
    const int cg = threadIdx.x % kDeltaGroups, rl = threadIdx.x / kDeltaGroups;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    grid_dependency_wait();
    auto place = [&](int item, int &bh, int &col) {
        bh = item / slabs;
        col = (item % slabs) * kDeltaCols + cg * 4;
    };
    auto fetch = [&](int item, typename Smem::Stage &st) {
        if (item < items) {
            int bh, col;
            place(item, bh, col);
            const float *src = state + (size_t)bh * DK * dv + col;
#pragma unroll
            for (int i = 0; i < RPL; ++i)
                copy16(&st.s[i][threadIdx.x], src + (size_t)(rl + i * kDeltaLanes) * dv);
            const size_t row = (size_t)(bh / heads) * key_heads + (bh % heads) / group;
            if (threadIdx.x < kRowCopies)
                copy16((char *)st.q + 16 * threadIdx.x, (const char *)(q + row * DK) + 16 * threadIdx.x);
            else if (threadIdx.x - 128 < kRowCopies && threadIdx.x >= 128)
                copy16((char *)st.k + 16 * (threadIdx.x - 128), (const char *)(k + row * DK) + 16 * (threadIdx.x - 128));
            else if (threadIdx.x >= kDeltaThreads - kVCopies) {
                const int c = threadIdx.x - (kDeltaThreads - kVCopies);
                copy16((char *)st.v + 16 * c, (const char *)(v + (size_t)bh * dv + col - cg * 4) + 16 * c);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // decay, write strength and whether the sequence goes on, one item ahead
    float gn = 0.f, bn = 0.f;
    bool on = true;
    auto gates = [&](int item) {
        if (item >= items) return;
        const int bh = item / slabs;
        gn = to_f32(g[bh]);
        bn = to_f32(beta[bh]);
        on = !lengths || lengths[bh / heads] > 0;
    };
#pragma unroll
    for (int u = 0; u < S - 1; ++u) fetch(blockIdx.x + u * gridDim.x, m.stage[u]);
    gates(blockIdx.x);
    int slot = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncthreads();                             // q, k of all threads; the last slot is free
        fetch(item + (S - 1) * gridDim.x, m.stage[(slot + S - 1) % S]);
        typename Smem::Stage &st = m.stage[slot];
        slot = (slot + 1) % S;
        const float a = expf(gn), bt = bn;
        const bool live = on;
        gates(item + gridDim.x);
        if (!live) continue;                         // the whole CTA
        int bh, col;
        place(item, bh, col);
        float4 s[RPL];
#pragma unroll
        for (int i = 0; i < RPL; ++i) s[i] = st.s[i][threadIdx.x];
        token_products<RPL>(s, st.q, st.k, rl, lane, m.red[0][warp], m.red[1][warp]);
        if (warp == 0) {
            const float dot = token_dot<DK>(st.q, st.k, lane);
            if (lane == 0) m.qk = dot;
        }
        __syncthreads();
        const float4 x = token_update<RPL>(s, st.k, rl, m.red[0], cg,
                                           load_f4(&st.v[4 * cg]), a, bt);
        float *dst = state + (size_t)bh * DK * dv + col;
#pragma unroll
        for (int i = 0; i < RPL; ++i) store_f4(dst + (size_t)(rl + i * kDeltaLanes) * dv, s[i]);
        if (warp == 0 && lane < kDeltaGroups)
            store_f4(out + (size_t)bh * dv + col, token_output(m.red[1], cg, x, a, m.qk, scale));
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// N neighbouring values of a row.
template <int N, typename T>
__device__ __forceinline__ void load_row(T (&x)[N], const T *p) {
    constexpr int kBytes = N * (int)sizeof(T);
    if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t *>(x) = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(x) = *reinterpret_cast<const uint2 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            reinterpret_cast<uint4 *>(x)[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
}
constexpr int kWalkWarps = 4, kWalkCols = 4;         // columns per warp
constexpr int kWalkSlab = kWalkWarps * kWalkCols;    // and per CTA
constexpr int kWalkAhead = 4;                        // tokens loaded ahead

// Tokens [first, last) of a (sequence, head), from the state `from` (null:
// zero) to `to` (null: not wanted, may be the same), both [dk, width].  unit
// (kSweepCarry): the state starts as the identity and no values are written,
// so that it ends as the transition of these tokens.
struct DeltaSpan {
    int bh, col, first, last, width;
    const float *from;
    float *to;
    bool unit;
};
// v: the values (forward) or the output's gradient (reverse).
// save: x (kSweepSave; v - k S of tokens that write nothing) or r
// (kSweepReverse), float32 [B, n, H, dv];
// marks: the state before (D behind) every chunk of kDeltaChunk tokens,
// float32 [B, H, chunks, dk, dv].
template <typename T, int DK, DeltaSweep kSweep>
__device__ __forceinline__ void delta_walk(const T *__restrict__ q, const T *__restrict__ k,
                                           const T *__restrict__ v, const T *__restrict__ g,
                                           const T *__restrict__ beta,
                                           const int *__restrict__ lengths, T *__restrict__ out,
                                           float *__restrict__ save, float *__restrict__ marks,
                                           float scale, int heads, int key_heads, int tokens,
                                           int dv, const DeltaSpan &w) {
    constexpr int RPL = DK / 32;                     // rows RPL lane, RPL lane + 1, ...
    constexpr bool kFwd = kSweep == kSweepForward;
    constexpr bool kRev = kSweep == kSweepReverse || kSweep == kSweepCarryBack;
    constexpr bool kKeep = kSweep == kSweepSave || kSweep == kSweepReverse;
    constexpr bool kUsesQ = kFwd || kRev;
    const int bh = w.bh, b = bh / heads, h = bh % heads, kh = h / (heads / key_heads);
    const int lane = threadIdx.x % 32;
    const int col = w.col + (threadIdx.x / 32) * kWalkCols;
    const bool unit = kSweep == kSweepCarry && w.unit;

    grid_dependency_wait();
    const int end = min(w.last, delta_tokens_of(lengths, b, tokens)), begin = min(w.first, end);
    const int n = end - begin;
    const int nc = (tokens + kDeltaChunk - 1) / kDeltaChunk;
    const size_t sbase = (size_t)(RPL * lane) * w.width + col;
    float2 s[RPL][2];
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        float4 x = w.from ? load_f4(w.from + sbase + (size_t)i * w.width) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (unit) {
            const int one = RPL * lane + i - col;
            x = make_float4(one == 0, one == 1, one == 2, one == 3);
        }
        s[i][0] = make_float2(x.x, x.y);
        s[i][1] = make_float2(x.z, x.w);
    }
    auto store_state = [&](float *dst, int stride) {
#pragma unroll
        for (int i = 0; i < RPL; ++i)
            store_f4(dst + (size_t)i * stride, make_float4(s[i][0].x, s[i][0].y, s[i][1].x, s[i][1].y));
    };

    // the tokens ahead, as they lie in memory; pointers step along the walk
    struct Token {
        alignas(16) T k[RPL];
        alignas(16) T q[RPL];
        alignas(16) T v[4];
        T g, b;
    } ahead[kWalkAhead];
    const long long dir = kRev ? -1 : 1;
    const size_t start = (size_t)b * tokens + (kRev ? max(end - 1, 0) : begin);
    const T *kp = k + (start * key_heads + kh) * DK + RPL * lane;
    const T *qp = q + (start * key_heads + kh) * DK + RPL * lane;
    const T *vp = v + (start * heads + h) * dv + col;
    const T *gp = g + start * heads + h, *bp = beta + start * heads + h;
    const long long kstep = dir * key_heads * DK, vstep = dir * heads * dv, gstep = dir * heads;
    auto load = [&](Token &t, bool more) {
        if (more) {
            load_row<RPL>(t.k, kp);
            if (kUsesQ) load_row<RPL>(t.q, qp);
            if (!unit) load_row<4>(t.v, vp);
            t.g = *gp;
            t.b = *bp;
            kp += kstep;
            qp += kstep;
            vp += vstep;
            gp += gstep;
            bp += gstep;
        }
    };
#pragma unroll
    for (int u = 0; u < kWalkAhead; ++u) load(ahead[u], u < n);
    size_t vo = (start * heads + h) * dv + col;
    for (int s0 = 0; s0 < n; s0 += kWalkAhead) {
#pragma unroll
        for (int u = 0; u < kWalkAhead; ++u) {
            const int step = s0 + u;
            if (step >= n) break;
            float wk[RPL], wq[RPL];
#pragma unroll
            for (int i = 0; i < RPL; ++i) {
                wk[i] = to_f32(ahead[u].k[i]);
                if (kUsesQ) wq[i] = to_f32(ahead[u].q[i]);
            }
            const float2 v0 = unit ? both(0.f) : make_float2(to_f32(ahead[u].v[0]), to_f32(ahead[u].v[1]));
            const float2 v1 = unit ? both(0.f) : make_float2(to_f32(ahead[u].v[2]), to_f32(ahead[u].v[3]));
            const float a = expf(to_f32(ahead[u].g)), bt = to_f32(ahead[u].b);
            load(ahead[u], step + kWalkAhead < n);
            if (kKeep) {
                const int t = kRev ? end - 1 - step : begin + step;
                if (kRev ? step == 0 || t % kDeltaChunk == kDeltaChunk - 1 : t % kDeltaChunk == 0)
                    store_state(marks + (((size_t)bh * nc + t / kDeltaChunk) * DK + RPL * lane) * dv + col, dv);
            }
            float2 y0 = both(0.f), y1 = y0, z0 = y0, z1 = y0;
            float d = 0.f;                           // q.k
#pragma unroll
            for (int i = 0; i < RPL; ++i) {
                y0 = fma2(both(wk[i]), s[i][0], y0);
                y1 = fma2(both(wk[i]), s[i][1], y1);
                if (kFwd) {
                    z0 = fma2(both(wq[i]), s[i][0], z0);
                    z1 = fma2(both(wq[i]), s[i][1], z1);
                }
                if (kUsesQ) d = fmaf(wq[i], wk[i], d);
            }
            // sums over the lanes: a lane gives away the half of the values
            // that it does not keep, so that it ends with one; q.k goes along
            auto pass = [](float x, int m) { return __shfl_xor_sync(0xffffffffu, x, m); };
            if (kFwd) {                              // lanes 0-15 y, 16-31 z
                const bool up = lane & 16;
                const float2 k0 = up ? z0 : y0, k1 = up ? z1 : y1, g0 = up ? y0 : z0, g1 = up ? y1 : z1;
                y0 = add2(k0, make_float2(pass(g0.x, 16), pass(g0.y, 16)));
                y1 = add2(k1, make_float2(pass(g1.x, 16), pass(g1.y, 16)));
            }
            if (kUsesQ) d += pass(d, 16);
            const bool far = lane & 8, odd = lane & 4;
            const float2 k2 = far ? y1 : y0, g2 = far ? y0 : y1;
            const float2 h2 = add2(k2, make_float2(pass(g2.x, 8), pass(g2.y, 8)));
            if (kUsesQ) d += pass(d, 8);
            float e = (odd ? h2.y : h2.x) + pass(odd ? h2.x : h2.y, 4);
            if (kUsesQ) d += pass(d, 4);
            if (!kFwd) e += pass(e, 16);
            e += pass(e, 2);
            if (kUsesQ) d += pass(d, 2);
            e += pass(e, 1);
            if (kUsesQ) d += pass(d, 1);
            y0 = make_float2(__shfl_sync(0xffffffffu, e, 0), __shfl_sync(0xffffffffu, e, 4));
            y1 = make_float2(__shfl_sync(0xffffffffu, e, 8), __shfl_sync(0xffffffffu, e, 12));
            float2 x0, x1;
            if (kRev) {
                x0 = fma2(both(scale * d), v0, y0);                // r
                x1 = fma2(both(scale * d), v1, y1);
                const float2 b0 = mul2(both(-bt), x0), b1 = mul2(both(-bt), x1);
                const float2 o0 = mul2(both(scale), v0), o1 = mul2(both(scale), v1);
#pragma unroll
                for (int i = 0; i < RPL; ++i) {
                    s[i][0] = mul2(both(a), fma2(both(wk[i]), b0, fma2(both(wq[i]), o0, s[i][0])));
                    s[i][1] = mul2(both(a), fma2(both(wk[i]), b1, fma2(both(wq[i]), o1, s[i][1])));
                }
            } else {
                const float2 u0 = fma2(both(-a), y0, v0), u1 = fma2(both(-a), y1, v1);
                x0 = mul2(both(bt), u0);
                x1 = mul2(both(bt), u1);
#pragma unroll
                for (int i = 0; i < RPL; ++i) {
                    s[i][0] = fma2(both(wk[i]), x0, mul2(both(a), s[i][0]));
                    s[i][1] = fma2(both(wk[i]), x1, mul2(both(a), s[i][1]));
                }
                if (kSweep == kSweepSave && writes_nothing(bt)) {
                    x0 = u0;                         // v - k S is kept in the place of x
                    x1 = u1;
                }
            }
            if (kFwd) {
                // lanes 16, 20, 24, 28 hold z of columns 0 .. 3
                const float xe = far ? (odd ? x1.y : x1.x) : (odd ? x0.y : x0.x);
                if ((lane & 19) == 16) out[vo + (lane - 16) / 4] = from_f32<T>(scale * fmaf(d, xe, a * e));
            } else if (kKeep && lane == 0) {
                store_f4(save + vo, make_float4(x0.x, x0.y, x1.x, x1.y));
            }
            vo += vstep;
        }
    }
    if (w.to && (n > 0 || w.to != w.from)) store_state(w.to + sbase, w.width);
}

// All tokens, for the CTA's columns.
__device__ __forceinline__ DeltaSpan whole_span(int cta, int tokens, int dk, int dv, const float *from,
                                                float *to) {
    const int slabs = dv / kWalkSlab, bh = cta / slabs;
    const size_t at = (size_t)bh * dk * dv;
    return {bh, (cta % slabs) * kWalkSlab, 0, tokens, dv, from ? from + at : nullptr,
            to ? to + at : nullptr, false};
}

template <typename T, int DK>
__global__ void __launch_bounds__(32 * kWalkWarps)
delta_walk_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                  const T *__restrict__ g, const T *__restrict__ beta,
                  const int *__restrict__ lengths, const float *state_in, float *state_out,
                  T *__restrict__ out, float scale, int heads, int key_heads, int tokens, int dv) {
    delta_walk<T, DK, kSweepForward>(q, k, v, g, beta, lengths, out, nullptr, nullptr, scale, heads,
                                     key_heads, tokens, dv,
                                     whole_span(blockIdx.x, tokens, DK, dv, state_in, state_out));
}
// The backward's two sweeps: neither needs the other, so they share a launch.
template <typename T, int DK>
__global__ void __launch_bounds__(32 * kWalkWarps)
delta_sweeps_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                    const T *__restrict__ d_out, const T *__restrict__ g, const T *__restrict__ beta,
                    const int *__restrict__ lengths, float *xs, float *ss, float *rs, float *ds,
                    float scale, int heads, int key_heads, int tokens, int dv) {
    const int half = gridDim.x / 2, cta = (int)blockIdx.x < half ? blockIdx.x : blockIdx.x - half;
    const DeltaSpan w = whole_span(cta, tokens, DK, dv, nullptr, nullptr);
    if ((int)blockIdx.x < half)
        delta_walk<T, DK, kSweepSave>(q, k, v, g, beta, lengths, nullptr, xs, ss, scale, heads,
                                      key_heads, tokens, dv, w);
    else
        delta_walk<T, DK, kSweepReverse>(q, k, d_out, g, beta, lengths, nullptr, rs, ds, scale,
                                         heads, key_heads, tokens, dv, w);
}

// ---- in segments, as the tensor-core walk goes with few heads (see
// delta_segments_kernel): segment 0 as it is and what the later ones do to a
// state, S -> M S + N, all at once; the states between, by launch_delta_join;
// then the later segments' outputs all at once.
// starts [segments - 1][BH][dk, dv], units [segments - 2][BH][dk, dk].
struct DeltaSegments {
    int count, tokens;                     // of a segment
    float *starts, *units, *back;          // back: starts of the reverse sweep
};
template <int DK>
__global__ void __launch_bounds__(32 * kWalkWarps)
delta_walk_segments_kernel(const float *__restrict__ q, const float *__restrict__ k,
                           const float *__restrict__ v, const float *__restrict__ g,
                           const float *__restrict__ beta, const int *__restrict__ lengths,
                           const float *state_in, float *state_out, float *__restrict__ out,
                           float scale, int heads, int key_heads, int tokens, int dv,
                           DeltaSegments x, int bhs, int last) {
    const int walks = bhs * (dv / kWalkSlab);
    const size_t ssize = (size_t)DK * dv;
    int cta = blockIdx.x;
    if (last || cta < walks) {                               // outputs
        const int seg = last ? 1 + cta / walks : 0;
        DeltaSpan w = whole_span(cta % walks, tokens, DK, dv, state_in, state_out);
        if (last) w.from = x.starts + ((size_t)(seg - 1) * bhs + w.bh) * ssize;
        else w.to = x.starts + (size_t)w.bh * ssize;
        if (last && seg < x.count - 1) w.to = nullptr;
        w.first = seg * x.tokens;
        w.last = w.first + x.tokens;
        delta_walk<float, DK, kSweepForward>(q, k, v, g, beta, lengths, out, nullptr, nullptr, scale,
                                         heads, key_heads, tokens, dv, w);
    } else {
        DeltaSpan w;
        int seg;
        if (cta < walks * (x.count - 1)) {                   // N
            seg = cta / walks;
            w = whole_span(cta % walks, tokens, DK, dv, nullptr, nullptr);
            w.to = x.starts + ((size_t)seg * bhs + w.bh) * ssize;
        } else {                                             // M
            constexpr int kSlabs = DK / kWalkSlab;
            cta -= walks * (x.count - 1);
            seg = 1 + cta / (bhs * kSlabs);
            w = whole_span(cta % (bhs * kSlabs), tokens, DK, DK, nullptr, nullptr);
            w.to = x.units + ((size_t)(seg - 1) * bhs + w.bh) * DK * DK;
            w.unit = true;
        }
        w.first = seg * x.tokens;
        w.last = w.first + x.tokens;
        delta_walk<float, DK, kSweepCarry>(q, k, v, g, beta, lengths, nullptr, nullptr, nullptr, scale,
                                       heads, key_heads, tokens, dv, w);
    }
}

// The backward's two sweeps in segments.  Back through segment j the gradient
// of the state goes by D -> M_j^T D + N'_j, so the units serve both.
// back [segments - 1]: D behind segment segments - 2 first.
template <typename T, int DK>
__global__ void __launch_bounds__(32 * kWalkWarps)
delta_sweeps_segments_kernel(const T *__restrict__ q, const T *__restrict__ k,
                             const T *__restrict__ v, const T *__restrict__ d_out,
                             const T *__restrict__ g, const T *__restrict__ beta,
                             const int *__restrict__ lengths, float *xs, float *ss, float *rs,
                             float *ds, float scale, int heads, int key_heads, int tokens, int dv,
                             DeltaSegments x, int bhs, int last) {
    const int walks = bhs * (dv / kWalkSlab), ends = last ? walks * (x.count - 1) : walks;
    const size_t ssize = (size_t)DK * dv;
    int cta = blockIdx.x;
    auto span = [&](int seg, const float *from, float *to) {
        DeltaSpan w = whole_span(cta % walks, tokens, DK, dv, from, to);
        w.first = seg * x.tokens;
        w.last = w.first + x.tokens;
        return w;
    };
    auto state = [&](float *base, int i) { return base + (size_t)i * bhs * ssize; };
    if (cta < ends) {                                        // kept, forward
        const int seg = last ? 1 + cta / walks : 0;
        delta_walk<T, DK, kSweepSave>(q, k, v, g, beta, lengths, nullptr, xs, ss, scale, heads,
                                      key_heads, tokens, dv,
                                      last ? span(seg, state(x.starts, seg - 1), nullptr)
                                           : span(0, nullptr, x.starts));
    } else if ((cta -= ends) < ends) {                       // kept, back
        const int seg = last ? x.count - 2 - cta / walks : x.count - 1;
        delta_walk<T, DK, kSweepReverse>(q, k, d_out, g, beta, lengths, nullptr, rs, ds, scale,
                                         heads, key_heads, tokens, dv,
                                         last ? span(seg, state(x.back, x.count - 2 - seg), nullptr)
                                              : span(seg, nullptr, x.back));
    } else if ((cta -= ends) < walks * (x.count - 2)) {      // N'
        const int seg = 1 + cta / walks;
        delta_walk<T, DK, kSweepCarryBack>(q, k, d_out, g, beta, lengths, nullptr, nullptr, nullptr,
                                           scale, heads, key_heads, tokens, dv,
                                           span(seg, nullptr, state(x.back, x.count - 1 - seg)));
    } else {
        cta -= walks * (x.count - 2);
        DeltaSpan w;
        if (cta < walks * (x.count - 2)) {                   // N
            const int seg = 1 + cta / walks;
            w = span(seg, nullptr, state(x.starts, seg));
        } else {                                             // M
            constexpr int kSlabs = DK / kWalkSlab;
            cta -= walks * (x.count - 2);
            const int seg = 1 + cta / (bhs * kSlabs);
            w = whole_span(cta % (bhs * kSlabs), tokens, DK, DK, nullptr, nullptr);
            w.first = seg * x.tokens;
            w.last = w.first + x.tokens;
            w.to = x.units + ((size_t)(seg - 1) * bhs + w.bh) * DK * DK;
            w.unit = true;
        }
        delta_walk<T, DK, kSweepCarry>(q, k, v, g, beta, lengths, nullptr, nullptr, nullptr, scale,
                                       heads, key_heads, tokens, dv, w);
    }
}

// ------------------------------------------------------------------ gradients
// One CTA per chunk of 64 tokens of a (sequence, head).  With X, R (the
// gradients of X), the state S before the chunk and D (the gradient of the
// state behind it), G the running sum of g inside the chunk:
//   A_ij = scale (do_i . x_j) e^{G_i - G_j},  i >= j
//   B_ij = -b_i (r_i . x_j) e^{G_i - G_j},    i > j
//   dq = scale e^G (do S^T) + A K
//   dk = e^{G_L - G} (X D^T) - b e^G (R S^T) + A^T Q + (B + B^T) K
//   dv = b R,   dbeta = R . X / b  (R . X of tokens that write nothing: the
//   walk has left v - k S in X for them, which A, B and dk leave out)
// dg_t is the sum of everything that crosses token t, each term formed once
// and added to the tokens it crosses: the pairs E = A (.) QK^T + B (.) KK^T
// with j < t <= i (rows minus columns of E summed from t on: the same float
// for both, so what does not cross cancels), what leaves S at i >= t, what
// reaches D from j < t, and e^{G_L} <S, D>.
constexpr int kGradThreads = 256;
constexpr int kGradPad = 36;           // row stride of a 64 x 32 tile
constexpr int kGradPadK = 68;          // row stride of a 64 x 64 tile

struct DeltaGradSmem {
    float A[64][kGradPadK], B[64][kGradPadK];
    float Ks[64][kGradPadK], Qs[64][kGradPadK];
    float X[64][kGradPad], R[64][kGradPad], O[64][kGradPad];
    float S[64][kGradPad], D[64][kGradPad];
    DecaySums G;
    float e[64], rest[64];                 // e^G, e^{G_L - G}
    float beta[64], rowsum[64], colsum[64], inter[64], ahead[64], db[64];
    float part[kGradThreads / 32];
};

// acc[4][4] += rows r0.. of a times rows c0.. of b over 32 columns
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float (*a)[kGradPad],
                                         const float (*b)[kGradPad], int r0, int c0) {
#pragma unroll 2
    for (int j = 0; j < 32; j += 4) {
        float4 av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = *reinterpret_cast<const float4 *>(&a[r0 + 16 * i][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) bv[i] = *reinterpret_cast<const float4 *>(&b[c0 + 16 * i][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                acc[i][l] = fmaf(av[i].x, bv[l].x, acc[i][l]);
                acc[i][l] = fmaf(av[i].y, bv[l].y, acc[i][l]);
                acc[i][l] = fmaf(av[i].z, bv[l].z, acc[i][l]);
                acc[i][l] = fmaf(av[i].w, bv[l].w, acc[i][l]);
            }
    }
}

template <typename T>
__global__ void __launch_bounds__(kGradThreads)
delta_grad_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ d_out,
                  const T *__restrict__ g, const T *__restrict__ beta,
                  const int *__restrict__ lengths, const float *__restrict__ xs,
                  const float *__restrict__ rs, const float *__restrict__ ss,
                  const float *__restrict__ ds, T *dq, T *dk_, T *dv_, T *dg, T *dbeta,
                  float *dq_wide, float *dk_wide, float scale, int heads, int key_heads,
                  int tokens, int dk, int dv) {
    extern __shared__ __align__(16) char raw[];
    DeltaGradSmem &m = *reinterpret_cast<DeltaGradSmem *>(raw);
    const int nc = (tokens + kDeltaChunk - 1) / kDeltaChunk;
    const int bh = blockIdx.x / nc, c = blockIdx.x % nc;
    const int b = bh / heads, h = bh % heads, kh = h / (heads / key_heads);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    grid_dependency_wait();
    const int n = delta_tokens_of(lengths, b, tokens);
    const int t0 = c * kDeltaChunk;
    const int room = min(kDeltaChunk, tokens - t0);          // rows of the chunk
    const int cnt = min(max(n - t0, 0), room);               // tokens of the sequence
    const size_t row0 = (size_t)b * tokens + t0;
    const bool shared_keys = heads != key_heads;

    // rows behind the sequence have no gradient
    for (int i = cnt + warp; i < room; i += kGradThreads / 32) {
        T *v = dv_ + ((row0 + i) * heads + h) * (size_t)dv;
        for (int j = lane; j < dv; j += 32) v[j] = from_f32<T>(0.f);
        for (int j = lane; j < dk; j += 32) {
            const size_t o = ((row0 + i) * (shared_keys ? heads : key_heads) + h) * (size_t)dk + j;
            if (shared_keys) {
                dq_wide[o] = 0.f;
                dk_wide[o] = 0.f;
            } else {
                dq[o] = from_f32<T>(0.f);
                dk_[o] = from_f32<T>(0.f);
            }
        }
        if (lane == 0) {
            dg[(row0 + i) * heads + h] = from_f32<T>(0.f);
            dbeta[(row0 + i) * heads + h] = from_f32<T>(0.f);
        }
    }
    if (cnt == 0) return;                                    // the whole CTA

    if (tid < 64) {
        m.beta[tid] = tid < cnt ? to_f32(beta[(row0 + tid) * heads + h]) : 0.f;
        m.rowsum[tid] = m.colsum[tid] = m.inter[tid] = m.ahead[tid] = m.db[tid] = 0.f;
    }
    if (warp == 0) {
        const float lo = lane < cnt ? log_decay(to_f32(g[(row0 + lane) * heads + h])) : 0.f;
        const float hi = lane + 32 < cnt ? log_decay(to_f32(g[(row0 + lane + 32) * heads + h])) : 0.f;
        sum_decays(m.G, lane, lo, hi);
        __syncwarp();
#pragma unroll
        for (int t = lane; t < 64; t += 32) {
            m.e[t] = expf(m.G.since_start(t));
            m.rest[t] = expf(m.G.until(t, 3));
        }
    }
    __syncthreads();

    auto load_rows = [&](float (*dst)[kGradPad], auto src, size_t stride, int rows) {
        const int r = tid / 8, j = (tid % 8) * 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = r + 32 * i;
            const float4 x = rr < rows ? load_f4(src + (size_t)rr * stride + j)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(&dst[rr][j]) = x;
        }
    };
    auto load_keys = [&](float (*dst)[kGradPadK], const T *src) {
        const int r = tid / 16, j = (tid % 16) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = r + 16 * i;
            const float4 x = rr < cnt ? load_f4(src + (size_t)rr * key_heads * dk + j)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(&dst[rr][j]) = x;
        }
    };
    const size_t vrow = (row0 * heads + h) * (size_t)dv, vstep = (size_t)heads * dv;
    const size_t krow = (row0 * key_heads + kh) * (size_t)dk;
    const float *S0 = ss + ((size_t)bh * nc + c) * dk * dv, *D0 = ds + ((size_t)bh * nc + c) * dk * dv;
    const int r0 = tid / 16, c0 = tid % 16;                  // rows r0 + 16 i, columns c0 + 16 l

    // ---- the pairs of the chunk
    float pa[4][4] = {}, pb[4][4] = {}, fq[4][4] = {}, fk[4][4] = {};
    for (int j = 0; j < dv; j += 32) {
        load_rows(m.X, xs + vrow + j, vstep, cnt);
        load_rows(m.R, rs + vrow + j, vstep, cnt);
        load_rows(m.O, d_out + vrow + j, vstep, cnt);
        __syncthreads();
        dot_tile(pa, m.O, m.X, r0, c0);
        dot_tile(pb, m.R, m.X, r0, c0);
        for (int i = warp; i < cnt; i += kGradThreads / 32) {
            const float r = m.R[i][lane];
            dv_[vrow + (size_t)i * vstep + j + lane] = from_f32<T>(m.beta[i] * r);
            float d = r * m.X[i][lane];
#pragma unroll
            for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            if (lane == 0) m.db[i] += d;                     // one warp owns row i
        }
        __syncthreads();
    }
    for (int j = 0; j < dk; j += 32) {                       // through the X and R tiles
        load_rows(m.X, k + krow + j, (size_t)key_heads * dk, cnt);
        load_rows(m.R, q + krow + j, (size_t)key_heads * dk, cnt);
        __syncthreads();
        dot_tile(fq, m.R, m.X, r0, c0);
        dot_tile(fk, m.X, m.X, r0, c0);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ri = r0 + 16 * i;
        float rsum = 0.f;
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            const int cj = c0 + 16 * l;
            float dec = 0.f;
            if (ri >= cj && ri < cnt)
                dec = expf(ri / 16 == cj / 16 ? m.G.within(ri, cj)
                                              : m.G.until(cj, ri / 16 - 1) + (m.G.in[ri].x + m.G.in[ri].y));
            const bool none = writes_nothing(m.beta[cj]);
            const float va = none ? 0.f : scale * dec * pa[i][l];
            const float vb = ri > cj && !none ? -m.beta[ri] * dec * pb[i][l] : 0.f;
            m.A[ri][cj] = va;
            m.B[ri][cj] = vb;
            fq[i][l] = ri == cj ? 0.f : fmaf(va, fq[i][l], vb * fk[i][l]);   // E off the diagonal
            rsum += fq[i][l];
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) rsum += __shfl_xor_sync(0xffffffffu, rsum, o, 16);
        if (c0 == 0) m.rowsum[ri] = rsum;
    }
    // columns of E through the (free) X, R tiles' space: 16 partial rows of 64
    float *cols = &m.X[0][0];
#pragma unroll
    for (int l = 0; l < 4; ++l)
        cols[r0 * 64 + c0 + 16 * l] = fq[0][l] + fq[1][l] + fq[2][l] + fq[3][l];
    __syncthreads();
    if (tid < 64) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a += cols[i * 64 + tid];
        m.colsum[tid] = a;
    }
    __syncthreads();

    // ---- through the states, 64 rows of S and D at a time
    float sd = 0.f;
    for (int j0 = 0; j0 < dk; j0 += 64) {
        float aq[4][4] = {}, ar[4][4] = {}, ax[4][4] = {};
        load_keys(m.Ks, k + krow + j0);
        load_keys(m.Qs, q + krow + j0);
        for (int j = 0; j < dv; j += 32) {
            load_rows(m.X, xs + vrow + j, vstep, cnt);
            load_rows(m.R, rs + vrow + j, vstep, cnt);
            load_rows(m.O, d_out + vrow + j, vstep, cnt);
            load_rows(m.S, S0 + (size_t)j0 * dv + j, dv, 64);
            load_rows(m.D, D0 + (size_t)j0 * dv + j, dv, 64);
            __syncthreads();
            dot_tile(aq, m.O, m.S, r0, c0);
            dot_tile(ar, m.R, m.S, r0, c0);
            dot_tile(ax, m.X, m.D, r0, c0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = tid + i * kGradThreads;
                sd = fmaf(m.S[e / 32][e % 32], m.D[e / 32][e % 32], sd);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ri = r0 + 16 * i;
            const float e = m.e[ri], rest = m.rest[ri];
            const float bt = m.beta[ri];
            float inter = 0.f, ahead = 0.f;
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const int cj = c0 + 16 * l;
                aq[i][l] *= scale * e;
                ar[i][l] *= -bt * e;
                ax[i][l] = writes_nothing(bt) ? 0.f : ax[i][l] * rest;
                inter = fmaf(m.Qs[ri][cj], aq[i][l], inter);
                inter = fmaf(m.Ks[ri][cj], ar[i][l], inter);
                ahead = fmaf(m.Ks[ri][cj], ax[i][l], ahead);
                ar[i][l] += ax[i][l];
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) {
                inter += __shfl_xor_sync(0xffffffffu, inter, o, 16);
                ahead += __shfl_xor_sync(0xffffffffu, ahead, o, 16);
            }
            if (c0 == 0) {
                m.inter[ri] += inter;
                m.ahead[ri] += ahead;
            }
        }
        for (int t = 0; t < cnt; ++t) {                      // A K; A^T Q + (B + B^T) K
            float kv[4], qv[4];
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                kv[l] = m.Ks[t][c0 + 16 * l];
                qv[l] = m.Qs[t][c0 + 16 * l];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ri = r0 + 16 * i;
                const float a = m.A[ri][t], at = m.A[t][ri], bb = m.B[ri][t] + m.B[t][ri];
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    aq[i][l] = fmaf(a, kv[l], aq[i][l]);
                    ar[i][l] = fmaf(at, qv[l], ar[i][l]);
                    ar[i][l] = fmaf(bb, kv[l], ar[i][l]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ri = r0 + 16 * i;
            if (ri < cnt) {
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    const int cj = j0 + c0 + 16 * l;
                    if (shared_keys) {
                        const size_t o = ((row0 + ri) * heads + h) * (size_t)dk + cj;
                        dq_wide[o] = aq[i][l];
                        dk_wide[o] = ar[i][l];
                    } else {
                        const size_t o = krow + (size_t)ri * key_heads * dk + cj;
                        dq[o] = from_f32<T>(aq[i][l]);
                        dk_[o] = from_f32<T>(ar[i][l]);
                    }
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
    if (lane == 0) m.part[warp] = sd;
    __syncthreads();
    if (tid < cnt) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kGradThreads / 32; ++w) s += m.part[w];
        s *= m.e[63];
        for (int i = cnt - 1; i >= tid; --i) s += (m.rowsum[i] - m.colsum[i]) + m.inter[i];
        for (int i = 0; i < tid; ++i) s += m.ahead[i];
        dg[(row0 + tid) * heads + h] = from_f32<T>(s);
        dbeta[(row0 + tid) * heads + h] = from_f32<T>(writes_nothing(m.beta[tid]) ? m.db[tid] : m.db[tid] / m.beta[tid]);
    }
}

// dq, dk of a shared key head: the sum over its value heads, in head order.
template <typename T>
__global__ void __launch_bounds__(256)
delta_share_kernel(const float *__restrict__ dq_wide, const float *__restrict__ dk_wide, T *dq,
                   T *dk_, long long vecs, int group, int dk) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;   // a float4 of (row, key head)
    grid_dependency_wait();
    if (i >= vecs) return;
    const int per = dk / 4;
    const long long rh = i / per;
    const size_t src = (size_t)rh * group * dk + (i % per) * 4;
    const float *from = blockIdx.y ? dk_wide : dq_wide;
    float4 a = load_f4(from + src);
    for (int w = 1; w < group; ++w) add4(a, load_f4(from + src + (size_t)w * dk));
    store_f4((blockIdx.y ? dk_ : dq) + (size_t)i * 4, a);
}

// ------------------------------------------------------------------ launches
static size_t walk_ctas(const DeltaArgs &a) {
    return (size_t)a.batch * a.heads * (a.dv / kWalkSlab);
}
template <typename T, int DK>
static cudaError_t launch_walk(const DeltaArgs &a, cudaStream_t stream) {
    return launch_overlapped(delta_walk_kernel<T, DK>, dim3((unsigned)walk_ctas(a)),
                             dim3(32 * kWalkWarps), 0, stream, (const T *)a.q, (const T *)a.k,
                             (const T *)a.v, (const T *)a.g, (const T *)a.beta, a.lengths,
                             a.state_in, a.state_out, (T *)a.out, a.scale, a.heads, a.key_heads,
                             a.seqlen, a.dv);
}
template <int DK>
static cudaError_t launch_walk_segments(const DeltaArgs &a, const DeltaSegments &x, int ctas,
                                        int last, cudaStream_t stream) {
    return launch_overlapped(delta_walk_segments_kernel<DK>, dim3((unsigned)ctas),
                             dim3(32 * kWalkWarps), 0, stream, (const float *)a.q, (const float *)a.k,
                             (const float *)a.v, (const float *)a.g, (const float *)a.beta, a.lengths,
                             a.state_in, a.state_out, (float *)a.out, a.scale, a.heads, a.key_heads,
                             a.seqlen, a.dv, x, a.batch * a.heads, last);
}
struct DeltaSweepOut {
    float *xs, *ss, *rs, *ds;
};
template <typename T, int DK>
static cudaError_t launch_sweeps(const DeltaArgs &a, const DeltaSweepOut &o, cudaStream_t stream) {
    return launch_overlapped(delta_sweeps_kernel<T, DK>, dim3((unsigned)(2 * walk_ctas(a))),
                             dim3(32 * kWalkWarps), 0, stream, (const T *)a.q, (const T *)a.k,
                             (const T *)a.v, (const T *)a.d_out, (const T *)a.g,
                             (const T *)a.beta, a.lengths, o.xs, o.ss, o.rs, o.ds, a.scale,
                             a.heads, a.key_heads, a.seqlen, a.dv);
}
template <typename T, int DK>
static cudaError_t launch_sweeps_segments(const DeltaArgs &a, const DeltaSweepOut &o,
                                          const DeltaSegments &x, int ctas, int last,
                                          cudaStream_t stream) {
    return launch_overlapped(delta_sweeps_segments_kernel<T, DK>, dim3((unsigned)ctas),
                             dim3(32 * kWalkWarps), 0, stream, (const T *)a.q, (const T *)a.k,
                             (const T *)a.v, (const T *)a.d_out, (const T *)a.g,
                             (const T *)a.beta, a.lengths, o.xs, o.ss, o.rs, o.ds, a.scale,
                             a.heads, a.key_heads, a.seqlen, a.dv, x, a.batch * a.heads, last);
}
template <typename T, int DK>
static cudaError_t launch_step(const DeltaArgs &a, cudaStream_t stream) {
    constexpr int kBytes = (int)sizeof(DeltaStepSmem<T, DK>);
    cudaError_t e = cudaFuncSetAttribute(delta_step_kernel<T, DK>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    const int items = a.batch * a.heads * (a.dv / kDeltaCols), resident = 148 * 3;
    return launch_overlapped(delta_step_kernel<T, DK>, dim3((unsigned)(items < resident ? items : resident)),
                             dim3(kDeltaThreads), kBytes, stream, (const T *)a.q, (const T *)a.k,
                             (const T *)a.v, (const T *)a.g, (const T *)a.beta, a.lengths,
                             a.state_out, (T *)a.out, a.scale, a.heads, a.key_heads, a.dv, items);
}

#define RETNET_DELTA_CASES(CALL, ...)                                            \
    if (a.dtype == RETNET_BF16) switch (a.dk) {                                  \
            case 64: return CALL<__nv_bfloat16, 64>(__VA_ARGS__);                \
            case 128: return CALL<__nv_bfloat16, 128>(__VA_ARGS__);              \
            default: return CALL<__nv_bfloat16, 256>(__VA_ARGS__);               \
        }                                                                        \
    switch (a.dk) {                                                              \
        case 64: return CALL<float, 64>(__VA_ARGS__);                            \
        case 128: return CALL<float, 128>(__VA_ARGS__);                          \
        default: return CALL<float, 256>(__VA_ARGS__);                           \
    }

cudaError_t launch_delta_step(const DeltaArgs &a, cudaStream_t stream) {
    KernelTimer timer("delta_step", stream);
    count_launch();
    RETNET_DELTA_CASES(launch_step, a, stream)
}

cudaError_t launch_delta_walk(const DeltaArgs &a, cudaStream_t stream) {
    KernelTimer timer("delta_walk", stream);
    count_launch();
    RETNET_DELTA_CASES(launch_walk, a, stream)
}

static cudaError_t sweep(const DeltaArgs &a, const DeltaSweepOut &o, cudaStream_t stream) {
    KernelTimer timer("delta_sweeps", stream);
    count_launch();
    RETNET_DELTA_CASES(launch_sweeps, a, o, stream)
}

// ---- segments of the walks
// How many segments, and tokens of each (a multiple of `unit`).  Time in
// tokens behind one another (0.26 us): both passes with the waves of CTAs that
// their registers allow (two CTAs of an SM take 1.2 times as long as one,
// three 1.5), 30 for the further launches, 10 a join of states (4 for dk 64).
// Measured: 8 heads, 1000 tokens, 128 x 64: 263 us whole, 129 in 6 segments;
// 1 head, 8192 tokens, 128 x 128: 2120 and 288 in 24; 64 heads, 512 tokens:
// 343 and 518 in 3 (whole).  Backward, 1 head, 4096 tokens: 1221 and 302 in
// 16; 18 heads, 333 tokens: 142 and 173 in 3 (whole).  A join reads whole
// transitions, for dk 256 four times those of 128, so dk 256 walks whole.
static DeltaSegments walk_segments(int batch, int heads, int seqlen, int dk, int dv, int unit,
                                   bool backward) {
    DeltaSegments x = {1, seqlen, nullptr, nullptr, nullptr};
    if (dk > 128) return x;
    const long long bh = (long long)batch * heads, units = bh * (dk / kWalkSlab);
    const long long walks = bh * (dv / kWalkSlab) * (backward ? 2 : 1);
    const int resident = dk == 64 ? 4 : 3;                   // CTAs of an SM
    auto level = [](long long per_sm) { return per_sm < 2 ? (double)per_sm : 1.2 + 0.3 * (per_sm - 2); };
    auto load = [&](long long ctas) {
        return (double)(ctas / (148 * resident)) * level(resident) + level((ctas % (148 * resident) + 147) / 148);
    };
    double best = 0.95 * seqlen * load(walks);
    for (int s = 3; s <= 64; ++s) {
        const long long part = ((long long)seqlen + s - 1) / s, tokens = (part + unit - 1) / unit * unit;
        if (tokens * (s - 1) >= seqlen) continue;            // the last would be empty
        const double cost = 30 + (dk == 64 ? 4 : 10) * (s - 2) +
            (double)tokens * (load(walks * (s - 1) + units * (s - 2)) + load(walks * (s - 1)));
        if (cost < best) {
            best = cost;
            x.count = s;
            x.tokens = (int)tokens;
        }
    }
    return x;
}
static size_t starts_bytes(const DeltaSegments &x, int batch, int heads, int dk, int dv) {
    return x.count > 1 ? (size_t)(x.count - 1) * batch * heads * dk * dv * 4 : 0;
}
static size_t units_bytes(const DeltaSegments &x, int batch, int heads, int dk) {
    return x.count > 1 ? (size_t)(x.count - 2) * batch * heads * dk * dk * 4 : 0;
}

size_t delta_walk_workspace(int batch, int heads, int seqlen, int dk, int dv) {
    const DeltaSegments x = walk_segments(batch, heads, seqlen, dk, dv, 1, false);
    return starts_bytes(x, batch, heads, dk, dv) + units_bytes(x, batch, heads, dk);
}

static cudaError_t walk_pass(const DeltaArgs &a, const DeltaSegments &x, int last, cudaStream_t stream) {
    const int bhs = a.batch * a.heads, walks = (int)walk_ctas(a);
    const int ctas = walks * (x.count - 1) + (last ? 0 : bhs * (a.dk / kWalkSlab) * (x.count - 2));
    KernelTimer timer("delta_walk_segments", stream);
    count_launch();
    return a.dk == 64 ? launch_walk_segments<64>(a, x, ctas, last, stream)
                      : launch_walk_segments<128>(a, x, ctas, last, stream);
}

cudaError_t launch_delta_walk_segments(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    DeltaSegments x = walk_segments(a.batch, a.heads, a.seqlen, a.dk, a.dv, 1, false);
    if (x.count == 1) return launch_delta_walk(a, stream);
    x.starts = (float *)workspace;
    x.units = (float *)((char *)workspace + starts_bytes(x, a.batch, a.heads, a.dk, a.dv));
    cudaError_t e = walk_pass(a, x, 0, stream);
    if (e != cudaSuccess) return e;
    e = launch_delta_join(x.starts, nullptr, x.units, a.batch * a.heads, a.dk, a.dv, x.count - 2, stream);
    return e != cudaSuccess ? e : walk_pass(a, x, 1, stream);
}

static cudaError_t sweep_pass(const DeltaArgs &a, const DeltaSweepOut &o, const DeltaSegments &x,
                              int last, cudaStream_t stream) {
    const int bhs = a.batch * a.heads, walks = (int)walk_ctas(a);
    const int ctas = 2 * walks * (x.count - 1) + (last ? 0 : bhs * (a.dk / kWalkSlab) * (x.count - 2));
    KernelTimer timer("delta_sweeps_segments", stream);
    count_launch();
    if (a.dtype == RETNET_BF16)
        return a.dk == 64 ? launch_sweeps_segments<__nv_bfloat16, 64>(a, o, x, ctas, last, stream)
                          : launch_sweeps_segments<__nv_bfloat16, 128>(a, o, x, ctas, last, stream);
    return a.dk == 64 ? launch_sweeps_segments<float, 64>(a, o, x, ctas, last, stream)
                      : launch_sweeps_segments<float, 128>(a, o, x, ctas, last, stream);
}

static cudaError_t sweep_segments(const DeltaArgs &a, const DeltaSweepOut &o, const DeltaSegments &x,
                                  cudaStream_t stream) {
    cudaError_t e = sweep_pass(a, o, x, 0, stream);
    if (e != cudaSuccess) return e;
    e = launch_delta_join(x.starts, x.back, x.units, a.batch * a.heads, a.dk, a.dv, x.count - 2, stream);
    return e != cudaSuccess ? e : sweep_pass(a, o, x, 1, stream);
}

static size_t up1k(size_t x) { return (x + 1023) & ~(size_t)1023; }

struct DeltaGradLayout {
    size_t x, r, s, d, dq, dk, starts, back, units, total;
    DeltaSegments segments;
};
static DeltaGradLayout grad_layout(int batch, int heads, int key_heads, int seqlen, int dk, int dv) {
    const size_t rows = (size_t)batch * seqlen * heads;
    const size_t nc = ((size_t)seqlen + kDeltaChunk - 1) / kDeltaChunk;
    const size_t rv = up1k(rows * dv * 4), rk = heads != key_heads ? up1k(rows * dk * 4) : 0;
    const size_t st = up1k((size_t)batch * heads * nc * dk * dv * 4);
    DeltaGradLayout l;
    l.x = 0;
    l.r = l.x + rv;
    l.s = l.r + rv;
    l.d = l.s + st;
    l.dq = l.d + st;
    l.dk = l.dq + rk;
    l.segments = walk_segments(batch, heads, seqlen, dk, dv, kDeltaChunk, true);
    l.starts = l.dk + rk;
    l.back = l.starts + starts_bytes(l.segments, batch, heads, dk, dv);
    l.units = l.back + starts_bytes(l.segments, batch, heads, dk, dv);
    l.total = l.units + units_bytes(l.segments, batch, heads, dk);
    return l;
}

size_t delta_backward_simt_workspace(int batch, int heads, int key_heads, int seqlen, int dk,
                                     int dv) {
    return grad_layout(batch, heads, key_heads, seqlen, dk, dv).total;
}

template <typename T>
static cudaError_t launch_grad(const DeltaArgs &a, const DeltaGradLayout &l, char *ws,
                               cudaStream_t stream) {
    const long long nc = (a.seqlen + kDeltaChunk - 1) / kDeltaChunk;
    cudaError_t e = cudaFuncSetAttribute(delta_grad_kernel<T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DeltaGradSmem));
    if (e != cudaSuccess) return e;
    {
        KernelTimer timer("delta_grad", stream);
        count_launch();
        e = launch_overlapped(
            delta_grad_kernel<T>, dim3((unsigned)(nc * a.batch * a.heads)), dim3(kGradThreads),
            sizeof(DeltaGradSmem), stream, (const T *)a.q, (const T *)a.k, (const T *)a.d_out,
            (const T *)a.g, (const T *)a.beta, a.lengths, (const float *)(ws + l.x),
            (const float *)(ws + l.r), (const float *)(ws + l.s), (const float *)(ws + l.d),
            (T *)a.dq, (T *)a.dk_grad, (T *)a.dv_grad, (T *)a.dg, (T *)a.dbeta,
            (float *)(ws + l.dq), (float *)(ws + l.dk), a.scale, a.heads, a.key_heads, a.seqlen,
            a.dk, a.dv);
        if (e != cudaSuccess) return e;
    }
    return launch_delta_share(a, (const float *)(ws + l.dq), (const float *)(ws + l.dk), stream);
}

cudaError_t launch_delta_share(const DeltaArgs &a, const float *dq_wide, const float *dk_wide,
                               cudaStream_t stream) {
    if (a.heads == a.key_heads) return cudaSuccess;
    const long long vecs = (long long)a.batch * a.seqlen * a.key_heads * a.dk / 4;
    const dim3 grid((unsigned)((vecs + 255) / 256), 2);
    KernelTimer timer("delta_share", stream);
    count_launch();
    if (a.dtype == RETNET_BF16)
        return launch_overlapped(delta_share_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream,
                                 dq_wide, dk_wide, (__nv_bfloat16 *)a.dq,
                                 (__nv_bfloat16 *)a.dk_grad, vecs, a.heads / a.key_heads, a.dk);
    return launch_overlapped(delta_share_kernel<float>, grid, dim3(256), 0, stream, dq_wide,
                             dk_wide, (float *)a.dq, (float *)a.dk_grad, vecs,
                             a.heads / a.key_heads, a.dk);
}

cudaError_t launch_delta_backward_simt(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    const DeltaGradLayout l = grad_layout(a.batch, a.heads, a.key_heads, a.seqlen, a.dk, a.dv);
    char *ws = (char *)workspace;
    const DeltaSweepOut o = {(float *)(ws + l.x), (float *)(ws + l.s), (float *)(ws + l.r), (float *)(ws + l.d)};
    DeltaSegments x = l.segments;
    x.starts = (float *)(ws + l.starts);
    x.back = (float *)(ws + l.back);
    x.units = (float *)(ws + l.units);
    cudaError_t e = x.count > 1 ? sweep_segments(a, o, x, stream) : sweep(a, o, stream);
    if (e != cudaSuccess) return e;
    return a.dtype == RETNET_BF16 ? launch_grad<__nv_bfloat16>(a, l, ws, stream)
                                  : launch_grad<float>(a, l, ws, stream);
}

}  // namespace retnet
