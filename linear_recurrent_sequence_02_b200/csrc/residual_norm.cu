// The norms before and after a block, its gate and the residual, in one pass.
//
// For a residual row x, a block's output y and a gate g (hidden channels):
//   z = rms(y) * post            rms(a) = a / sqrt(mean(a^2) + eps)
//   h = x + s swish(g) z         the residual stream
//   n = rms(h) * pre             the next block's input
// and for dh, dn (the gradients of h and n), with a^ = rms(a):
//   dx  = dh + r_h (t - h^ mean(t h^)),  t = dn pre,       dpre  = sum_rows dn h^
//   dg  = s dx z swish'(g),  dz = s dx swish(g),           dpost = sum_rows dz y^
//   dy  = r_y (u - y^ mean(u y^)),       u = dz post.
// Every row comes from HBM once and is written once: a stream of 5 tensors
// forward (x, y, g; h, n) and 8 backward (x, y, g, dh, dn; dx, dy, dg); h is
// formed from x, y and g again in the backward, which reads no more than a
// stored h would.
// Forward a row stays in the registers of the threads that own it (up to 4
// vectors of 8 channels each), so that nothing is read twice and its two sums
// cost shuffles and one barrier each.  Backward a thread owns up to 2 vectors
// and keeps h; the other tensors are read again in each of the three passes
// over the row (y in up to four, dn and g in two), from the copies in shared
// memory or, where there are none (float32, and bf16 above 8192 channels),
// through L1 and L2.  Its sums share two barriers a row: h^2 with t h, and u y^
// with the next row's y^2.
#include "kernels.h"
#include "pairs.cuh"

namespace retnet {

constexpr int kNormWarpRows = 8;           // rows per CTA where a warp owns a row

struct NormArgs {
    const void *x, *y, *gate, *dh, *dn;
    void *h, *n, *dx, *dy, *dgate;
    const float *post, *pre;
    float *part_post, *part_pre;           // [grid rows][hidden] partial sums, or null
    float scale, eps;
    long long rows;
    int hidden, post_norm;
};

// Sums over the TPR threads that own a row; every one of them gets them.
// `red` is this call's own slot, so calls need no barrier between them.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*red)[TPR / 32]) {
    constexpr int W = TPR / 32;
#pragma unroll
    for (int m = 16; m; m >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
    if (W > 1) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[i][threadIdx.x >> 5] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a = 0.f;
            if constexpr (W % 4 == 0) {
#pragma unroll
                for (int w = 0; w < W; w += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(&red[i][w]);
                    a += (v.x + v.y) + (v.z + v.w);
                }
            } else {
#pragma unroll
                for (int w = 0; w < W; ++w) a += red[i][w];
            }
            s[i] = a;
        }
    }
}

// The fast exponential and reciprocal (a few 2^-22 relative, and 0 where the
// exponential overflows): with the exact ones the arithmetic of a gated row
// takes longer than its traffic.
__device__ __forceinline__ float sigmoid(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-x)));
    return r;
}

// 8 channels as they lie in memory: rows stay packed until they are used, or
// a row's registers would leave too few warps to hide its loads.
template <typename T>
struct Packed;
template <>
struct Packed<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    // 16-byte pieces `stride` apart
    __device__ __forceinline__ void load(const uint8_t *p, int) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float2 at(int e) const {    // channels 2 e, 2 e + 1
        const uint32_t w = e == 0 ? u.x : e == 1 ? u.y : e == 2 ? u.z : u.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <>
struct Packed<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void load(const uint8_t *p, int stride) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + stride);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float2 at(int e) const {
        const float4 &v = e < 2 ? a : b;
        return e & 1 ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
    }
};
__device__ __forceinline__ void store8(float *p, const float2 (&v)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float2 (&v)[4]) {
    uint4 u;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(v[i]);
    *reinterpret_cast<uint4 *>(p) = u;
}
// A weight's 8 channels (1 where there is none).
__device__ __forceinline__ void load_weight(const float *w, int c, float2 (&o)[4]) {
    if (w) {
        const float4 *p = reinterpret_cast<const float4 *>(w + c * 8);
        const float4 a = p[0], b = p[1];
        o[0] = make_float2(a.x, a.y); o[1] = make_float2(a.z, a.w);
        o[2] = make_float2(b.x, b.y); o[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = make_float2(1.f, 1.f);
    }
}
__device__ __forceinline__ float2 sigmoid2(float2 x) { return make_float2(sigmoid(x.x), sigmoid(x.y)); }

template <typename T, int TPR, int kVecs>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarpRows : TPR)
residual_norm_kernel(NormArgs a) {
    constexpr int kRows = TPR == 32 ? kNormWarpRows : 1;
    __shared__ __align__(16) float red[2][1][TPR / 32];
    const int lane = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long long row = (long long)blockIdx.x * kRows + (TPR == 32 ? threadIdx.x >> 5 : 0);
    grid_dependency_wait();
    if (row >= a.rows) return;             // a whole warp, or no thread of a CTA
    const size_t base = (size_t)row * a.hidden;
    const bool gated = a.gate != nullptr;
    const int vecs = a.hidden / 8;

    Packed<T> xp[kVecs], yp[kVecs], gp[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            yp[i].load((const T *)a.y + base + c * 8);
            xp[i].load((const T *)a.x + base + c * 8);
            if (gated) gp[i].load((const T *)a.gate + base + c * 8);
        } else {
            yp[i].zero();
            xp[i].zero();
            gp[i].zero();
        }
    }
    float ry = 1.f;
    if (a.post_norm) {
        float2 q = both(0.f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) q = fma2(yp[i].at(e), yp[i].at(e), q);
        float s[1] = {q.x + q.y};
        row_sum<TPR>(s, red[0]);
        ry = rsqrtf(s[0] / (float)a.hidden + a.eps);
    }
    float2 q = both(0.f), h[kVecs][4];
    const float *post = a.post_norm ? a.post : nullptr;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            float2 w[4];
            load_weight(post, c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 z = mul2(mul2(yp[i].at(e), both(ry)), w[e]);
                if (gated) z = mul2(z, mul2(gp[i].at(e), sigmoid2(gp[i].at(e))));
                h[i][e] = fma2(both(a.scale), z, xp[i].at(e));
                q = fma2(h[i][e], h[i][e], q);
            }
            store8((T *)a.h + base + c * 8, h[i]);
        }
    }
    float s[1] = {q.x + q.y};
    row_sum<TPR>(s, red[1]);
    const float rh = rsqrtf(s[0] / (float)a.hidden + a.eps);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            float2 w[4];
            load_weight(a.pre, c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[i][e] = mul2(h[i][e], mul2(both(rh), w[e]));
            store8((T *)a.n + base + c * 8, h[i]);
        }
    }
}

// A CTA takes rows blockIdx.x, + gridDim.x, ... and keeps the weights'
// gradients of its channels in registers until the end, so they cost one
// partial row a CTA instead of an atomic a channel and row, and their order
// does not change from run to run.  With kAhead every thread copies its
// vectors of the next row to shared memory while it works on this one (8192 x
// 4096 bf16: 163 us without, 126 with), and reads them again in each pass
// instead of holding them; without they come from global memory as they are
// needed.  A row costs two barriers: the next row's sum of y^2 shares the last.
template <typename T, int TPR, int kVecs, bool kAhead>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarpRows : TPR, TPR <= 256 ? 512 / (TPR == 32 ? 256 : TPR) : 1)
residual_norm_backward_kernel(NormArgs a) {
    enum { kX, kY, kGate, kDn, kDh, kTensors };
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kVecBytes = 8 * sizeof(T), kThreads = TPR == 32 ? 32 * kNormWarpRows : TPR;
    constexpr int kRows = TPR == 32 ? kNormWarpRows : 1;
    __shared__ __align__(16) float red1[2][2][TPR / 32], red2[2][2][TPR / 32];
    const int lane = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long long first = (long long)blockIdx.x * kRows + (TPR == 32 ? threadIdx.x >> 5 : 0);
    const int vecs = a.hidden / 8;
    const bool gated = a.gate != nullptr;
    const float *post = a.post_norm ? a.post : nullptr;
    const float inv = 1.f / (float)a.hidden;
    float2 apost[kVecs][4] = {}, apre[kVecs][4] = {};
    grid_dependency_wait();

    const T *from[kTensors] = {(const T *)a.x, (const T *)a.y, (const T *)a.gate, (const T *)a.dn,
                               (const T *)a.dh};
    const long long step = (long long)gridDim.x * kRows;
    // this thread's vector i of a tensor in slot `turn`; 16-byte pieces of the
    // CTA's threads side by side
    auto place = [&](int turn, int t, int i, int half) {
        return smem + ((((turn * kTensors + t) * kVecs + i) * (kVecBytes / 16) + half) * kThreads + threadIdx.x) * 16;
    };
    auto fetch = [&](long long row, int turn) {
        if (kAhead && row < a.rows)
#pragma unroll
            for (int t = 0; t < kTensors; ++t)
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (from[t] && lane + i * TPR < vecs)
#pragma unroll
                        for (int half = 0; half < kVecBytes / 16; ++half)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                             (uint32_t)__cvta_generic_to_shared(place(turn, t, i, half))),
                                         "l"((const char *)(from[t] + (size_t)row * a.hidden + (lane + i * TPR) * 8) + 16 * half)
                                         : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load = [&](long long row, int turn, int t, int i) {
        Packed<T> v;
        if (kAhead) v.load(place(turn, t, i, 0), 16 * kThreads);
        else v.load(from[t] + (size_t)row * a.hidden + (lane + i * TPR) * 8);
        return v;
    };
    // this thread's part of the sum of y^2
    auto squares = [&](long long row, int turn) {
        float2 q = both(0.f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (lane + i * TPR < vecs) {
                const Packed<T> y = load(row, turn, kY, i);
#pragma unroll
                for (int e = 0; e < 4; ++e) q = fma2(y.at(e), y.at(e), q);
            }
        return q.x + q.y;
    };
    int turn = 0;                          // alternating slots
    float ry = 1.f;
    fetch(first, 0);
    if (a.post_norm && first < a.rows) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        float s[1] = {squares(first, 0)};
        row_sum<TPR>(s, red2[1]);          // the first row's own sums go to the other slot
        ry = rsqrtf(s[0] * inv + a.eps);
    }
    for (long long row = first; row < a.rows; row += step, turn ^= 1) {
        const size_t base = (size_t)row * a.hidden;
        fetch(row + step, turn ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        auto get = [&](int t, int i) { return load(row, turn, t, i); };
        // h, and the sums of h^2 and (dn pre) h
        float2 q0 = both(0.f), q1 = q0, h[kVecs][4], sg[kVecs][4];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                float2 w[4], p[4];
                load_weight(post, c, w);
                load_weight(a.pre, c, p);
                const Packed<T> x = get(kX, i), y = get(kY, i), dn = get(kDn, i);
                Packed<T> g;
                if (gated) g = get(kGate, i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 z = mul2(mul2(y.at(e), both(ry)), w[e]);
                    if (gated) {
                        sg[i][e] = sigmoid2(g.at(e));
                        z = mul2(z, mul2(g.at(e), sg[i][e]));
                    }
                    h[i][e] = fma2(both(a.scale), z, x.at(e));
                    q0 = fma2(h[i][e], h[i][e], q0);
                    q1 = fma2(mul2(dn.at(e), p[e]), h[i][e], q1);
                }
            }
        }
        float s2[2] = {q0.x + q0.y, q1.x + q1.y};
        row_sum<TPR>(s2, red1[turn]);
        const float rh = rsqrtf(s2[0] * inv + a.eps);
        const float mh = s2[1] * rh * inv;                // mean(t h^)
        float2 q3 = both(0.f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                float2 w[4], p[4], dg[4], dx[4];
                load_weight(post, c, w);
                load_weight(a.pre, c, p);
                const Packed<T> y = get(kY, i), dn = get(kDn, i);
                Packed<T> g, dh;
                if (gated) g = get(kGate, i);
                if (a.dh) dh = get(kDh, i);
                else dh.zero();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 hh = mul2(h[i][e], both(rh));     // h^
                    const float2 yh = mul2(y.at(e), both(ry));     // y^
                    apre[i][e] = fma2(dn.at(e), hh, apre[i][e]);
                    dx[e] = fma2(both(rh), fma2(hh, both(-mh), mul2(dn.at(e), p[e])), dh.at(e));
                    float2 dz = mul2(both(a.scale), dx[e]);
                    if (gated) {
                        const float2 sw = mul2(g.at(e), sg[i][e]);
                        // swish' = sg + sw (1 - sg)
                        const float2 ds = add2(fma2(sw, mul2(sg[i][e], both(-1.f)), sw), sg[i][e]);
                        dg[e] = mul2(mul2(dz, mul2(yh, w[e])), ds);
                        dz = mul2(dz, sw);
                    }
                    apost[i][e] = fma2(dz, yh, apost[i][e]);
                    h[i][e] = mul2(dz, w[e]);                      // u
                    q3 = fma2(h[i][e], yh, q3);
                }
                store8((T *)a.dx + base + c * 8, dx);
                if (gated) store8((T *)a.dgate + base + c * 8, dg);
            }
        }
        float my = 0.f, ry_next = 1.f;
        if (a.post_norm) {                                // with the next row's sum of y^2
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            float s3[2] = {q3.x + q3.y, row + step < a.rows ? squares(row + step, turn ^ 1) : 0.f};
            row_sum<TPR>(s3, red2[turn]);
            my = s3[0] * inv;                             // mean(u y^)
            ry_next = rsqrtf(s3[1] * inv + a.eps);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                if (a.post_norm) {
                    const Packed<T> y = get(kY, i);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        h[i][e] = mul2(both(ry), fma2(y.at(e), both(-ry * my), h[i][e]));
                }
                store8((T *)a.dy + base + c * 8, h[i]);
            }
        }
        ry = ry_next;
    }
    // this CTA's (this warp's) partial sums over its rows
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            if (a.part_post) store8(a.part_post + (size_t)first * a.hidden + c * 8, apost[i]);
            if (a.part_pre) store8(a.part_pre + (size_t)first * a.hidden + c * 8, apre[i]);
        }
    }
}

// out[c] = sum of `parts` partial rows, in a fixed order.
constexpr int kSumCols = 32, kSumLanes = 32;
__global__ void __launch_bounds__(kSumCols *kSumLanes)
norm_weight_sum_kernel(const float *part_post, const float *part_pre, float *dpost, float *dpre,
                       int parts, int hidden) {
    __shared__ float red[kSumLanes][kSumCols + 1];
    const float *part = blockIdx.y ? part_pre : part_post;
    float *out = blockIdx.y ? dpre : dpost;
    const int c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    grid_dependency_wait();
    if (!out) return;
    float s = 0.f;
    if (c < hidden)
#pragma unroll 8
        for (int p = r; p < parts; p += kSumLanes) s += part[(size_t)p * hidden + c];
    red[r][threadIdx.x % kSumCols] = s;
    __syncthreads();
    if (r == 0 && c < hidden) {
#pragma unroll
        for (int i = 1; i < kSumLanes; ++i) s += red[i][threadIdx.x % kSumCols];
        out[c] = s;
    }
}

// Threads per row, each with up to `vecs` vectors of 8 channels.
static int norm_threads(int hidden, int vecs) {
    int t = 32;
    while (t < 1024 && hidden > 8 * vecs * t) t *= 2;
    return t;
}
static int rows_per_cta(int tpr) { return tpr == 32 ? kNormWarpRows : 1; }
constexpr int kForwardVecs = 4;
// Of the backward: two, but one for shorter float32 rows (16384 x 512: 60 us
// against 66; 4096 x 2048: 67 against 61).
static int backward_vecs(int hidden, int size) { return size == 4 && hidden < 2048 ? 1 : 2; }
// Shared memory of the backward: two rows of five tensors.  Float32 rows come
// from global memory as they are needed: copied ahead they leave an SM one or
// two CTAs (8192 x 4096: 345 us ahead, 230 so; bf16: 126 ahead, 163 so).
constexpr int backward_bytes(int threads, int vecs, int size) { return 2 * 5 * vecs * 8 * size * threads; }
constexpr bool copies_ahead(int bytes, int size) { return size == 2 && bytes <= 220 * 1024; }

// CTAs of the backward: as many as registers and shared memory let reside on
// 148 SMs, and no more than there are rows for.
static long long norm_backward_grid(long long rows, int hidden, int size) {
    const int tpr = norm_threads(hidden, backward_vecs(hidden, size)), per_cta = rows_per_cta(tpr);
    const long long resident = 148ll * (tpr <= 256 ? 512 / (tpr * per_cta) : 1);
    const long long want = (rows + per_cta - 1) / per_cta;
    return want < resident ? want : resident;
}
static long long norm_backward_parts(long long rows, int hidden, int size) {
    return norm_backward_grid(rows, hidden, size) * rows_per_cta(norm_threads(hidden, backward_vecs(hidden, size)));
}
size_t residual_norm_backward_workspace(long long rows, int hidden) {
    const long long b = norm_backward_parts(rows, hidden, 2), f = norm_backward_parts(rows, hidden, 4);
    return (size_t)(b > f ? b : f) * hidden * 2 * sizeof(float);
}

template <typename T>
static cudaError_t launch_forward(const NormArgs &a, cudaStream_t stream) {
    constexpr int V = kForwardVecs;
    const int tpr = norm_threads(a.hidden, V), per_cta = rows_per_cta(tpr);
    const dim3 g((unsigned)((a.rows + per_cta - 1) / per_cta)), b(tpr * per_cta);
    switch (tpr) {
        case 32:                                            // no more registers than a short row needs
            if (a.hidden <= 256) return launch_overlapped(residual_norm_kernel<T, 32, 1>, g, b, 0, stream, a);
            if (a.hidden <= 512) return launch_overlapped(residual_norm_kernel<T, 32, 2>, g, b, 0, stream, a);
            return launch_overlapped(residual_norm_kernel<T, 32, V>, g, b, 0, stream, a);
        case 64: return launch_overlapped(residual_norm_kernel<T, 64, V>, g, b, 0, stream, a);
        case 128: return launch_overlapped(residual_norm_kernel<T, 128, V>, g, b, 0, stream, a);
        case 256: return launch_overlapped(residual_norm_kernel<T, 256, V>, g, b, 0, stream, a);
    }
    return launch_overlapped(residual_norm_kernel<T, 512, V>, g, b, 0, stream, a);
}

template <typename T, int TPR, int V>
static cudaError_t launch_backward_tpr(const NormArgs &a, unsigned grid, cudaStream_t stream) {
    constexpr int kThreads = TPR == 32 ? 32 * kNormWarpRows : TPR;
    constexpr int kBytes = backward_bytes(kThreads, V, (int)sizeof(T));
    constexpr bool kAhead = copies_ahead(kBytes, (int)sizeof(T));
    auto kernel = residual_norm_backward_kernel<T, TPR, V, kAhead>;
    if (kAhead) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
    }
    return launch_overlapped(kernel, dim3(grid), dim3(kThreads), kAhead ? kBytes : 0, stream, a);
}

template <typename T, int V>
static cudaError_t launch_backward(const NormArgs &a, unsigned grid, cudaStream_t stream) {
    switch (norm_threads(a.hidden, V)) {
        case 32: return launch_backward_tpr<T, 32, V>(a, grid, stream);
        case 64: return launch_backward_tpr<T, 64, V>(a, grid, stream);
        case 128: return launch_backward_tpr<T, 128, V>(a, grid, stream);
        case 256: return launch_backward_tpr<T, 256, V>(a, grid, stream);
    }
    if constexpr (V == 1) return cudaErrorInvalidValue;      // shorter rows only
    else return norm_threads(a.hidden, V) == 512 ? launch_backward_tpr<T, 512, V>(a, grid, stream)
                                                 : launch_backward_tpr<T, 1024, V>(a, grid, stream);
}

static NormArgs norm_args(const retnet_block_norm &p, long long rows, int hidden) {
    NormArgs a = {};
    a.gate = p.gate;
    a.post_norm = p.post_norm;
    a.post = p.post_weight;
    a.pre = p.pre_weight;
    a.scale = p.residual_scale;
    a.eps = p.eps;
    a.rows = rows;
    a.hidden = hidden;
    return a;
}

cudaError_t launch_residual_norm(const void *x, const void *y, const retnet_block_norm &p,
                                 long long rows, int hidden, retnet_dtype dtype, void *h, void *n,
                                 cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    NormArgs a = norm_args(p, rows, hidden);
    a.x = x; a.y = y; a.h = h; a.n = n;
    KernelTimer timer("residual_norm", stream);
    count_launch();
    return dtype == RETNET_BF16 ? launch_forward<__nv_bfloat16>(a, stream)
                                : launch_forward<float>(a, stream);
}

cudaError_t launch_residual_norm_backward(const void *x, const void *y, const void *dn,
                                          const void *dh, const retnet_block_norm &p,
                                          long long rows, int hidden, retnet_dtype dtype, void *dx,
                                          void *dy, void *dgate, float *dpost, float *dpre,
                                          void *workspace, cudaStream_t stream) {
    const int size = dtype == RETNET_BF16 ? 2 : 4;
    const long long grid = norm_backward_grid(rows, hidden, size);
    const int parts = (int)norm_backward_parts(rows, hidden, size);
    float *part_post = (float *)workspace;
    float *part_pre = part_post + (size_t)parts * hidden;
    if (rows > 0) {
        NormArgs a = norm_args(p, rows, hidden);
        a.x = x; a.y = y; a.dn = dn; a.dh = dh; a.dx = dx; a.dy = dy; a.dgate = dgate;
        a.part_post = dpost ? part_post : nullptr;
        a.part_pre = dpre ? part_pre : nullptr;
        KernelTimer timer("residual_norm_backward", stream);
        count_launch();
        cudaError_t e = dtype == RETNET_BF16 ? launch_backward<__nv_bfloat16, 2>(a, (unsigned)grid, stream)
                        : backward_vecs(hidden, 4) == 1 ? launch_backward<float, 1>(a, (unsigned)grid, stream)
                                                        : launch_backward<float, 2>(a, (unsigned)grid, stream);
        if (e != cudaSuccess) return e;
    }
    if (!dpost && !dpre) return cudaSuccess;
    KernelTimer timer("norm_weight_sum", stream);
    count_launch();
    const dim3 g((hidden + kSumCols - 1) / kSumCols, 2);
    return launch_overlapped(norm_weight_sum_kernel, g, dim3(kSumCols * kSumLanes), 0, stream,
                             (const float *)part_post, (const float *)part_pre, dpost, dpre,
                             parts, hidden);
}

}  // namespace retnet
