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
// Every row is read once and written once: an HBM stream of 5 tensors
// forward (x, y, g; h, n) and 8 backward (x, y, g, dh, dn; dx, dy, dg).  A
// row stays in the registers of the threads that own it (two vectors of 8
// channels each at most), so the two (three) sums over the row cost
// shuffles and one barrier each and nothing is read twice; h is formed from
// x, y and g again in the backward, which reads no more than a stored h would.
#include "kernels.h"

namespace retnet {

constexpr int kNormVecs = 2;               // vectors of 8 channels per thread
constexpr int kNormWarpRows = 4;           // rows per CTA where a warp owns a row

struct NormArgs {
    const void *x, *y, *gate, *dh, *dn;
    void *h, *n, *dx, *dy, *dgate;
    const float *post, *pre;
    float *part_post, *part_pre;           // [grid rows][hidden] partial sums, or null
    float scale, eps;
    long long rows;
    int hidden, post_norm;
};

// Sum over the TPR threads that own a row; every one of them gets it.
// `red` is this call's own slot, so calls need no barrier between them.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*red)[N]) {
#pragma unroll
    for (int m = 16; m; m >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[threadIdx.x >> 5][i] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) a += red[w][i];
            s[i] = a;
        }
    }
}

// The fast exponential and quotient (a few 2^-22 relative, and 0 where the
// exponential overflows): with the exact ones the arithmetic of a gated row
// takes about as long as its traffic.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <typename T, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarpRows : TPR)
residual_norm_kernel(NormArgs a) {
    constexpr int kRows = TPR == 32 ? kNormWarpRows : 1;
    __shared__ float red[2][TPR / 32][1];
    const int lane = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long long row = (long long)blockIdx.x * kRows + (TPR == 32 ? threadIdx.x >> 5 : 0);
    grid_dependency_wait();
    if (row >= a.rows) return;             // a whole warp, or no thread of a CTA
    const size_t base = (size_t)row * a.hidden;
    const T *x = (const T *)a.x + base, *y = (const T *)a.y + base;
    const T *g = a.gate ? (const T *)a.gate + base : nullptr;
    const int vecs = a.hidden / 8;

    float xv[kNormVecs][8], yv[kNormVecs][8], gv[kNormVecs][8];
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            load8(y + c * 8, yv[i]);
            load8(x + c * 8, xv[i]);
            if (g) load8(g + c * 8, gv[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) xv[i][e] = yv[i][e] = gv[i][e] = 0.f;
        }
    }
    float ry = 1.f;
    if (a.post_norm) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] = fmaf(yv[i][e], yv[i][e], s[0]);
        row_sum<TPR>(s, red[0]);
        ry = rsqrtf(s[0] / (float)a.hidden + a.eps);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            float w[8];
            if (a.post_norm && a.post) load8(a.post + c * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float z = yv[i][e] * ry;
                if (a.post_norm && a.post) z *= w[e];
                if (g) z *= gv[i][e] * sigmoid(gv[i][e]);
                xv[i][e] = fmaf(a.scale, z, xv[i][e]);
                s[0] = fmaf(xv[i][e], xv[i][e], s[0]);
            }
        }
    }
    row_sum<TPR>(s, red[1]);
    const float rh = rsqrtf(s[0] / (float)a.hidden + a.eps);
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            store8((T *)a.h + base + c * 8, xv[i]);
            float w[8];
            if (a.pre) load8(a.pre + c * 8, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) xv[i][e] *= a.pre ? rh * w[e] : rh;
            store8((T *)a.n + base + c * 8, xv[i]);
        }
    }
}

// A CTA takes rows blockIdx.x, + gridDim.x, ... and keeps the weights'
// gradients of its channels in registers until the end, so they cost one
// partial row a CTA instead of an atomic a channel and row, and their order
// does not change from run to run.
template <typename T, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarpRows : TPR)
residual_norm_backward_kernel(NormArgs a) {
    constexpr int kRows = TPR == 32 ? kNormWarpRows : 1;
    __shared__ float red1[2][TPR / 32][1], red2[2][TPR / 32][2], red3[2][TPR / 32][1];
    const int lane = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long long first = (long long)blockIdx.x * kRows + (TPR == 32 ? threadIdx.x >> 5 : 0);
    const int vecs = a.hidden / 8;
    const bool gated = a.gate != nullptr, weighted = a.post_norm && a.post;
    const float inv = 1.f / (float)a.hidden;
    float apost[kNormVecs][8] = {}, apre[kNormVecs][8] = {};
    grid_dependency_wait();

    int turn = 0;                          // alternating slots of the sums
    for (long long row = first; row < a.rows; row += (long long)gridDim.x * kRows, turn ^= 1) {
        const size_t base = (size_t)row * a.hidden;
        float xv[kNormVecs][8], yv[kNormVecs][8], gv[kNormVecs][8], tv[kNormVecs][8];
        float dv[kNormVecs][8];
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                const size_t o = base + c * 8;
                load8((const T *)a.y + o, yv[i]);
                load8((const T *)a.x + o, xv[i]);
                if (gated) load8((const T *)a.gate + o, gv[i]);
                load8((const T *)a.dn + o, tv[i]);
                if (a.dh) load8((const T *)a.dh + o, dv[i]);
            }
        }
        float ry = 1.f;
        if (a.post_norm) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < kNormVecs; ++i)
                if (lane + i * TPR < vecs)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[0] = fmaf(yv[i][e], yv[i][e], s[0]);
            row_sum<TPR>(s, red1[turn]);
            ry = rsqrtf(s[0] * inv + a.eps);
        }
        // h, and the sums of h^2 and (dn pre) h
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                float w[8], p[8];
                if (weighted) load8(a.post + c * 8, w);
                if (a.pre) load8(a.pre + c * 8, p);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    yv[i][e] *= ry;                       // y^
                    float z = weighted ? yv[i][e] * w[e] : yv[i][e];
                    if (gated) z *= gv[i][e] * sigmoid(gv[i][e]);
                    xv[i][e] = fmaf(a.scale, z, xv[i][e]);
                    const float t = a.pre ? tv[i][e] * p[e] : tv[i][e];
                    s2[0] = fmaf(xv[i][e], xv[i][e], s2[0]);
                    s2[1] = fmaf(t, xv[i][e], s2[1]);
                }
            }
        }
        row_sum<TPR>(s2, red2[turn]);
        const float rh = rsqrtf(s2[0] * inv + a.eps);
        const float mh = s2[1] * rh * inv;                // mean(t h^)
        float s3[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                float w[8], p[8];
                if (weighted) load8(a.post + c * 8, w);
                if (a.pre) load8(a.pre + c * 8, p);
                float dg[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float hh = xv[i][e] * rh;       // h^
                    apre[i][e] = fmaf(tv[i][e], hh, apre[i][e]);
                    const float t = a.pre ? tv[i][e] * p[e] : tv[i][e];
                    float d = rh * (t - hh * mh);
                    if (a.dh) d += dv[i][e];
                    dv[i][e] = d;                         // dx
                    float dz = a.scale * d;
                    if (gated) {
                        const float sg = sigmoid(gv[i][e]), sw = gv[i][e] * sg;
                        const float z = weighted ? yv[i][e] * w[e] : yv[i][e];
                        dg[e] = dz * z * fmaf(sw, 1.f - sg, sg);
                        dz *= sw;
                    }
                    apost[i][e] = fmaf(dz, yv[i][e], apost[i][e]);
                    const float u = weighted ? dz * w[e] : dz;
                    tv[i][e] = u;
                    s3[0] = fmaf(u, yv[i][e], s3[0]);
                }
                store8((T *)a.dx + base + c * 8, dv[i]);
                if (gated) store8((T *)a.dgate + base + c * 8, dg);
            }
        }
        float my = 0.f;
        if (a.post_norm) {
            row_sum<TPR>(s3, red3[turn]);
            my = s3[0] * inv;                             // mean(u y^)
        }
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = a.post_norm ? ry * (tv[i][e] - yv[i][e] * my) : tv[i][e];
                store8((T *)a.dy + base + c * 8, o);
            }
        }
    }
    // this CTA's (this warp's) partial sums over its rows
    const long long part = first;          // < gridDim.x * kRows
#pragma unroll
    for (int i = 0; i < kNormVecs; ++i) {
        const int c = lane + i * TPR;
        if (c < vecs) {
            if (a.part_post) store8(a.part_post + (size_t)part * a.hidden + c * 8, apost[i]);
            if (a.part_pre) store8(a.part_pre + (size_t)part * a.hidden + c * 8, apre[i]);
        }
    }
}

// out[c] = sum of `parts` partial rows, in a fixed order.
constexpr int kSumCols = 32, kSumLanes = 16;
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
#pragma unroll 4
        for (int p = r; p < parts; p += kSumLanes) s += part[(size_t)p * hidden + c];
    red[r][threadIdx.x % kSumCols] = s;
    __syncthreads();
    if (r == 0 && c < hidden) {
#pragma unroll
        for (int i = 1; i < kSumLanes; ++i) s += red[i][threadIdx.x % kSumCols];
        out[c] = s;
    }
}

// Threads per row: two vectors of 8 channels a thread at most.
static int norm_threads(int hidden) {
    if (hidden <= 512) return 32;
    if (hidden <= 2048) return 128;
    if (hidden <= 4096) return 256;
    return hidden <= 8192 ? 512 : 1024;
}

// CTAs of the backward: as many as are resident on 148 SMs at 64 registers a
// thread, and no more than there are rows for.
static long long norm_backward_grid(long long rows, int hidden) {
    const int tpr = norm_threads(hidden);
    const int per_cta = tpr == 32 ? kNormWarpRows : 1;
    const int threads = tpr == 32 ? 32 * kNormWarpRows : tpr;
    const long long resident = 148ll * (1024 / threads);
    const long long want = (rows + per_cta - 1) / per_cta;
    return want < resident ? want : resident;
}

size_t residual_norm_backward_workspace(long long rows, int hidden) {
    const int per_cta = norm_threads(hidden) == 32 ? kNormWarpRows : 1;
    return (size_t)norm_backward_grid(rows, hidden) * per_cta * hidden * 2 * sizeof(float);
}

template <typename T>
static cudaError_t launch_forward(const NormArgs &a, cudaStream_t stream) {
    const int tpr = norm_threads(a.hidden);
    const long long grid = tpr == 32 ? (a.rows + kNormWarpRows - 1) / kNormWarpRows : a.rows;
    const dim3 g((unsigned)grid), b(tpr == 32 ? 32 * kNormWarpRows : tpr);
    switch (tpr) {
        case 32: return launch_overlapped(residual_norm_kernel<T, 32>, g, b, 0, stream, a);
        case 128: return launch_overlapped(residual_norm_kernel<T, 128>, g, b, 0, stream, a);
        case 256: return launch_overlapped(residual_norm_kernel<T, 256>, g, b, 0, stream, a);
        case 512: return launch_overlapped(residual_norm_kernel<T, 512>, g, b, 0, stream, a);
    }
    return launch_overlapped(residual_norm_kernel<T, 1024>, g, b, 0, stream, a);
}

template <typename T>
static cudaError_t launch_backward(const NormArgs &a, unsigned grid, cudaStream_t stream) {
    const int tpr = norm_threads(a.hidden);
    const dim3 g(grid), b(tpr == 32 ? 32 * kNormWarpRows : tpr);
    switch (tpr) {
        case 32: return launch_overlapped(residual_norm_backward_kernel<T, 32>, g, b, 0, stream, a);
        case 128: return launch_overlapped(residual_norm_backward_kernel<T, 128>, g, b, 0, stream, a);
        case 256: return launch_overlapped(residual_norm_backward_kernel<T, 256>, g, b, 0, stream, a);
        case 512: return launch_overlapped(residual_norm_backward_kernel<T, 512>, g, b, 0, stream, a);
    }
    return launch_overlapped(residual_norm_backward_kernel<T, 1024>, g, b, 0, stream, a);
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
    const long long grid = norm_backward_grid(rows, hidden);
    const int parts = (int)grid * (norm_threads(hidden) == 32 ? kNormWarpRows : 1);
    float *part_post = (float *)workspace;
    float *part_pre = part_post + (size_t)parts * hidden;
    if (rows > 0) {
        NormArgs a = norm_args(p, rows, hidden);
        a.x = x; a.y = y; a.dn = dn; a.dh = dh; a.dx = dx; a.dy = dy; a.dgate = dgate;
        a.part_post = dpost ? part_post : nullptr;
        a.part_pre = dpre ? part_pre : nullptr;
        KernelTimer timer("residual_norm_backward", stream);
        count_launch();
        cudaError_t e = dtype == RETNET_BF16
                            ? launch_backward<__nv_bfloat16>(a, (unsigned)grid, stream)
                            : launch_backward<float>(a, (unsigned)grid, stream);
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
