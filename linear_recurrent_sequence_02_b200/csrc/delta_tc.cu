// Gated delta rule on the tensor cores, in chunks of 64 tokens (bf16, dk 64
// or 128).
//
// Inside a chunk, with G the running sum of g, the tokens' x_t solve a unit
// lower triangular system, so that with the state S before the chunk
//   M_ij = b_i (k_i . k_j) e^{G_i - G_j}  (i > j),   T = (1 + M)^-1,
//   T^ = T diag(b),   W = T^ diag(e^G) K,   Q~ = scale diag(e^G) Q,
//   P_ij = scale (q_i . k_j) e^{G_i - G_j}  (i >= j):
//   X = T^ V - W S,   O = Q~ S + P X,   S <- e^{G_L} S + K^T diag(e^{G_L - G}) X.
// T^, W, Q~ and P do not depend on the state: delta_prep_kernel forms them
// for all chunks at once.  What remains is a walk over the chunks
// (delta_scan_kernel) of three products a chunk, of which the second needs
// the first and the next chunk's first the second.
//
// The walk keeps everything transposed, v channels as rows: a CTA owns 128
// columns of S (128 tensor-memory lanes), so that a thread owns one v
// channel of S, X and O, and what passes between products (S^T, X^T) is an
// A operand in tensor memory that the thread writes where it read its
// accumulator.  Nothing but the prepared tiles, K and V goes through shared
// memory, all of it by bulk copies one chunk ahead.
#include "delta.cuh"
#include "sm100.cuh"

namespace retnet {
namespace {

using namespace sm100;

constexpr int kC = kDeltaChunk;
constexpr uint32_t kBox64 = 8192;          // 64 rows x 64 bf16, 128-byte swizzled

// One chunk's prepared operands, in shared-memory order.  Every tile is
// boxes of 64 rows (tokens) of 64 columns, 128-byte swizzled.
// kSplit: T^ and W in two bf16 parts (16 bits together), which the final
// state's float32 precision needs.
template <int DK, bool kSplit>
struct DeltaBlock {
    static constexpr uint32_t kKB = DK / 64;
    static constexpr uint32_t kT = 0;
    static constexpr uint32_t kTlo = kBox64;
    static constexpr uint32_t kW = kSplit ? 2 * kBox64 : kBox64;
    static constexpr uint32_t kWlo = kW + kKB * kBox64;
    static constexpr uint32_t kQ = kSplit ? kWlo + kKB * kBox64 : kWlo;
    static constexpr uint32_t kP = kQ + kKB * kBox64;
    static constexpr uint32_t kHdr = kP + kBox64;       // float rest[64] = e^{G_L - G}, then e^{G_L}
    static constexpr uint32_t kBytes = kHdr + 1024;
};

// Byte offset of element (row, col) of a 64-row tile of boxes.
__device__ __forceinline__ uint32_t tile_off(int row, int col) {
    return (uint32_t)(col >> 6) * kBox64 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) +
           (col & 7) * 2;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t &r0, uint32_t &r1, const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                 : "=r"(r0), "=r"(r1)
                 : "r"(smem_u32(p)));
}
// One arrival for the warp (32 on one barrier are served one by one).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Two bf16 parts of a pair: hi the rounding, lo the rounding of what it left.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(a, b);
    lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

// ------------------------------------------------------------------ prep
// One CTA of four warps per chunk of a (sequence, value head): the two
// products by mma.sync (a 64 x 64 x dk product has too few rows to fill a
// tcgen05 tile, and a grid of thousands of chunks hides its latency), the
// inverse in float32: two 32 x 32 triangles by substitution, a column a
// lane, then the square below them by two products.
constexpr int kPrepThreads = 128;
constexpr int kMPad = 68;

template <int DK>
struct DeltaPrepSmem {
    __nv_bfloat16 K[kC][DK + 8], Q[kC][DK + 8];
    float M[kC][kMPad], T[kC][kMPad];
    double G[kC];
    float beta[kC], e[kC];
};

struct DeltaPrepArgs {
    const __nv_bfloat16 *q, *k, *g, *beta;
    const int *lengths;
    uint8_t *blocks;
    float scale;
    int heads, key_heads, tokens, nc, backward;
};

template <int DK, bool kSplit>
__global__ void __launch_bounds__(kPrepThreads)
delta_prep_kernel(DeltaPrepArgs a) {
    using Block = DeltaBlock<DK, kSplit>;
    extern __shared__ __align__(16) uint8_t raw[];
    DeltaPrepSmem<DK> &m = *reinterpret_cast<DeltaPrepSmem<DK> *>(raw);
    const int bh = blockIdx.x / a.nc, c = blockIdx.x % a.nc;
    const int b = bh / a.heads, h = bh % a.heads, kh = h / (a.heads / a.key_heads);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int gr = lane / 4, tq = lane % 4;
    grid_dependency_wait();
    const int n = delta_tokens_of(a.lengths, b, a.tokens);
    const int cnt = min(kC, n - c * kC);
    if (cnt <= 0) return;                                  // the whole CTA
    const size_t row0 = (size_t)b * a.tokens + c * kC;
    uint8_t *out = a.blocks + (size_t)blockIdx.x * Block::kBytes;

    {   // K and Q, rows behind the sequence as zeros
        constexpr int kVecs = DK / 8;
        const size_t step = (size_t)a.key_heads * DK;
        const __nv_bfloat16 *ks = a.k + (row0 * a.key_heads + kh) * (size_t)DK;
        const __nv_bfloat16 *qs = a.q + (row0 * a.key_heads + kh) * (size_t)DK;
#pragma unroll 4
        for (int i = tid; i < kC * kVecs; i += kPrepThreads) {
            const int r = i / kVecs, j = (i % kVecs) * 8;
            uint4 kv = make_uint4(0, 0, 0, 0), qv = kv;
            if (r < cnt) {
                kv = *reinterpret_cast<const uint4 *>(ks + r * step + j);
                qv = *reinterpret_cast<const uint4 *>(qs + r * step + j);
            }
            *reinterpret_cast<uint4 *>(&m.K[r][j]) = kv;
            *reinterpret_cast<uint4 *>(&m.Q[r][j]) = qv;
        }
    }
    if (warp == 0) {                                       // running sums of g
        const size_t at = row0 * a.heads + h;
        double lo = lane < cnt ? log_decay(to_f32(a.g[at + (size_t)lane * a.heads])) : 0.0;
        double hi = lane + 32 < cnt ? log_decay(to_f32(a.g[at + (size_t)(lane + 32) * a.heads])) : 0.0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double ul = __shfl_up_sync(0xffffffffu, lo, o);
            const double uh = __shfl_up_sync(0xffffffffu, hi, o);
            if (lane >= o) {
                lo += ul;
                hi += uh;
            }
        }
        hi += __shfl_sync(0xffffffffu, lo, 31);
        const double GL = __shfl_sync(0xffffffffu, hi, 31);
        m.G[lane] = lo;
        m.G[lane + 32] = hi;
        m.e[lane] = expf((float)lo);
        m.e[lane + 32] = expf((float)hi);
        float *hdr = reinterpret_cast<float *>(out + Block::kHdr);
        hdr[lane] = expf((float)(GL - lo));
        hdr[lane + 32] = expf((float)(GL - hi));
        if (lane == 0) hdr[64] = expf((float)GL);
    } else if (warp == 1) {
#pragma unroll
        for (int i = lane; i < kC; i += 32) {
            float bt = 0.f;
            if (i < cnt) {
                bt = to_f32(a.beta[(row0 + i) * a.heads + h]);
                if (a.backward) bt = nonzero_beta(bt);
            }
            m.beta[i] = bt;
        }
    }
    __syncthreads();

    // rows 16 rb .. of (a row-major operand) times the rows of K, up to the diagonal
    auto gram = [&](float (&acc)[8][4], const __nv_bfloat16 (*A)[DK + 8], int rb) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
        for (int k0 = 0; k0 < DK; k0 += 16) {
            uint32_t av[4];
            const int r = 16 * rb + gr;
            av[0] = *reinterpret_cast<const uint32_t *>(&A[r][k0 + 2 * tq]);
            av[1] = *reinterpret_cast<const uint32_t *>(&A[r + 8][k0 + 2 * tq]);
            av[2] = *reinterpret_cast<const uint32_t *>(&A[r][k0 + 2 * tq + 8]);
            av[3] = *reinterpret_cast<const uint32_t *>(&A[r + 8][k0 + 2 * tq + 8]);
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t < 2 * rb + 2) {
                    const uint32_t b0 = *reinterpret_cast<const uint32_t *>(&m.K[8 * t + gr][k0 + 2 * tq]);
                    const uint32_t b1 = *reinterpret_cast<const uint32_t *>(&m.K[8 * t + gr][k0 + 2 * tq + 8]);
                    mma16816(acc[t], av, b0, b1);
                }
        }
    };
    {   // M: warp w the rows 16 w ..
        float acc[8][4];
        gram(acc, m.K, warp);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * warp + gr + (e >= 2 ? 8 : 0), j = 8 * t + 2 * tq + (e & 1);
                m.M[i][j] = i > j ? acc[t][e] * m.beta[i] * expf((float)(m.G[i] - m.G[j])) : 0.f;
            }
    }
    __syncthreads();
    if (warp < 2) {
        // lane's column of the inverse of triangle `warp`
        const int o = 32 * warp;
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) {
                const float mv = m.M[o + i][o + j];
                if (j & 1) s1 = fmaf(-mv, x[j], s1);
                else s0 = fmaf(-mv, x[j], s0);
            }
            x[i] = s0 + s1;
            m.T[o + i][o + lane] = x[i];
        }
        if (warp == 0)                                     // the square above them
#pragma unroll
            for (int i = 0; i < 32; ++i) m.T[i][32 + lane] = 0.f;
    } else {
        // P and Q~: warps 2, 3 take row blocks {0, 3} and {1, 2}
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int rb = u ? (warp == 2 ? 3 : 2) : warp - 2;
            float acc[8][4];
            gram(acc, m.Q, rb);
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int i = 16 * rb + gr + 8 * hf, j = 8 * t + 2 * tq;
                    const float p0 = i >= j ? a.scale * acc[t][2 * hf] * expf((float)(m.G[i] - m.G[j])) : 0.f;
                    const float p1 = i >= j + 1 ? a.scale * acc[t][2 * hf + 1] * expf((float)(m.G[i] - m.G[j + 1])) : 0.f;
                    *reinterpret_cast<uint32_t *>(out + Block::kP + tile_off(i, j)) = pack_bf16x2(p0, p1);
                }
            constexpr int kVecs = DK / 8;
#pragma unroll 2
            for (int i = lane; i < 16 * kVecs; i += 32) {
                const int r = 16 * rb + i / kVecs, j = (i % kVecs) * 8;
                float qv[8];
                load8(&m.Q[r][j], qv);
                const float s = a.scale * m.e[r];
#pragma unroll
                for (int e = 0; e < 8; ++e) qv[e] *= s;
                store8(reinterpret_cast<__nv_bfloat16 *>(out + Block::kQ + tile_off(r, j)), qv);
            }
        }
    }
    __syncthreads();
    // T_10 = -T_11 (M_10 T_00): the inner product into M's free upper square
    {
        const int r = tid / 8 * 2, cc = (tid % 8) * 4;      // 2 x 4 outputs a thread
        float s[2][4] = {};
#pragma unroll 4
        for (int j = 0; j < 32; ++j) {
            const float4 t = *reinterpret_cast<const float4 *>(&m.T[j][cc]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mv = m.M[32 + r + i][j];
                s[i][0] = fmaf(mv, t.x, s[i][0]); s[i][1] = fmaf(mv, t.y, s[i][1]);
                s[i][2] = fmaf(mv, t.z, s[i][2]); s[i][3] = fmaf(mv, t.w, s[i][3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4 *>(&m.M[r + i][32 + cc]) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        __syncthreads();
        float u[2][4] = {};
#pragma unroll 4
        for (int j = 0; j < 32; ++j) {
            const float4 t = *reinterpret_cast<const float4 *>(&m.M[j][32 + cc]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float tv = m.T[32 + r + i][32 + j];
                u[i][0] = fmaf(-tv, t.x, u[i][0]); u[i][1] = fmaf(-tv, t.y, u[i][1]);
                u[i][2] = fmaf(-tv, t.z, u[i][2]); u[i][3] = fmaf(-tv, t.w, u[i][3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4 *>(&m.T[32 + r + i][cc]) = make_float4(u[i][0], u[i][1], u[i][2], u[i][3]);
    }
    __syncthreads();
    // T^ = T diag(b) in its tiles; W = T^ diag(e^G) K in two parts of T^, K being exact
    {
        const int r = 16 * warp + gr;
        float acc[DK / 8][4] = {};
#pragma unroll
        for (int j0 = 0; j0 < kC; j0 += 16) {
            if (j0 <= 16 * warp) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = r + (e & 1) * 8, j = j0 + 2 * tq + (e >> 1) * 8;
                    const float2 t = *reinterpret_cast<const float2 *>(&m.T[i][j]);
                    const float t0 = t.x * m.beta[j], t1 = t.y * m.beta[j + 1];
                    uint32_t th, tl;
                    split_pair(t0, t1, th, tl);
                    *reinterpret_cast<uint32_t *>(out + Block::kT + tile_off(i, j)) = th;
                    if (kSplit) *reinterpret_cast<uint32_t *>(out + Block::kTlo + tile_off(i, j)) = tl;
                    split_pair(-t0 * m.e[j], -t1 * m.e[j + 1], hi[e], lo[e]);
                }
#pragma unroll
                for (int t = 0; t < DK / 8; ++t) {
                    uint32_t b0, b1;
                    ldmatrix_x2_trans(b0, b1, &m.K[j0 + (lane & 15)][8 * t]);
                    mma16816(acc[t], hi, b0, b1);
                    mma16816(acc[t], lo, b0, b1);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = r + (e & 1) * 8, j = j0 + 2 * tq + (e >> 1) * 8;
                    *reinterpret_cast<uint32_t *>(out + Block::kT + tile_off(i, j)) = 0u;
                    if (kSplit) *reinterpret_cast<uint32_t *>(out + Block::kTlo + tile_off(i, j)) = 0u;
                }
            }
        }
#pragma unroll
        for (int t = 0; t < DK / 8; ++t)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t o = tile_off(r + 8 * hf, 8 * t + 2 * tq);
                uint32_t wh, wl;
                split_pair(acc[t][2 * hf], acc[t][2 * hf + 1], wh, wl);
                *reinterpret_cast<uint32_t *>(out + Block::kW + o) = wh;
                if (kSplit) *reinterpret_cast<uint32_t *>(out + Block::kWlo + o) = wl;
            }
    }
}

// ------------------------------------------------------------------ scan
// A CTA walks the chunks of a (sequence, head) with 128 columns of S.
// Warps: 0 copies, 1 MMAs, 2-9 two warpgroups of the chain (the columns of
// an accumulator, tokens or k, split between them), 10-13 the output.
// Per chunk, in the order the MMAs are issued:
//   X^T  = V^T T^^T + S^T (-W)^T    [needs S]       -> chain: X, Xs = e^{G_L-G} X
//   O^T  = S^T Q~^T                 (while the chain rounds X)
//   Z^T  = Xs^T K                   [needs X]       -> chain: S = e^{G_L} S + Z
//   O^T += X^T P^T                  (while the chain rounds S)
// S and Z go 64 rows of S at a time, so that the chain's work on one piece
// runs beside the MMAs of the other.  S itself stays in the chain's registers
// in float32.  With kSplit its operand copies are two bf16 parts: X^T takes
// S_hi (W_hi + W_lo) + S_lo W_hi, Z takes both parts of Xs against the exact
// K, so each product carries 16 bits (the lowest parts' product, 2^-18, is
// left out) and the state keeps float32 accuracy over the walk (measured
// 3e-6 after 8192 tokens); without it S is only ever seen through bf16
// outputs and one part is enough.
constexpr int kScanThreads = 448;
constexpr int kChainWarps = 8;

struct DeltaScanBars {
    uint64_t full[2], empty[2], s_ready[2], z_full[2], x_full, xs_ready, o_full, o_free, drain;
    uint32_t tmem_slot;
    int abort_flag;
};
template <int DK, bool kSplit>
struct DeltaScanSmem {
    using Block = DeltaBlock<DK, kSplit>;
    static constexpr uint32_t kK = Block::kBytes;
    static constexpr uint32_t kV = kK + Block::kKB * kBox64;
    static constexpr uint32_t kStage = kV + 2 * kBox64;
    static constexpr uint32_t kOut = 2 * kStage;          // 64 tokens x 128 channels
    static constexpr uint32_t kBars = kOut + 2 * kBox64;
    static constexpr uint32_t kBytes = kBars + 256;
    static_assert(sizeof(DeltaScanBars) <= 256 && kBytes <= 227 * 1024, "shared memory");
};
// tensor memory columns
template <int DK, bool kSplit>
struct DeltaScanTmem {
    static constexpr uint32_t kShi = 0;
    static constexpr uint32_t kSlo = DK / 2;
    static constexpr uint32_t kZ = kSplit ? DK : DK / 2;
    static constexpr uint32_t kX = kZ + DK;
    static constexpr uint32_t kXs = kX + 64;              // Xs hi, lo
    static constexpr uint32_t kXslo = kXs + 32;
    static constexpr uint32_t kXb = kXslo + 32;           // X
    static constexpr uint32_t kO = kXb + 32;
    static_assert(kO + 64 <= 512, "tensor memory");
};

struct DeltaScanArgs {
    const uint8_t *blocks;
    const int *lengths;
    const float *state_in;
    float *state_out;
    __nv_bfloat16 *out;
    __nv_bfloat16 *x_save, *s_save;        // kSave: X^T [.., dv, 64], S^T [.., dv, DK] per chunk
    int heads, key_heads, tokens, nc, dv;
    unsigned *err;
};

template <int DK, bool kSplit, bool kOut, bool kSave>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_scan_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_o, DeltaScanArgs a) {
    using Smem = DeltaScanSmem<DK, kSplit>;
    using Block = DeltaBlock<DK, kSplit>;
    using Tm = DeltaScanTmem<DK, kSplit>;
    constexpr int kPieces = DK / 64;
    // the only shared memory of the kernel, so it starts on its alignment
    extern __shared__ __align__(1024) uint8_t smem[];
    DeltaScanBars &bar = *reinterpret_cast<DeltaScanBars *>(smem + Smem::kBars);

    // warp-uniform as the compiler sees it
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int slabs = (a.dv + 127) / 128;
    const int bh = blockIdx.x / slabs, v0 = (blockIdx.x % slabs) * 128;
    const int b = bh / a.heads, h = bh % a.heads;
    unsigned *err = a.err;
    int *abort_flag = &bar.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
            mbar_init(&bar.s_ready[s], kChainWarps);
            mbar_init(&bar.z_full[s], 1);
        }
        mbar_init(&bar.x_full, 1);
        mbar_init(&bar.xs_ready, kChainWarps);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 4);
        mbar_init(&bar.drain, 1);
        bar.abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        if (kOut) tma_prefetch_desc(&tm_o);
    }
    if (warp == 1) {
        tmem_alloc(&bar.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_slot;
    grid_dependency_wait();
    const int n = delta_tokens_of(a.lengths, b, a.tokens);
    const int nc = (n + kC - 1) / kC;

    int it = 0;                                            // chunks whose copies were issued
    if (warp == 0) {
        if (lane == 0) {
            const int kh = h / (a.heads / a.key_heads);
            for (; it < nc && !*(volatile int *)abort_flag; ++it) {
                const int s = it & 1;
                if (it >= 2 && !mbar_wait(&bar.empty[s], ((it >> 1) - 1) & 1, abort_flag, err)) break;
                uint8_t *st = smem + s * Smem::kStage;
                mbar_expect_tx(&bar.full[s], Smem::kStage);
                bulk_load(st, a.blocks + ((size_t)bh * a.nc + it) * Block::kBytes, Block::kBytes,
                          &bar.full[s]);
                for (int x = 0; x < DK / 64; ++x)
                    tma_load_4d(st + Smem::kK + x * kBox64, &tm_k, &bar.full[s], 64 * x, kh, it * kC, b);
                for (int x = 0; x < 2; ++x)
                    tma_load_4d(st + Smem::kV + x * kBox64, &tm_v, &bar.full[s], v0 + 64 * x, h, it * kC, b);
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t id_tv = idesc_bf16(128, 64, 1, 0);   // A: V tile, v contiguous
        constexpr uint32_t id_x = idesc_bf16(128, 64, 0, 0);
        constexpr uint32_t id_z = idesc_bf16(128, 64, 0, 1);    // B: K box, k contiguous
        for (int c = 0; c < nc; ++c) {
            const int s = c & 1;
            uint8_t *st = smem + s * Smem::kStage;
            // K-major tiles and MN-major boxes; offsets are added >> 4
            const uint64_t kmaj = smem_desc_sw128(smem_u32(st), 16, 1024);
            const uint64_t mnmaj = smem_desc_sw128(smem_u32(st), kBox64, 1024);
            if (!warp_spin_wait(&bar.full[s], (c >> 1) & 1, abort_flag, err)) break;
            const int cnt = n - c * kC;
            if (cnt < kC) {
                // rows behind the sequence may hold anything: their products
                // meet zeros in T^ and Xs, but 0 * NaN would not be 0
                for (int i = lane; i < (kC - cnt) * 8; i += 32) {
                    const uint32_t o = (cnt + i / 8) * 128 + (i % 8) * 16;
                    for (uint32_t x = 0; x < DK / 64 + 2; ++x)
                        *reinterpret_cast<uint4 *>(st + Smem::kK + x * kBox64 + o) = make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                __syncwarp();
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t ad = mnmaj + ((Smem::kV + ks * 2048) >> 4);
                    mma_bf16(tmem + Tm::kX, ad, kmaj + ((Block::kT + ks * 32) >> 4), id_tv, ks > 0);
                    if (kSplit)
                        mma_bf16(tmem + Tm::kX, ad, kmaj + ((Block::kTlo + ks * 32) >> 4), id_tv, 1);
                }
            }
            __syncwarp();
            bool ok = true;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                ok = ok && warp_spin_wait(&bar.s_ready[p], c & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        const int ks = 4 * p + k4;
                        const uint32_t o = p * kBox64 + k4 * 32;
                        const uint64_t w = kmaj + ((Block::kW + o) >> 4);
                        mma_bf16_ts(tmem + Tm::kX, tmem + Tm::kShi + 8 * ks, w, id_x, 1);
                        if (kSplit) {
                            mma_bf16_ts(tmem + Tm::kX, tmem + Tm::kSlo + 8 * ks, w, id_x, 1);
                            mma_bf16_ts(tmem + Tm::kX, tmem + Tm::kShi + 8 * ks,
                                        kmaj + ((Block::kWlo + o) >> 4), id_x, 1);
                        }
                    }
                    if (p == kPieces - 1) mma_commit(&bar.x_full);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (kOut) {
                if (c > 0 && !warp_spin_wait(&bar.o_free, (c - 1) & 1, abort_flag, err)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < DK / 16; ++ks)
                        mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kShi + 8 * ks,
                                    kmaj + ((Block::kQ + (ks / 4) * kBox64 + (ks % 4) * 32) >> 4),
                                    id_x, ks > 0);
                }
                __syncwarp();
            }
            if (!warp_spin_wait(&bar.xs_ready, c & 1, abort_flag, err)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t kd = mnmaj + ((Smem::kK + p * kBox64 + ks * 2048) >> 4);
                        mma_bf16_ts(tmem + Tm::kZ + 64 * p, tmem + Tm::kXs + 8 * ks, kd, id_z, ks > 0);
                        if (kSplit)
                            mma_bf16_ts(tmem + Tm::kZ + 64 * p, tmem + Tm::kXslo + 8 * ks, kd, id_z, 1);
                    }
                    mma_commit(&bar.z_full[p]);
                }
                if (kOut) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kXb + 8 * ks,
                                    kmaj + ((Block::kP + ks * 32) >> 4), id_x, 1);
                    mma_commit(&bar.o_full);
                }
                mma_commit(&bar.empty[s]);
            }
            __syncwarp();
        }
    } else if (warp < 10) {
        const int wg = (warp - 2) / 4;                     // k columns 64 p + 32 wg ..
        const int v = v0 + 32 * (warp % 4) + lane;
        const bool live = v < a.dv;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
        const size_t sbase = ((size_t)bh * DK + 32 * wg) * a.dv + v;
        float S[kPieces][32];
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                S[p][j] = a.state_in && live ? a.state_in[sbase + (size_t)(64 * p + j) * a.dv] : 0.f;
        // the operand copies of a piece of S; c: the chunk that starts with it
        auto put_state = [&](int p, int c) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (kSplit) split_pair(S[p][2 * j], S[p][2 * j + 1], hi[j], lo[j]);
                else hi[j] = pack_bf16x2(S[p][2 * j], S[p][2 * j + 1]);
            }
            tmem_st16(tl + Tm::kShi + 32 * p + 16 * wg, hi);
            if (kSplit) tmem_st16(tl + Tm::kSlo + 32 * p + 16 * wg, lo);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar.s_ready[p]);
            if (kSave && live && c < nc) {
                uint4 *dst = reinterpret_cast<uint4 *>(
                    a.s_save + (((size_t)bh * a.nc + c) * a.dv + v) * DK + 64 * p + 32 * wg);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dst[j] = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
            }
        };
#pragma unroll
        for (int p = 0; p < kPieces; ++p) put_state(p, 0);
        for (int c = 0; c < nc; ++c) {
            const int s = c & 1;
            const float *hdr = reinterpret_cast<const float *>(smem + s * Smem::kStage + Block::kHdr);
            if (!warp_spin_wait(&bar.full[s], (c >> 1) & 1, abort_flag, err)) break;
            const float eL = hdr[64];
            if (!warp_spin_wait(&bar.x_full, c & 1, abort_flag, err)) break;
            tc_fence_after();
            {
                uint32_t x[32], hi[16], lo[16], xb[16];
                tmem_ld32(tl + Tm::kX + 32 * wg, x);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 r = *reinterpret_cast<const float2 *>(hdr + 32 * wg + 2 * j);
                    const float x0 = __uint_as_float(x[2 * j]), x1 = __uint_as_float(x[2 * j + 1]);
                    if (kSplit) split_pair(x0 * r.x, x1 * r.y, hi[j], lo[j]);
                    else hi[j] = pack_bf16x2(x0 * r.x, x1 * r.y);
                    if (kOut || kSave) xb[j] = pack_bf16x2(x0, x1);
                }
                tmem_st16(tl + Tm::kXs + 16 * wg, hi);
                if (kSplit) tmem_st16(tl + Tm::kXslo + 16 * wg, lo);
                if (kOut) tmem_st16(tl + Tm::kXb + 16 * wg, xb);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.xs_ready);
                if (kSave && live) {
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        a.x_save + (((size_t)bh * a.nc + c) * a.dv + v) * kC + 32 * wg);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dst[j] = make_uint4(xb[4 * j], xb[4 * j + 1], xb[4 * j + 2], xb[4 * j + 3]);
                }
            }
            bool ok = true;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                ok = ok && warp_spin_wait(&bar.z_full[p], c & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
                uint32_t z[32];
                tmem_ld32(tl + Tm::kZ + 64 * p + 32 * wg, z);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    S[p][j] = fmaf(eL, S[p][j], __uint_as_float(z[j]));
                put_state(p, c + 1);
            }
            if (!ok) break;
        }
        if (a.state_out && live)
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
#pragma unroll
                for (int j = 0; j < 32; ++j) a.state_out[sbase + (size_t)(64 * p + j) * a.dv] = S[p][j];
    } else if (kOut) {
        // O through shared memory, token rows of 64 channels (the swizzle of
        // the copy out), so that global memory sees whole lines
        const int col = 32 * (warp % 4) + lane, tid = threadIdx.x - 320;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
        uint8_t *box = smem + Smem::kOut + (col / 64) * kBox64 + (col & 7) * 2;
        for (int c = 0; c < nc; ++c) {
            if (!warp_spin_wait(&bar.o_full, c & 1, abort_flag, err)) break;
            tc_fence_after();
            uint32_t o[2][32];
            tmem_ld32(tl + Tm::kO, o[0]);
            tmem_ld32(tl + Tm::kO + 32, o[1]);
            tmem_wait_ld();
            tc_fence_before();
            warp_arrive(&bar.o_free);
            if (tid == 0) tma_store_wait_read();           // the last tile has left
            named_barrier(1, 128);
#pragma unroll
            for (int i = 0; i < kC; ++i)
                *reinterpret_cast<__nv_bfloat16 *>(box + i * 128 + ((((col & 63) >> 3) ^ (i & 7)) << 4)) =
                    __float2bfloat16_rn(__uint_as_float(o[i / 32][i % 32]));
            const int cnt = n - c * kC;
            if (cnt >= kC) fence_async_shared();
            named_barrier(1, 128);
            if (cnt >= kC) {
                if (tid == 0) {
                    for (int x = 0; x < 2; ++x)
                        if (v0 + 64 * x < a.dv)
                            tma_store_4d(&tm_o, smem + Smem::kOut + x * kBox64, v0 + 64 * x, h, c * kC, b);
                    tma_store_commit();
                }
            } else {                                       // rows behind the sequence stay
                for (int i = tid; i < cnt * 16; i += 128) {
                    const int r = i / 16, ch = i % 16;
                    if (v0 + ch * 8 < a.dv)
                        *reinterpret_cast<uint4 *>(
                            a.out + (((size_t)b * a.tokens + c * kC + r) * a.heads + h) * a.dv + v0 + ch * 8) =
                            *reinterpret_cast<const uint4 *>(smem + Smem::kOut + (ch / 8) * kBox64 + r * 128 +
                                                             (((ch & 7) ^ (r & 7)) << 4));
                }
            }
        }
        if (tid == 0) tma_store_wait_read();
    }
    tc_fence_before();
    __syncthreads();
    // After an abort, wait (bounded) for the copies still in flight before
    // shared memory goes away and for the MMAs before tensor memory is freed.
    if (*abort_flag && warp == 0 && lane == 0)
        for (int j = max(0, it - 2); j < it; ++j) mbar_drain(&bar.full[j & 1], (j >> 1) & 1, err);
    if (warp == 1) {
        if (*abort_flag && lane == 0) {
            mma_commit(&bar.drain);
            mbar_drain(&bar.drain, 0, err);
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ launches
// Map of [batch, n, heads, d] in boxes of 64 tokens x 64 channels of one head.
bool token_map(CUtensorMap *tm, const void *p, int batch, int n, int heads, int d) {
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n, (cuuint64_t)batch};
    cuuint64_t str[3] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2, (cuuint64_t)n * heads * d * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kC, 1};
    return make_tensor_map_bf16(tm, p, 4, dims, str, box);
}

template <int DK, bool kSplit>
cudaError_t launch_prep(const DeltaArgs &a, int nc, uint8_t *blocks, bool backward,
                        cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(delta_prep_kernel<DK, kSplit>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DeltaPrepSmem<DK>));
    if (e != cudaSuccess) return e;
    DeltaPrepArgs p = {(const __nv_bfloat16 *)a.q, (const __nv_bfloat16 *)a.k,
                       (const __nv_bfloat16 *)a.g, (const __nv_bfloat16 *)a.beta, a.lengths,
                       blocks, a.scale, a.heads, a.key_heads, a.seqlen, nc, backward ? 1 : 0};
    KernelTimer timer("delta_prep", stream);
    count_launch();
    return launch_overlapped(delta_prep_kernel<DK, kSplit>,
                             dim3((unsigned)((long long)a.batch * a.heads * nc)), dim3(kPrepThreads),
                             sizeof(DeltaPrepSmem<DK>), stream, p);
}

template <int DK, bool kSplit, bool kOut, bool kSave>
cudaError_t launch_scan(const DeltaArgs &a, int nc, const uint8_t *blocks, __nv_bfloat16 *x_save,
                        __nv_bfloat16 *s_save, cudaStream_t stream) {
    using Smem = DeltaScanSmem<DK, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(delta_scan_kernel<DK, kSplit, kOut, kSave>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Smem::kBytes);
    if (e != cudaSuccess) return e;
    CUtensorMap tm_k, tm_v, tm_o;
    if (!token_map(&tm_k, a.k, a.batch, a.seqlen, a.key_heads, a.dk) ||
        !token_map(&tm_v, a.v, a.batch, a.seqlen, a.heads, a.dv) ||
        !token_map(&tm_o, kOut ? a.out : a.v, a.batch, a.seqlen, a.heads, a.dv))
        return cudaErrorInvalidValue;
    DeltaScanArgs s = {blocks, a.lengths, a.state_in, a.state_out, (__nv_bfloat16 *)a.out, x_save,
                       s_save, a.heads, a.key_heads, a.seqlen, nc, a.dv, device_error_word()};
    const int slabs = (a.dv + 127) / 128;
    KernelTimer timer("delta_scan", stream);
    count_launch();
    return launch_overlapped(delta_scan_kernel<DK, kSplit, kOut, kSave>,
                             dim3((unsigned)(a.batch * a.heads * slabs)), dim3(kScanThreads),
                             Smem::kBytes, stream, tm_k, tm_v, tm_o, s);
}

template <int DK, bool kSplit>
cudaError_t launch_forward(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    const int nc = (a.seqlen + kC - 1) / kC;
    cudaError_t e = launch_prep<DK, kSplit>(a, nc, (uint8_t *)workspace, false, stream);
    if (e != cudaSuccess) return e;
    return launch_scan<DK, kSplit, true, false>(a, nc, (const uint8_t *)workspace, nullptr, nullptr,
                                                stream);
}

}  // namespace

bool delta_tc_shape_ok(int dk, int dv, retnet_dtype dtype) {
    return dtype == RETNET_BF16 && (dk == 64 || dk == 128) && dv >= 64;
}

size_t delta_tc_workspace(int batch, int heads, int seqlen, int dk) {
    const size_t chunks = (size_t)batch * heads * ((seqlen + kC - 1) / kC);
    return chunks * (dk == 64 ? DeltaBlock<64, true>::kBytes : DeltaBlock<128, true>::kBytes);
}

cudaError_t launch_delta_tc(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    if (a.dk == 64)
        return a.state_out ? launch_forward<64, true>(a, workspace, stream)
                           : launch_forward<64, false>(a, workspace, stream);
    return a.state_out ? launch_forward<128, true>(a, workspace, stream)
                       : launch_forward<128, false>(a, workspace, stream);
}

}  // namespace retnet
