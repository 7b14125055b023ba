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
// memory, all of it by bulk copies one chunk ahead; outputs go from registers
// to global memory, 64 bytes a warp and token.
//
// Roundings.  Accumulators, states, sums and decays are float32; the operands
// of a product are bf16, in one part or, where one moved a result by more than
// its own rounding and a second costs little, in two (2^-17; each part more is
// a product more).  In two: P and X, which alone made an output's error 3.1e-3
// instead of 2.1e-3; X, A, B and dV where the gradients are formed of them
// (dq 3.0 to 1.9e-3, dbeta 3.5 to 1.8e-3); e^{G_L - G} X and, in the backward,
// Q~, whose errors stay in the state and its gradient while decays are slow
// (dg with mean log decays of -0.002: 4.6 to 2.8e-3); dX for dV.  With these
// in one part calls of the backward of few heads were up to 6e-3 off in dg.
// What the others move a result by (2-norm, 400 tokens of 128 x 128, mean log
// decay -0.02; made one at a time by oracle/delta_chunks.py, and the kernels'
// errors are those of all of them within 1 %): the result 1.7e-3, Q~ of an
// output and S 0.8e-3, D 0.8e-3, T^ 0.3e-3, W 0.2e-3, dX 0.2e-3, dV as it left
// 0.4e-3 of dk; together 2.1e-3 of an output, 1.8 to 2.2e-3 of the gradients
// (1.7e-3 and 1.7 to 1.8e-3 at -0.2, 2.7e-3 and 2.3 to 2.8e-3 at -0.002).  A
// final state has no rounding of a result behind it, so all that it depends on
// goes in two parts (kSplit): 3.4e-6 instead of 0.4e-3.
#include "delta.cuh"
#include "pairs.cuh"
#include "sm100_chain.cuh"

namespace retnet {
namespace {

using namespace sm100;

constexpr int kC = kDeltaChunk;
constexpr uint32_t kBox64 = 8192;          // 64 rows x 64 bf16, 128-byte swizzled

#ifdef RETNET_TEST_HOOKS
// Test hook (debug build only): when set, the walks of the first (sequence,
// head)'s first columns and the gradient kernel's first CTA never issue their
// second stage's copies, so that waits run out with MMAs of the first issued.
static __device__ int g_hook_skip_second_load = 0;
__device__ __forceinline__ bool hook_skips(bool first, int it) {
    return first && it == 1 && *(volatile int *)&g_hook_skip_second_load;
}
#else
__device__ __forceinline__ constexpr bool hook_skips(bool, int) { return false; }
#endif

// One chunk's prepared operands, in shared-memory order.  Every tile is
// boxes of 64 rows (tokens) of 64 columns, 128-byte swizzled.
// kSplit: T^ and W in two bf16 parts (16 bits together), which the final
// state's float32 precision needs.  P is in two in any case.
template <int DK, bool kSplit>
struct DeltaBlock {
    static constexpr uint32_t kKB = DK / 64;
    static constexpr uint32_t kT = 0;
    static constexpr uint32_t kTlo = kBox64;
    static constexpr uint32_t kW = kSplit ? 2 * kBox64 : kBox64;
    static constexpr uint32_t kWlo = kW + kKB * kBox64;
    // float rest[64] = e^{G_L - G}, then e^{G_L}; a walk without output stops
    // here.  Of the backward: whether any token writes nothing, at 65, and
    // which do, at 128.
    static constexpr uint32_t kHdr = kSplit ? kWlo + kKB * kBox64 : kWlo;
    static constexpr uint32_t kQ = kHdr + 1024;
    // P in two parts; the prep's copy in shared memory ends with the first
    static constexpr uint32_t kP = kQ + kKB * kBox64;
    static constexpr uint32_t kPlo = kP + kBox64;
    static constexpr uint32_t kBytes = kPlo + kBox64;
    // the backward's blocks, with Q~'s second part
    static constexpr uint32_t kQlo = kBytes;
    static constexpr uint32_t kBack = kQlo + kKB * kBox64;
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
// One arrival for the warp (32 on one barrier are served one by one).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Waits (bounded) for the MMAs that this warp has in flight.  A commit only
// tracks what its own thread issued, and elect.sync chooses the same lane for
// the same mask each time, so it is issued as the MMAs were.
__device__ __forceinline__ void drain_mmas(uint64_t *bar, unsigned *err) {
    __syncwarp();
    if (elect_one()) mma_commit(bar);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_drain(bar, 0, err);
    __syncwarp();
}
// Two bf16 parts of a pair: hi the rounding, lo the rounding of what it left.
__device__ __forceinline__ void split_pair(float2 x, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(x.x, x.y);
    const float2 left = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                             both(-1.f), x);
    lo = pack_bf16x2(left.x, left.y);
}
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    split_pair(make_float2(a, b), hi, lo);
}
__device__ __forceinline__ float2 as_pair(uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// Rows cnt.. of `boxes` 64-row boxes as zeros, by one warp.  Rows behind a
// sequence may hold anything; the products that sum over tokens meet zeros
// there on their other side, but 0 * NaN would not be 0.
__device__ __forceinline__ void clear_rows(uint8_t *box, int boxes, int cnt, int lane) {
    for (int i = lane; i < (kC - cnt) * 8; i += 32) {
        const uint32_t o = (cnt + i / 8) * 128 + (i % 8) * 16;
        for (int x = 0; x < boxes; ++x)
            *reinterpret_cast<uint4 *>(box + x * kBox64 + o) = make_uint4(0, 0, 0, 0);
    }
    fence_async_shared();
    __syncwarp();
}
// Rows of the tokens that write nothing (flags[row] != 0) as zeros, likewise.
__device__ __forceinline__ void clear_flagged(uint8_t *box, int boxes, const float *flags, int lane) {
    for (int r = 0; r < kC; ++r)
        if (flags[r] != 0.f && lane < 8 * boxes)
            *reinterpret_cast<uint4 *>(box + (lane / 8) * kBox64 + r * 128 + (lane % 8) * 16) = make_uint4(0, 0, 0, 0);
    fence_async_shared();
    __syncwarp();
}
// 64 tokens of a v channel's accumulator into a tile of token rows (two
// boxes of 64 channels), bf16: col is the channel in the tile.  x becomes the
// pairs' second parts, in its first half.
__device__ __forceinline__ void put_channel(uint8_t *tile, int col, uint32_t (&x)[64]) {
    uint8_t *box = tile + (col / 64) * kBox64 + (col & 7) * 2;
    const int seg = (col & 63) >> 3;
#pragma unroll
    for (int i = 0; i < kC; i += 2) {
        uint32_t hi;
        split_pair(as_pair(x[i], x[i + 1]), hi, x[i / 2]);
        *reinterpret_cast<uint16_t *>(box + i * 128 + ((seg ^ (i & 7)) << 4)) = (uint16_t)hi;
        *reinterpret_cast<uint16_t *>(box + (i + 1) * 128 + ((seg ^ ((i + 1) & 7)) << 4)) = (uint16_t)(hi >> 16);
    }
}

// What the walks keep for the gradients (X^T, S^T, D^T: a row of `cols`
// values per v channel and chunk; in bf16, as the operands that they have just
// been and will be again) lies as [chunk][block of 64 channels][group
// of 8 columns][channel][8]: a warp, whose lanes are channels, writes 512
// consecutive bytes at a time, and a block is one copy and, as it is, an
// MN-major operand without swizzle (columns by channels).  Offset, in
// elements, of 8 columns of channel v.
__device__ __forceinline__ size_t kept_off(size_t chunk, int dv, int v, int cols, int col) {
    return ((chunk * (dv / 64) + v / 64) * (cols / 8) + col / 8) * 512 + (v % 64) * 8;
}
__device__ __forceinline__ void keep_row(__nv_bfloat16 *kept, size_t chunk, int dv, int v, int cols,
                                         int col, const uint32_t (&x)[16]) {
    uint4 *dst = reinterpret_cast<uint4 *>(kept + kept_off(chunk, dv, v, cols, col));
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[64 * j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}

// ------------------------------------------------------------------ prep
// One CTA of eight warps per chunk of a (sequence, value head): the products
// by mma.sync, whose accumulators are in the registers that apply the decays
// and split the results; the inverse in float32: four 16 x 16 triangles by
// substitution, a column a lane, then the squares below them by products, 16
// and then 32 rows at a time.  77 us for 2048 chunks of 128 x 256 (69 before
// P's second part, of which its copies took 33); what bounds it is half the
// issue slots and its barriers.
// [Q; K] K^T as one tcgen05 product of 128 rows, as delta_grad_tc_kernel forms
// it, and CTAs that stay for several chunks have not been built here.
// The chunk's block is put together in shared memory, K and Q first where W
// and Q~ replace them, and leaves by one copy; second parts of P and Q~, for
// which three CTAs leave no room there, go from registers to global memory.
// Decays e^{G_i - G_j}: of rows and columns in different 16-row blocks as
// e^{G_i - G_r} e^{G_r - G_j} with r the row before the block of i, so that
// both factors are at most 1 and 160 exponentials replace 2000.
constexpr int kPrepThreads = 256;
constexpr int kMPad = 68;

template <int DK, bool kSplit>
struct DeltaPrepSmem {
    uint8_t block[DeltaBlock<DK, kSplit>::kPlo];
    float M[kC][kMPad];                    // M, then T in its place
    DecaySums G;
    float beta[kC], own[kC];               // b; 1 where a token of the backward writes nothing
    float e[kC], in[kC];                   // e^G; e^{G_i - G_r}
    float across[3][kC];                   // [block - 1][j]: e^{G_r - G_j}
    float diag[kC][20];                    // [i][j - r - 1]: e^{G_i - G_j} in a block, 0 above
};

struct DeltaPrepArgs {
    const __nv_bfloat16 *q, *k, *g, *beta;
    const int *lengths;
    uint8_t *blocks;
    float scale;
    int heads, key_heads, tokens, nc, backward;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}

// Rows 16 RB .. and 16-column tiles T0 .. T0 + NT - 1 of M or P.  P's second
// part goes straight to the block in global memory: there is no room for it
// beside three CTAs an SM.
template <int DK, bool kSplit, int RB, int T0, int NT>
__device__ __forceinline__ void pair_tiles(DeltaPrepSmem<DK, kSplit> &m, uint8_t *plo, bool isP, float scale,
                                           int lane) {
    using Block = DeltaBlock<DK, kSplit>;
    const uint8_t *Kt = m.block + Block::kW, *At = isP ? m.block + Block::kQ : Kt;
    const int gr = lane / 4, tq = lane % 4;
    float acc[2 * NT][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < DK; k0 += 16) {
        uint32_t av[4];
        ldmatrix_x4(av, At + tile_off(16 * RB + (lane & 15), k0 + 8 * (lane >> 4)));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t bv[4];
            ldmatrix_x4(bv, Kt + tile_off(16 * (T0 + t) + (lane & 7) + ((lane >> 4) << 3),
                                          k0 + 8 * ((lane >> 3) & 1)));
            mma16816(acc[2 * t], av, bv[0], bv[1]);
            mma16816(acc[2 * t + 1], av, bv[2], bv[3]);
        }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int i = 16 * RB + gr + 8 * hf;
        const float f = isP ? scale : m.beta[i], far = f * m.in[i];
#pragma unroll
        for (int t = 0; t < 2 * NT; ++t) {
            const int j = 16 * T0 + 8 * t + 2 * tq;
            float2 w = make_float2(acc[t][2 * hf], acc[t][2 * hf + 1]);
            if (T0 + t / 2 < RB) {
                w = mul2(mul2(w, both(far)), *reinterpret_cast<const float2 *>(&m.across[RB > 0 ? RB - 1 : 0][j]));
            } else {                                       // M has no diagonal
                w = mul2(mul2(w, both(f)), *reinterpret_cast<const float2 *>(&m.diag[i][j & 15]));
                if (!isP && i == j) w.x = 0.f;
                if (!isP && i == j + 1) w.y = 0.f;
            }
            if (isP) {
                uint32_t hi, lo;
                split_pair(w, hi, lo);
                *reinterpret_cast<uint32_t *>(m.block + Block::kP + tile_off(i, j)) = hi;
                *reinterpret_cast<uint32_t *>(plo + tile_off(i, j)) = lo;
            } else
                *reinterpret_cast<float2 *>(&m.M[i][j]) = w;
        }
    }
}

// An 8-column tile of sign A B for 16 rows of A (both kMPad wide, K columns
// deep) by one warp, in three tf32 products (x = hi + lo, lo lo left out:
// 2^-22), to C.
template <int K>
__device__ __forceinline__ void square_tile(const float *A, const float *B, float *C, float sign,
                                            int lane) {
    const int gr = lane / 4, tq = lane % 4;
    float acc[4] = {};
    auto part = [](float x, uint32_t &hi, uint32_t &lo) {
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
    };
    auto mma = [&acc](const uint32_t (&x)[4], const uint32_t (&y)[2]) {
        asm volatile(
            "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
            : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(y[0]), "r"(y[1]));
    };
#pragma unroll
    for (int k = 0; k < K; k += 8) {
        uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            part(A[(gr + 8 * (e & 1)) * kMPad + k + tq + 4 * (e >> 1)], ah[e], al[e]);
#pragma unroll
        for (int e = 0; e < 2; ++e) part(B[(k + tq + 4 * e) * kMPad + gr], bh[e], bl[e]);
        mma(ah, bh);
        mma(ah, bl);
        mma(al, bh);
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
        *reinterpret_cast<float2 *>(&C[(gr + 8 * hf) * kMPad + 2 * tq]) =
            make_float2(sign * acc[2 * hf], sign * acc[2 * hf + 1]);
}

template <int DK, bool kSplit>
__global__ void __launch_bounds__(kPrepThreads, DK == 128 && kSplit ? 2 : 3)
delta_prep_kernel(DeltaPrepArgs a) {
    using Block = DeltaBlock<DK, kSplit>;
    extern __shared__ __align__(1024) uint8_t smem[];
    DeltaPrepSmem<DK, kSplit> &m = *reinterpret_cast<DeltaPrepSmem<DK, kSplit> *>(smem);
    uint8_t *Kt = m.block + Block::kW, *Qt = m.block + Block::kQ;
    const int bh = blockIdx.x / a.nc, c = blockIdx.x % a.nc;
    const int b = bh / a.heads, h = bh % a.heads, kh = h / (a.heads / a.key_heads);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int gr = lane / 4, tq = lane % 4;
    grid_dependency_wait();
    const int n = delta_tokens_of(a.lengths, b, a.tokens);
    const int cnt = min(kC, n - c * kC);
    if (cnt <= 0) return;                                  // the whole CTA
    const size_t row0 = (size_t)b * a.tokens + c * kC;

    {   // K and Q, rows behind the sequence as zeros
        constexpr int kVecs = DK / 8, kEach = kC * kVecs / kPrepThreads;
        const size_t step = (size_t)a.key_heads * DK;
        const __nv_bfloat16 *ks = a.k + (row0 * a.key_heads + kh) * (size_t)DK;
        const __nv_bfloat16 *qs = a.q + (row0 * a.key_heads + kh) * (size_t)DK;
        uint4 kv[kEach], qv[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int i = tid + u * kPrepThreads, r = i / kVecs, j = (i % kVecs) * 8;
            kv[u] = qv[u] = make_uint4(0, 0, 0, 0);
            if (r < cnt) {
                kv[u] = *reinterpret_cast<const uint4 *>(ks + r * step + j);
                qv[u] = *reinterpret_cast<const uint4 *>(qs + r * step + j);
            }
        }
        if (warp == 0) {                                   // running sums of g
            const size_t at = row0 * a.heads + h;
            const float lo = lane < cnt ? log_decay(to_f32(a.g[at + (size_t)lane * a.heads])) : 0.f;
            const float hi = lane + 32 < cnt ? log_decay(to_f32(a.g[at + (size_t)(lane + 32) * a.heads])) : 0.f;
            sum_decays(m.G, lane, lo, hi);
        } else if (warp == 1) {
            float *hdr = reinterpret_cast<float *>(m.block + Block::kHdr);
            unsigned any = 0;
#pragma unroll
            for (int i = lane; i < kC; i += 32) {
                const float bt = i < cnt ? to_f32(a.beta[(row0 + i) * a.heads + h]) : 0.f;
                const bool none = a.backward && i < cnt && writes_nothing(bt);
                m.beta[i] = none ? 0.f : bt;
                m.own[i] = none ? 1.f : bt;
                hdr[128 + i] = none ? 1.f : 0.f;
                any |= __ballot_sync(0xffffffffu, none);
            }
            if (lane == 0) hdr[65] = any ? 1.f : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int i = tid + u * kPrepThreads, r = i / kVecs, j = (i % kVecs) * 8;
            *reinterpret_cast<uint4 *>(Kt + tile_off(r, j)) = kv[u];
            *reinterpret_cast<uint4 *>(Qt + tile_off(r, j)) = qv[u];
        }
    }
    __syncthreads();
    if (tid < 64) {
        m.e[tid] = expf(m.G.since_start(tid));
        m.in[tid] = expf(m.G.in[tid].x + m.G.in[tid].y);
    } else if (tid < 128) {
        float *hdr = reinterpret_cast<float *>(m.block + Block::kHdr);
        hdr[tid - 64] = expf(m.G.until(tid - 64, 3));
        if (tid == 64) hdr[64] = expf(m.G.since_start(kC - 1));
    } else if (tid < 224) {                                // 16, 32 and 48 columns
        const int t = tid - 128, blk = t < 16 ? 1 : t < 48 ? 2 : 3;
        const int j = t - (blk == 1 ? 0 : blk == 2 ? 16 : 48);
        m.across[blk - 1][j] = expf(m.G.until(j, blk - 1));
    }
    uint8_t *block = a.blocks + (size_t)blockIdx.x * (a.backward ? Block::kBack : Block::kBytes);
    uint8_t *plo = block + Block::kPlo;
    if (tid < 192) {                                       // of P's second part: six squares above the diagonal
        const int q = tid / 32, rb = q < 3 ? 0 : q < 5 ? 1 : 2, cb = q < 3 ? 1 + q : q < 5 ? q - 1 : 3;
        *reinterpret_cast<uint4 *>(plo + tile_off(16 * rb + (tid & 31) / 2, 16 * cb + 8 * (tid & 1))) =
            make_uint4(0, 0, 0, 0);
    }
    {   // above the diagonal: P, and M where its triangles' inverses are multiplied
        const int r = tid / 4;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint4 *>(m.block + Block::kP + tid * 32 + 16 * u) = make_uint4(0, 0, 0, 0);
        if ((r & 16) == 0) *reinterpret_cast<float4 *>(&m.M[r][(r & 32) + 16 + 4 * (tid % 4)]) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = tid / 4, j = 4 * (tid % 4) + u;
        m.diag[i][j] = (i & 15) >= j ? expf(m.G.within(i, (i & ~15) + j)) : 0.f;
    }
    __syncthreads();

    // warps 0-3: M from K K^T, warps 4-7: P from Q K^T, two or three of the ten
    // 16 x 16 tiles up to the diagonal each
    switch (warp & 3) {
        case 0: pair_tiles<DK, kSplit, 3, 0, 2>(m, plo, warp >= 4, a.scale, lane); break;
        case 1: pair_tiles<DK, kSplit, 3, 2, 2>(m, plo, warp >= 4, a.scale, lane); break;
        case 2: pair_tiles<DK, kSplit, 2, 0, 3>(m, plo, warp >= 4, a.scale, lane); break;
        default:
            pair_tiles<DK, kSplit, 1, 0, 2>(m, plo, warp >= 4, a.scale, lane);
            pair_tiles<DK, kSplit, 0, 0, 1>(m, plo, warp >= 4, a.scale, lane);
    }
    __syncthreads();
    if (warp < 4) {
        // lane's column of the inverse of triangle `warp` (lanes 16.. repeat them)
        const int o = 16 * warp, col = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == col ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) {
                const float mv = m.M[o + i][o + j];
                if (j & 1) s1 = fmaf(-mv, x[j], s1);
                else s0 = fmaf(-mv, x[j], s0);
            }
            x[i] = s0 + s1;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) m.M[o + i][o + col] = x[i];
    } else {                                               // Q~ where Q was, bf16 as its operand
        constexpr int kVecs = DK / 8;
#pragma unroll 2
        for (int i = tid - 128; i < kC * kVecs; i += 128) {
            const int r = i / kVecs, j = (i % kVecs) * 8;
            __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(Qt + tile_off(r, j));
            float qv[8];
            load8(p, qv);
            const float f = a.scale * m.e[r];
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_pair(qv[2 * e] * f, qv[2 * e + 1] * f, hi[e], lo[e]);
            *reinterpret_cast<uint4 *>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (a.backward)
                *reinterpret_cast<uint4 *>(block + Block::kQlo + tile_off(r, j)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    __syncthreads();
    // T_10 = -T_11 (M_10 T_00), for the two pairs of triangles of 16 rows and
    // then for those of 32; the inner product goes to the square of M above
    // the diagonal of 32, which is not read otherwise
    {
        const int o = 32 * (warp & 1), t8 = 8 * ((warp >> 1) & 1);     // warps 0-3
        if (warp < 4) square_tile<16>(&m.M[o + 16][o], &m.M[o][o + t8], &m.M[o / 2][32 + t8], 1.f, lane);
        __syncthreads();
        if (warp < 4)
            square_tile<16>(&m.M[o + 16][o + 16], &m.M[o / 2][32 + t8], &m.M[o + 16][o + t8], -1.f, lane);
        __syncthreads();
        const int r = 16 * (warp & 1), c8 = 8 * (warp >> 1);           // a tile a warp
        square_tile<32>(&m.M[32 + r][0], &m.M[0][c8], &m.M[r][32 + c8], 1.f, lane);
        __syncthreads();
        square_tile<32>(&m.M[32 + r][32], &m.M[0][32 + c8], &m.M[32 + r][c8], -1.f, lane);
        __syncthreads();
    }
    // T^ = T diag(b) in its tiles; W = T^ diag(e^G) K in two parts of T^, K
    // being exact: warp w the rows 16 (w % 4) and a half of the columns.
    // Where a token of the backward writes nothing, T^ has T itself in the
    // tiles: dV = T^^T dX is then the gradient of x, and the forward walk
    // meets a row of zeros there instead of V's.
    {
        constexpr int kTiles = DK / 16;                    // of 8 columns
        const int rb = warp & 3, half = warp >> 2, r = 16 * rb + gr;
        float acc[kTiles][4] = {};
#pragma unroll
        for (int j0 = 0; j0 < kC; j0 += 16) {
            if (j0 <= 16 * rb) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = r + (e & 1) * 8, j = j0 + 2 * tq + (e >> 1) * 8;
                    const float2 t = *reinterpret_cast<const float2 *>(&m.M[i][j]);
                    const float2 bt = *reinterpret_cast<const float2 *>(&m.beta[j]);
                    const float2 ej = *reinterpret_cast<const float2 *>(&m.e[j]);
                    const float t0 = t.x * bt.x, t1 = t.y * bt.y;
                    if (half == 0) {
                        uint32_t th, tl;
                        const float2 own = *reinterpret_cast<const float2 *>(&m.own[j]);
                        split_pair(t.x * own.x, t.y * own.y, th, tl);
                        *reinterpret_cast<uint32_t *>(m.block + Block::kT + tile_off(i, j)) = th;
                        if (kSplit) *reinterpret_cast<uint32_t *>(m.block + Block::kTlo + tile_off(i, j)) = tl;
                    }
                    split_pair(-t0 * ej.x, -t1 * ej.y, hi[e], lo[e]);
                }
#pragma unroll
                for (int t = 0; t < kTiles; t += 2) {
                    uint32_t bv[4];
                    ldmatrix_x4_trans(bv, Kt + tile_off(j0 + (lane & 15), half * (DK / 2) + 8 * t + 8 * (lane >> 4)));
                    mma16816(acc[t], hi, bv[0], bv[1]);
                    mma16816(acc[t], lo, bv[0], bv[1]);
                    mma16816(acc[t + 1], hi, bv[2], bv[3]);
                    mma16816(acc[t + 1], lo, bv[2], bv[3]);
                }
            } else if (half == 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t o = tile_off(r + (e & 1) * 8, j0 + 2 * tq + (e >> 1) * 8);
                    *reinterpret_cast<uint32_t *>(m.block + Block::kT + o) = 0u;
                    if (kSplit) *reinterpret_cast<uint32_t *>(m.block + Block::kTlo + o) = 0u;
                }
            }
        }
        __syncthreads();                                   // K has been read
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t o = tile_off(r + 8 * hf, half * (DK / 2) + 8 * t + 2 * tq);
                uint32_t wh, wl;
                split_pair(acc[t][2 * hf], acc[t][2 * hf + 1], wh, wl);
                *reinterpret_cast<uint32_t *>(m.block + Block::kW + o) = wh;
                if (kSplit) *reinterpret_cast<uint32_t *>(m.block + Block::kWlo + o) = wl;
            }
    }
    fence_async_shared();
    __syncthreads();
    if (tid == 0) {
        bulk_store(block, m.block, Block::kPlo);
        tma_store_commit();
        tma_store_wait_read();
    }
}

// ------------------------------------------------------------------ scan
// A CTA walks the chunks of a (sequence, head) with 128 columns of S.
// Warps: 0 copies, 1 MMAs, 2-9 two warpgroups of the chain (the columns of
// an accumulator, tokens or k, split between them), 10-13 the output.
// Per chunk, in the order the MMAs are issued:
//   X^T  = V^T T^^T + S^T (-W)^T    [needs S]       -> chain: Xs = e^{G_L-G} X, then X
//   O^T  = S^T Q~^T                 (while the chain rounds X)
//   Z^T  = Xs^T K                   [needs Xs]      -> chain: S = e^{G_L} S + Z
//   O^T += X^T P^T                  (while the chain rounds S)
// S and Z go 64 rows of S at a time, so that the chain's work on one piece
// runs beside the MMAs of the other.  S itself stays in the chain's registers
// in float32.  Z takes both bf16 parts of Xs against the exact K.  With kSplit
// S's operand copies have two parts too: X^T takes S_hi (W_hi + W_lo) + S_lo
// W_hi, so each product carries 16 bits (the lowest parts' product, 2^-18, is
// left out) and the state keeps float32 accuracy over the walk (measured 3e-6
// to 4e-6 after 8192 tokens); without it S is only ever seen through bf16
// outputs, and one part of it and of T^ and W is enough.
constexpr int kScanThreads = 448;
constexpr int kChainWarps = 8;

struct DeltaScanBars {
    uint64_t full[2], empty[2], s_ready[2], z_full[2], x_full, xs_ready, xb_ready, o_full, o_free, drain;
    uint32_t tmem_slot;
    int abort_flag;
};
template <int DK, bool kSplit>
struct DeltaScanSmem {
    using Block = DeltaBlock<DK, kSplit>;
    static constexpr uint32_t kK = Block::kBytes;
    static constexpr uint32_t kV = kK + Block::kKB * kBox64;
    static constexpr uint32_t kStage = kV + 2 * kBox64;
    static constexpr uint32_t kBars = 2 * kStage;
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
    static constexpr uint32_t kXb = kXslo + 32;           // X hi, lo
    static constexpr uint32_t kXblo = kXb + 32;
    static constexpr uint32_t kO = kXblo + 32;
    static_assert(kO + 64 <= 512, "tensor memory");
};

struct DeltaScanArgs {
    const uint8_t *blocks;
    const int *lengths;
    const float *state_in;
    float *state_out;
    __nv_bfloat16 *out;
    __nv_bfloat16 *x_save, *s_save;        // kSave: X^T, S^T of every chunk (keep_row)
    int heads, key_heads, tokens, nc, dv;
    unsigned *err;
    // walks in segments (delta_segments_kernel)
    int segments, segment;                 // how many, and chunks of each
    float *starts, *units;
};
// What one CTA walks: chunks [first, last) of (sequence, head) bh with the
// columns v0 .. of the state, from `from` (may be null: zero) to `to` (may be
// null), both [dk, width].  unit: the state starts as the identity and no
// values are written, so that it ends as the segment's transition.  keep: what
// the gradients need is kept.
struct DeltaWalk {
    int bh, v0, first, last, width;
    const float *from;
    float *to;
    bool out, unit, keep;
};
__device__ __forceinline__ DeltaWalk whole_walk(const DeltaScanArgs &a, int dk, int cta, bool out) {
    const int slabs = (a.dv + 127) / 128, bh = cta / slabs;
    const size_t at = (size_t)bh * dk * a.dv;
    return {bh, (cta % slabs) * 128, 0, a.nc, a.dv, a.state_in ? a.state_in + at : nullptr,
            a.state_out ? a.state_out + at : nullptr, out, false, true};
}

// kFine: in two parts; kSplit: the blocks have two.
template <int DK, bool kSplit, bool kOut, bool kSave, bool kFine>
__device__ __forceinline__ void forward_walk(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                             const DeltaScanArgs &a,
                                             const DeltaWalk &w) {
    using Smem = DeltaScanSmem<DK, kSplit>;
    using Block = DeltaBlock<DK, kSplit>;
    using Tm = DeltaScanTmem<DK, kSplit>;
    constexpr int kPieces = DK / 64;
    // the only shared memory of the kernel, so it starts on its alignment
    extern __shared__ __align__(1024) uint8_t smem[];
    DeltaScanBars &bar = *reinterpret_cast<DeltaScanBars *>(smem + Smem::kBars);

    // warp-uniform as the compiler sees it
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int bh = w.bh, v0 = w.v0;
    const int b = bh / a.heads, h = bh % a.heads;
    const bool out = kOut && w.out, again = out || (kSave && w.keep);   // X itself is used
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
        mbar_init(&bar.xb_ready, kOut ? kChainWarps : 4);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 4);
        mbar_init(&bar.drain, 1);
        bar.abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) {
        tmem_alloc(&bar.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All 512 columns are this CTA's, so they start at address 0; as a
    // constant it keeps the MMAs' operands out of general registers.
    constexpr uint32_t tmem = 0;
    grid_dependency_wait();
    const int n = delta_tokens_of(a.lengths, b, a.tokens) - w.first * kC;   // from the first chunk on
    const int nc = max(0, min(w.last - w.first, (n + kC - 1) / kC));

    int it = 0;                                            // chunks whose copies were issued
    if (warp == 0) {
        const int kh = h / (a.heads / a.key_heads);
        constexpr uint32_t kStep = kSave ? Block::kBack : Block::kBytes;
        const uint8_t *blocks = a.blocks + ((size_t)bh * a.nc + w.first) * kStep;
        for (; it < nc; ++it) {
            const int s = it & 1;
            if (it >= 2 && !warp_spin_wait(&bar.empty[s], ((it >> 1) - 1) & 1, abort_flag, err)) break;
            if (hook_skips(bh == 0 && v0 == 0, it)) continue;
            uint8_t *st = smem + s * Smem::kStage;
            if (elect_one()) {
                const uint32_t block = out ? Block::kBytes : Block::kQ;
                const int t0 = (w.first + it) * kC;
                const uint8_t *src = blocks + (size_t)it * kStep;
                const uint32_t rest = (w.unit ? Smem::kV : Smem::kStage) - Smem::kK;
                if (kFine || !kSplit) {
                    mbar_expect_tx(&bar.full[s], block + rest);
                    bulk_load(st, src, block, &bar.full[s]);
                } else {                                   // without the second parts
                    constexpr uint32_t kWBytes = Block::kWlo - Block::kW;
                    mbar_expect_tx(&bar.full[s], kBox64 + kWBytes + block - Block::kHdr + rest);
                    bulk_load(st + Block::kT, src + Block::kT, kBox64, &bar.full[s]);
                    bulk_load(st + Block::kW, src + Block::kW, kWBytes, &bar.full[s]);
                    bulk_load(st + Block::kHdr, src + Block::kHdr, block - Block::kHdr, &bar.full[s]);
                }
                if (!w.unit)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        tma_load_4d(st + Smem::kV + x * kBox64, &tm_v, &bar.full[s], v0 + 64 * x, h, t0, b);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x)
                    tma_load_4d(st + Smem::kK + x * kBox64, &tm_k, &bar.full[s], 64 * x, kh, t0, b);
            }
            __syncwarp();
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
            if (n - c * kC < kC) clear_rows(st + Smem::kK, DK / 64 + 2, n - c * kC, lane);
            if (kSave && !w.unit) {
                const float *hdr = reinterpret_cast<const float *>(st + Block::kHdr);
                if (hdr[65] != 0.f) clear_flagged(st + Smem::kV, 2, hdr + 128, lane);
            }
            tc_fence_after();
            if (!w.unit && elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t ad = mnmaj + ((Smem::kV + ks * 2048) >> 4);
                    mma_bf16(tmem + Tm::kX, ad, kmaj + ((Block::kT + ks * 32) >> 4), id_tv, ks > 0);
                    if (kFine)
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
                        const uint64_t wd = kmaj + ((Block::kW + o) >> 4);
                        mma_bf16_ts(tmem + Tm::kX, tmem + Tm::kShi + 8 * ks, wd, id_x, ks > 0 || !w.unit);
                        if (kFine) {
                            mma_bf16_ts(tmem + Tm::kX, tmem + Tm::kSlo + 8 * ks, wd, id_x, 1);
                            mma_bf16_ts(tmem + Tm::kX, tmem + Tm::kShi + 8 * ks,
                                        kmaj + ((Block::kWlo + o) >> 4), id_x, 1);
                        }
                    }
                    if (p == kPieces - 1) mma_commit(&bar.x_full);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (out) {
                if (c > 0 && !warp_spin_wait(&bar.o_free, (c - 1) & 1, abort_flag, err)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < DK / 16; ++ks) {
                        const uint64_t qd = kmaj + ((Block::kQ + (ks / 4) * kBox64 + (ks % 4) * 32) >> 4);
                        mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kShi + 8 * ks, qd, id_x, ks > 0);
                        if (kFine) mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kSlo + 8 * ks, qd, id_x, 1);
                    }
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
                        mma_bf16_ts(tmem + Tm::kZ + 64 * p, tmem + Tm::kXslo + 8 * ks, kd, id_z, 1);
                    }
                    mma_commit(&bar.z_full[p]);
                }
            }
            __syncwarp();
            // (X has been read for this, before the next chunk's takes its place)
            if (again) {
                if (!warp_spin_wait(&bar.xb_ready, c & 1, abort_flag, err)) break;
                tc_fence_after();
            }
            if (elect_one()) {
                if (out) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t pd = kmaj + ((Block::kP + ks * 32) >> 4);
                        mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kXb + 8 * ks, pd, id_x, 1);
                        mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kXblo + 8 * ks, pd, id_x, 1);
                        mma_bf16_ts(tmem + Tm::kO, tmem + Tm::kXb + 8 * ks,
                                    kmaj + ((Block::kPlo + ks * 32) >> 4), id_x, 1);
                    }
                    mma_commit(&bar.o_full);
                }
                mma_commit(&bar.empty[s]);
            }
            __syncwarp();
        }
    } else if (warp < 10) {
        const int wg = (warp - 2) / 4;                     // k columns 64 p + 32 wg ..
        const int v = v0 + 32 * (warp % 4) + lane;
        const bool live = v < w.width;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
        const size_t sbase = (size_t)(32 * wg) * w.width + v;
        float2 S[kPieces][16];
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int k = 64 * p + 32 * wg + 2 * j;
                const float *src = w.from + sbase + (size_t)(64 * p + 2 * j) * w.width;
                S[p][j] = w.unit ? make_float2(k == v ? 1.f : 0.f, k + 1 == v ? 1.f : 0.f)
                          : w.from && live ? make_float2(src[0], src[w.width]) : both(0.f);
            }
        // the operand copies of a piece of S, which itself stays float32; the
        // gradients keep the first.  c: the chunk that starts with it
        auto put_state = [&](int p, int c) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (kFine) split_pair(S[p][j], hi[j], lo[j]);
                else hi[j] = pack_bf16x2(S[p][j].x, S[p][j].y);
            }
            tmem_st16(tl + Tm::kShi + 32 * p + 16 * wg, hi);
            if (kFine) tmem_st16(tl + Tm::kSlo + 32 * p + 16 * wg, lo);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar.s_ready[p]);
            if (kSave && w.keep && live && c < nc)
                keep_row(a.s_save, (size_t)bh * a.nc + w.first + c, a.dv, v, DK, 64 * p + 32 * wg, hi);
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
                uint32_t x[16], hi[16], lo[16];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {           // 16 columns at a time, for the registers
                    tmem_ld16(tl + Tm::kX + 32 * wg + 16 * hf, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int i = 8 * hf + j;
                        const float2 r = *reinterpret_cast<const float2 *>(hdr + 32 * wg + 2 * i);
                        split_pair(mul2(as_pair(x[2 * j], x[2 * j + 1]), r), hi[i], lo[i]);
                    }
                }
                tmem_st16(tl + Tm::kXs + 16 * wg, hi);
                tmem_st16(tl + Tm::kXslo + 16 * wg, lo);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.xs_ready);
                if (out) {                                 // X in two parts, beside the MMAs on Xs
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        tmem_ld16(tl + Tm::kX + 32 * wg + 16 * hf, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            split_pair(as_pair(x[2 * j], x[2 * j + 1]), hi[8 * hf + j], lo[8 * hf + j]);
                    }
                    tmem_st16(tl + Tm::kXb + 16 * wg, hi);
                    tmem_st16(tl + Tm::kXblo + 16 * wg, lo);
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&bar.xb_ready);
                }
            }
            bool ok = true;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                ok = ok && warp_spin_wait(&bar.z_full[p], c & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t z[16];
                    tmem_ld16(tl + Tm::kZ + 64 * p + 32 * wg + 16 * hf, z);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        S[p][8 * hf + j] = fma2(both(eL), S[p][8 * hf + j], as_pair(z[2 * j], z[2 * j + 1]));
                }
                put_state(p, c + 1);
            }
            if (!ok) break;
        }
        if (w.to && live)
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float *dst = w.to + sbase + (size_t)(64 * p + 2 * j) * w.width;
                    dst[0] = S[p][j].x;
                    dst[w.width] = S[p][j].y;
                }
    } else if (again) {
        const int v = v0 + 32 * (warp % 4) + lane;
        const bool live = v < a.dv;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
        if (kSave) {                                       // X in two parts for the gradients
            for (int c = 0; c < nc; ++c) {
                if (!warp_spin_wait(&bar.x_full, c & 1, abort_flag, err)) break;
                tc_fence_after();
                uint32_t hi[2][16], lo[2][16];
#pragma unroll
                for (int q = 0; q < 4; ++q) {              // 16 tokens at a time
                    uint32_t x[16];
                    tmem_ld16(tl + Tm::kX + 16 * q, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        split_pair(as_pair(x[2 * j], x[2 * j + 1]), hi[q / 2][8 * (q & 1) + j],
                                   lo[q / 2][8 * (q & 1) + j]);
                }
                tc_fence_before();
                warp_arrive(&bar.xb_ready);
                if (live)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const size_t chunk = (size_t)bh * a.nc + w.first + c;
                        keep_row(a.x_save, chunk, a.dv, v, 2 * kC, 32 * hf, hi[hf]);
                        keep_row(a.x_save, chunk, a.dv, v, 2 * kC, kC + 32 * hf, lo[hf]);
                    }
            }
        } else {                                           // a thread's tokens of its channel
            const size_t step = (size_t)a.heads * a.dv;
            __nv_bfloat16 *dst = a.out + (((size_t)b * a.tokens + (size_t)w.first * kC) * a.heads + h) * a.dv + v;
            for (int c = 0; c < nc; ++c, dst += kC * step) {
                if (!warp_spin_wait(&bar.o_full, c & 1, abort_flag, err)) break;
                tc_fence_after();
                uint32_t o[2][32];
                tmem_ld32(tl + Tm::kO, o[0]);
                tmem_ld32(tl + Tm::kO + 32, o[1]);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(&bar.o_free);
                const int cnt = live ? n - c * kC : 0;     // rows behind the sequence stay
                __nv_bfloat16 *p = dst;
#pragma unroll
                for (int i = 0; i < kC; ++i, p += step)
                    if (i < cnt) *p = __float2bfloat16_rn(__uint_as_float(o[i / 32][i % 32]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // After an abort, wait (bounded) for the copies still in flight before
    // shared memory goes away and for the MMAs before tensor memory is freed.
    if (*abort_flag && warp == 0 && lane == 0)
        for (int j = max(0, it - 2); j < it; ++j)
            if (!hook_skips(bh == 0 && v0 == 0, j)) mbar_drain(&bar.full[j & 1], (j >> 1) & 1, err);
    if (warp == 1) {
        if (*abort_flag) drain_mmas(&bar.drain, err);
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DK, bool kSplit>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_scan_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  DeltaScanArgs a) {
    forward_walk<DK, kSplit, true, false, kSplit>(tm_k, tm_v, a, whole_walk(a, DK, blockIdx.x, true));
}

// ---- in segments
// With few (sequence, head)s and many chunks most SMs would have no walk.  A
// segment of chunks maps the state before it to the state behind it by
// S -> M S + N, so: first all segments' M (a walk from the identity without
// values) and N (a walk from zero without output) at once, and the first
// segment as it is; then the states between segments, S_{j+1} = M_j S_j + N_j,
// in float32; then all other segments' outputs at once.  Each chunk is walked
// up to three times, but on all SMs: 8192 tokens and 16 heads of 128 in 6
// segments, 431 us a call whole and 231 so, of which the join takes 11.
// Only what a final state depends on is walked in two parts: not the outputs
// of the second pass (it would take 0.2e-3 off their 2.1e-3), but its last
// segment, which is shorter for that.
// starts [segments - 1][BH][dk, dv]: N_j and then the state before segment
// j + 1; units [segments - 2][BH][dk, dk]: M of segments 1 ...
template <int DK, bool kSplit, bool kLast>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_segments_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      DeltaScanArgs a, int bhs) {
    const int slabs = (a.dv + 127) / 128, walks = bhs * slabs;
    const size_t ssize = (size_t)DK * a.dv;
    int cta = blockIdx.x;
    DeltaWalk w;
    if (kLast) {                                           // outputs of segments 1 ...
        const int seg = 1 + cta / walks;
        w = whole_walk(a, DK, cta % walks, true);
        w.from = a.starts + ((size_t)(seg - 1) * bhs + w.bh) * ssize;
        if (seg < a.segments - 1) w.to = nullptr;
        w.first = seg * a.segment;
    } else if (cta < walks) {                              // segment 0
        w = whole_walk(a, DK, cta, true);
        w.to = a.starts + (size_t)w.bh * ssize;
    } else if (cta < walks * (a.segments - 1)) {           // N of segments 1 ...
        const int seg = cta / walks;
        w = whole_walk(a, DK, cta % walks, false);
        w.from = nullptr;
        w.to = a.starts + ((size_t)seg * bhs + w.bh) * ssize;
        w.first = seg * a.segment;
    } else {                                               // M of segments 1 ...
        cta -= walks * (a.segments - 1);
        const int seg = 1 + cta / bhs;
        w.bh = cta % bhs;
        w.v0 = 0;
        w.width = DK;
        w.from = nullptr;
        w.to = a.units + ((size_t)(seg - 1) * bhs + w.bh) * DK * DK;
        w.out = false;
        w.unit = true;
        w.first = seg * a.segment;
    }
    w.last = w.first + a.segment;
    if constexpr (kSplit && kLast) {
        if (!w.to) {
            forward_walk<DK, kSplit, true, false, false>(tm_k, tm_v, a, w);
            return;
        }
    }
    forward_walk<DK, kSplit, true, false, kSplit>(tm_k, tm_v, a, w);
}

// starts[j] <- starts[j] + M starts[j - 1], j = 1 .. joins, with M of units
// [j - 1] (kBack: the transpose of units[joins - j]): a CTA takes 16 columns of
// a (sequence, head)'s states, a warp 16 rows, in three tf32 products as
// square_tile.  A warp's rows of M are its own, so they go from global memory
// to its registers, the next join's while this one is multiplied; only the
// state passes through shared memory, [column][k], its two parts.  4 joins for
// 16 heads of 128: 11 us, most of it the way of M from L2 (8 with every M the
// first; the products do not show).
constexpr int kJoinCols = 16;
template <int DK>
struct DeltaJoinSmem {
    float hi[2][kJoinCols][DK + 4], lo[2][kJoinCols][DK + 4];
};
template <int DK, bool kBack>
__device__ __forceinline__ void join_states(DeltaJoinSmem<DK> &m, float *starts, const float *units,
                                            int bhs, int dv, int joins) {
    const int bh = blockIdx.x / (dv / kJoinCols), col = (blockIdx.x % (dv / kJoinCols)) * kJoinCols;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gr = lane / 4, tq = lane % 4;
    // this thread's accumulators: rows r, r + 8, columns 2 tq, + 1 of two tiles;
    // its columns of M: 16 u + 4 tq .., of which each product takes two
    const int r = 16 * warp + gr;
    const size_t at = (size_t)bh * DK * dv + (size_t)r * dv + col + 2 * tq, step = (size_t)bhs * DK * dv;
    grid_dependency_wait();
    auto get_unit = [&](int j, float (&x)[2][DK / 16][4]) {
        const float *src = units + ((size_t)(kBack ? joins - j : j - 1) * bhs + bh) * DK * DK;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int u = 0; u < DK / 16; ++u) {
                const int row = r + 8 * hf, k = 16 * u + 4 * tq;
                if (kBack) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[hf][u][e] = src[(k + e) * DK + row];
                } else {
                    const float4 v = *reinterpret_cast<const float4 *>(src + row * DK + k);
                    x[hf][u][0] = v.x; x[hf][u][1] = v.y; x[hf][u][2] = v.z; x[hf][u][3] = v.w;
                }
            }
    };
    auto get = [&](int j, float (&x)[2][4]) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                *reinterpret_cast<float2 *>(&x[t][2 * hf]) =
                    *reinterpret_cast<const float2 *>(starts + j * step + at + (size_t)(8 * hf) * dv + 8 * t);
    };
    // x rounded to 11 bits (the split of Veltkamp and Dekker), and what that
    // leaves (of which the product takes 11)
    auto part = [](float x, float &hi, float &lo) {
        const float t = __fmul_rn(x, 8193.f);              // no contraction
        hi = __fsub_rn(t, __fsub_rn(t, x));
        lo = __fsub_rn(x, hi);
    };
    auto mma = [](float (&c)[4], const float (&x)[4], const float (&y)[2]) {
        asm volatile(
            "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])),
              "r"(__float_as_uint(x[3])), "r"(__float_as_uint(y[0])), "r"(__float_as_uint(y[1])));
    };
    float M[2][2][DK / 16][4], s[2][4], next[2][4];
    auto join = [&](int j, float (&cur)[2][DK / 16][4], float (&ahead)[2][DK / 16][4]) {
        if (j < joins) get_unit(j + 1, ahead);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = 8 * t + 2 * tq + (e & 1), k = r + 8 * (e >> 1);
                part(s[t][e], m.hi[j & 1][c][k], m.lo[j & 1][c][k]);
            }
        __syncthreads();                                   // and all are done with the state before the last
        float lo1[2][4] = {}, lo2[2][4] = {};              // products of the low parts
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = next[t][e];
        if (j < joins) get(j + 1, next);
#pragma unroll
        for (int u = 0; u < DK / 16; ++u) {
            float bh4[2][4], bl4[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                *reinterpret_cast<float4 *>(bh4[t]) =
                    *reinterpret_cast<const float4 *>(&m.hi[j & 1][8 * t + gr][16 * u + 4 * tq]);
                *reinterpret_cast<float4 *>(bl4[t]) =
                    *reinterpret_cast<const float4 *>(&m.lo[j & 1][8 * t + gr][16 * u + 4 * tq]);
            }
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                float ah[4], al[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) part(cur[e & 1][u][h + (e >> 1)], ah[e], al[e]);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float yh[2] = {bh4[t][h], bh4[t][h + 1]}, yl[2] = {bl4[t][h], bl4[t][h + 1]};
                    mma(s[t], ah, yh);
                    mma(lo1[t], ah, yl);
                    mma(lo2[t], al, yh);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                s[t][2 * hf] += lo1[t][2 * hf] + lo2[t][2 * hf];
                s[t][2 * hf + 1] += lo1[t][2 * hf + 1] + lo2[t][2 * hf + 1];
                *reinterpret_cast<float2 *>(starts + j * step + at + (size_t)(8 * hf) * dv + 8 * t) =
                    make_float2(s[t][2 * hf], s[t][2 * hf + 1]);
            }
    };
    get_unit(1, M[1]);
    get(0, s);
    get(1, next);
    for (int j = 1; j <= joins; j += 2) {
        join(j, M[1], M[0]);
        if (j < joins) join(j + 1, M[0], M[1]);
    }
}
template <int DK>
__global__ void __launch_bounds__(2 * DK)
delta_join_kernel(float *starts, float *back, const float *units, int bhs, int dv, int joins) {
    __shared__ __align__(16) DeltaJoinSmem<DK> m;
    if (blockIdx.y) join_states<DK, true>(m, back, units, bhs, dv, joins);
    else join_states<DK, false>(m, starts, units, bhs, dv, joins);
}
template <int DK>
cudaError_t launch_join(float *starts, float *back, const float *units, int bhs, int dv, int joins,
                        cudaStream_t stream) {
    KernelTimer timer("delta_join", stream);
    count_launch();
    return launch_overlapped(delta_join_kernel<DK>, dim3((unsigned)(bhs * (dv / kJoinCols)), back ? 2 : 1),
                             dim3(2 * DK), 0, stream, starts, back, units, bhs, dv, joins);
}

// ------------------------------------------------------------------ reverse scan
// The gradient's walk, last chunk first.  D is the gradient of the state
// behind a chunk; with dO the output's gradient
//   dX = P^T dO + diag(e^{G_L - G}) K D,   dV = T^^T dX,
//   D <- e^{G_L} D + Q~^T dO - W^T dX,
// transposed and laid out as in the forward walk (v channels as lanes, D in
// the chain's registers in float32, its operand copy and, for W, dX in one
// bf16 part, P and Q~ in two).  Per chunk, in the order of the MMAs:
//   Y1^T = dO^T P;  Y2^T = D^T K^T       [needs D]   -> chain: dX = Y1 + rest Y2
//   Z^T  = dO^T Q~                       (while the chain rounds dX)
//   Z^T += dX^T (-W)                     [needs dX]  -> chain: D = e^{G_L} D + Z
//   dV^T = dX^T T^                       (while the chain rounds D)
// D is kept for every chunk (d_save, as S^T in the forward walk), and what dV
// leaves behind its bf16 result (v_lo), for dbeta.
struct DeltaReverseBars {
    uint64_t full[2], empty[2], d_ready[2], z_full[2], y_full, dx_ready, lo_ready, v_full, v_free, drain;
    uint32_t tmem_slot;
    int abort_flag;
};

template <int DK>
struct DeltaReverseSmem {
    using Block = DeltaBlock<DK, false>;
    static constexpr uint32_t kK = Block::kBack;
    static constexpr uint32_t kDo = kK + Block::kKB * kBox64;
    static constexpr uint32_t kStage = kDo + 2 * kBox64;
    static constexpr uint32_t kOut = 2 * kStage;          // dV, 64 tokens x 128 channels
    static constexpr uint32_t kBars = kOut + 2 * kBox64;
    static constexpr uint32_t kBytes = kBars + 256;
    static_assert(sizeof(DeltaReverseBars) <= 256 && kBytes <= 227 * 1024, "shared memory");
};

struct DeltaReverseArgs {
    const uint8_t *blocks;
    const int *lengths;
    __nv_bfloat16 *d_save, *v_lo;          // D^T of every chunk; dV^T's second part (keep_row)
    int heads, key_heads, tokens, nc, dv;
    unsigned *err;
};

template <int DK>
__device__ __forceinline__ void reverse_walk(const CUtensorMap &tm_k, const CUtensorMap &tm_do,
                                             const CUtensorMap &tm_dv, const DeltaReverseArgs &a,
                                             const DeltaWalk &w) {
    using Smem = DeltaReverseSmem<DK>;
    using Block = DeltaBlock<DK, false>;
    constexpr int kPieces = DK / 64;
    constexpr uint32_t kD = 0, kZ = DK / 2, kY1 = kZ + DK, kY2 = kY1 + 64, kDx = kY2 + 64, kDxlo = kDx + 32, kDv = kDxlo + 32;
    static_assert(kDv + 64 <= 512, "tensor memory");
    extern __shared__ __align__(1024) uint8_t smem[];
    DeltaReverseBars &bar = *reinterpret_cast<DeltaReverseBars *>(smem + Smem::kBars);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int bh = w.bh, v0 = w.v0;
    const int b = bh / a.heads, h = bh % a.heads;
    unsigned *err = a.err;
    int *abort_flag = &bar.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
            mbar_init(&bar.d_ready[s], kChainWarps);
            mbar_init(&bar.z_full[s], 1);
        }
        mbar_init(&bar.y_full, 1);
        mbar_init(&bar.dx_ready, kChainWarps);
        mbar_init(&bar.lo_ready, kChainWarps);
        mbar_init(&bar.v_full, 1);
        mbar_init(&bar.v_free, 4);
        mbar_init(&bar.drain, 1);
        bar.abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_do);
        tma_prefetch_desc(&tm_dv);
    }
    if (warp == 1) {
        tmem_alloc(&bar.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                           // all 512 columns, as above
    grid_dependency_wait();
    const int n = delta_tokens_of(a.lengths, b, a.tokens);
    const int top = min(w.last, (n + kC - 1) / kC), nc = max(0, top - w.first);   // from chunk top - 1 on

    int it = 0;                                            // chunks whose copies were issued
    if (warp == 0) {
        const int kh = h / (a.heads / a.key_heads);
        const uint8_t *blocks = a.blocks + (size_t)bh * a.nc * Block::kBack;
        for (; it < nc; ++it) {
            const int s = it & 1, c = top - 1 - it;
            if (it >= 2 && !warp_spin_wait(&bar.empty[s], ((it >> 1) - 1) & 1, abort_flag, err)) break;
            if (hook_skips(bh == 0 && v0 == 0, it)) continue;
            uint8_t *st = smem + s * Smem::kStage;
            if (elect_one()) {
                mbar_expect_tx(&bar.full[s], Smem::kStage);
                bulk_load(st, blocks + (size_t)c * Block::kBack, Block::kBack, &bar.full[s]);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    tma_load_4d(st + Smem::kDo + x * kBox64, &tm_do, &bar.full[s], v0 + 64 * x, h, c * kC, b);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x)
                    tma_load_4d(st + Smem::kK + x * kBox64, &tm_k, &bar.full[s], 64 * x, kh, c * kC, b);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        constexpr uint32_t id_do = idesc_bf16(128, 64, 1, 1);   // A: dO tile, v contiguous
        constexpr uint32_t id_k = idesc_bf16(128, 64, 0, 0);    // B: K tile, k contiguous
        constexpr uint32_t id_w = idesc_bf16(128, 64, 0, 1);    // B: W, T^, columns contiguous
        for (int u = 0; u < nc; ++u) {
            const int s = u & 1, cnt = n - (top - 1 - u) * kC;
            uint8_t *st = smem + s * Smem::kStage;
            const uint64_t kmaj = smem_desc_sw128(smem_u32(st), 16, 1024);
            const uint64_t mnmaj = smem_desc_sw128(smem_u32(st), kBox64, 1024);
            if (!warp_spin_wait(&bar.full[s], (u >> 1) & 1, abort_flag, err)) break;
            if (cnt < kC) clear_rows(st + Smem::kK, DK / 64 + 2, cnt, lane);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t ad = mnmaj + ((Smem::kDo + ks * 2048) >> 4);
                    mma_bf16(tmem + kY1, ad, mnmaj + ((Block::kP + ks * 2048) >> 4), id_do, ks > 0);
                    mma_bf16(tmem + kY1, ad, mnmaj + ((Block::kPlo + ks * 2048) >> 4), id_do, 1);
                }
            }
            __syncwarp();
            bool ok = true;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                ok = ok && warp_spin_wait(&bar.d_ready[p], u & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4)
                        mma_bf16_ts(tmem + kY2, tmem + kD + 32 * p + 8 * k4,
                                    kmaj + ((Smem::kK + p * kBox64 + k4 * 32) >> 4), id_k, p + k4 > 0);
                    if (p == kPieces - 1) mma_commit(&bar.y_full);
                    // (a piece of D that is ready has been read from Z)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = mnmaj + ((Smem::kDo + ks * 2048) >> 4);
                        mma_bf16(tmem + kZ + 64 * p, ad,
                                 mnmaj + ((Block::kQ + p * kBox64 + ks * 2048) >> 4), id_do, ks > 0);
                        mma_bf16(tmem + kZ + 64 * p, ad,
                                 mnmaj + ((Block::kQlo + p * kBox64 + ks * 2048) >> 4), id_do, 1);
                    }
                }
                __syncwarp();
            }
            if (!ok || !warp_spin_wait(&bar.dx_ready, u & 1, abort_flag, err)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ts(tmem + kZ + 64 * p, tmem + kDx + 8 * ks,
                                    mnmaj + ((Block::kW + p * kBox64 + ks * 2048) >> 4), id_w, 1);
                    mma_commit(&bar.z_full[p]);
                }
            }
            __syncwarp();
            if (w.keep) {
                if (u > 0 && !warp_spin_wait(&bar.v_free, (u - 1) & 1, abort_flag, err)) break;
                if (!warp_spin_wait(&bar.lo_ready, u & 1, abort_flag, err)) break;
                tc_fence_after();
            }
            if (elect_one()) {
                if (w.keep) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t td = mnmaj + ((Block::kT + ks * 2048) >> 4);
                        mma_bf16_ts(tmem + kDv, tmem + kDx + 8 * ks, td, id_w, ks > 0);
                        mma_bf16_ts(tmem + kDv, tmem + kDxlo + 8 * ks, td, id_w, 1);
                    }
                    mma_commit(&bar.v_full);
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
        const size_t sbase = (size_t)(32 * wg) * a.dv + v;
        float2 D[kPieces][16];
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float *src = w.from + sbase + (size_t)(64 * p + 2 * j) * a.dv;
                D[p][j] = w.from && live ? make_float2(src[0], src[a.dv]) : both(0.f);
            }
        // the operand copy of a piece of D, kept for chunk c (the one in front of it)
        auto put_grad = [&](int p, int c) {
            uint32_t hi[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) hi[j] = pack_bf16x2(D[p][j].x, D[p][j].y);
            tmem_st16(tl + kD + 32 * p + 16 * wg, hi);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar.d_ready[p]);
            if (w.keep && live && c >= w.first)
                keep_row(a.d_save, (size_t)bh * a.nc + c, a.dv, v, DK, 64 * p + 32 * wg, hi);
        };
#pragma unroll
        for (int p = 0; p < kPieces; ++p) put_grad(p, top - 1);
        for (int u = 0; u < nc; ++u) {
            const int s = u & 1;
            const float *hdr = reinterpret_cast<const float *>(smem + s * Smem::kStage + Block::kHdr);
            if (!warp_spin_wait(&bar.full[s], (u >> 1) & 1, abort_flag, err)) break;
            const float eL = hdr[64];
            if (!warp_spin_wait(&bar.y_full, u & 1, abort_flag, err)) break;
            tc_fence_after();
            {
                uint32_t dx[16], lo[16];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {           // 16 columns at a time, for the registers
                    uint32_t y1[16], y2[16];
                    tmem_ld16(tl + kY1 + 32 * wg + 16 * hf, y1);
                    tmem_ld16(tl + kY2 + 32 * wg + 16 * hf, y2);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 r = *reinterpret_cast<const float2 *>(hdr + 32 * wg + 16 * hf + 2 * j);
                        split_pair(fma2(r, as_pair(y2[2 * j], y2[2 * j + 1]), as_pair(y1[2 * j], y1[2 * j + 1])),
                                   dx[8 * hf + j], lo[8 * hf + j]);
                    }
                }
                tmem_st16(tl + kDx + 16 * wg, dx);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.dx_ready);
                tmem_st16(tl + kDxlo + 16 * wg, lo);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.lo_ready);
            }
            bool ok = true;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                ok = ok && warp_spin_wait(&bar.z_full[p], u & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t z[16];
                    tmem_ld16(tl + kZ + 64 * p + 32 * wg + 16 * hf, z);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        D[p][8 * hf + j] = fma2(both(eL), D[p][8 * hf + j], as_pair(z[2 * j], z[2 * j + 1]));
                }
                put_grad(p, top - 2 - u);
            }
            if (!ok) break;
        }
        if (w.to && live)
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float *dst = w.to + sbase + (size_t)(64 * p + 2 * j) * a.dv;
                    dst[0] = D[p][j].x;
                    dst[a.dv] = D[p][j].y;
                }
    } else if (w.keep) {
        const int col = 32 * (warp % 4) + lane, tid = threadIdx.x - 320;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
        for (int u = 0; u < nc; ++u) {
            const bool ok = warp_spin_wait(&bar.v_full, u & 1, abort_flag, err);
            uint32_t o[64];
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld16(tl + kDv + 16 * q, *reinterpret_cast<uint32_t (*)[16]>(&o[16 * q]));
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(&bar.v_free);
            }
            if (tid == 0) tma_store_wait_read();
            if (named_barrier_or(1, 128, !ok)) break;
            put_channel(smem + Smem::kOut, col, o);        // zeros behind the sequence
            fence_async_shared();
            named_barrier(1, 128);
            if (v0 + col < a.dv)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    keep_row(a.v_lo, (size_t)bh * a.nc + top - 1 - u, a.dv, v0 + col, kC, 32 * hf,
                             *reinterpret_cast<const uint32_t (*)[16]>(&o[16 * hf]));
            if (tid == 0) {
                for (int x = 0; x < 2; ++x)
                    if (v0 + 64 * x < a.dv)
                        tma_store_4d(&tm_dv, smem + Smem::kOut + x * kBox64, v0 + 64 * x, h,
                                     (top - 1 - u) * kC, b);
                tma_store_commit();
            }
        }
        if (tid == 0) tma_store_wait_read();
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 0 && lane == 0)             // as in the forward walk
        for (int j = max(0, it - 2); j < it; ++j)
            if (!hook_skips(bh == 0 && v0 == 0, j)) mbar_drain(&bar.full[j & 1], (j >> 1) & 1, err);
    if (warp == 1) {
        if (*abort_flag) drain_mmas(&bar.drain, err);
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The backward's two walks.  Neither needs the other, and each has a CTA per
// (sequence, head) and 128 channels only, so they share a launch: the first
// half of the CTAs walks forward and keeps X^T and S^T, the second back.
template <int DK>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_walks_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_dv,
                   DeltaScanArgs f, DeltaReverseArgs r) {
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half)
        forward_walk<DK, false, false, true, false>(tm_k, tm_v, f, whole_walk(f, DK, blockIdx.x, false));
    else reverse_walk<DK>(tm_k, tm_do, tm_dv, r, whole_walk(f, DK, blockIdx.x - half, false));
}

// Both in segments.  Back through a segment the gradient of the state goes by
// D -> M^T D + N', so one set of transitions serves both ways, in one bf16
// part as the walks that go on from them (the joins between are float32).
// starts [segments - 1][BH][dk, dv] as above; back [segments - 1]: D behind
// segment segments - 2 first; units [segments - 2][BH][dk, dk].
struct DeltaBackSegments {
    int segments, segment;                                   // how many, chunks of each
    float *starts, *back, *units;
};
template <int DK>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_walks_segments_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_dv,
                            DeltaScanArgs f, DeltaReverseArgs r, DeltaBackSegments x, int bhs, int last) {
    const int walks = bhs * ((f.dv + 127) / 128), ends = walks * (x.segments - 1);
    const size_t ssize = (size_t)DK * f.dv;
    int cta = blockIdx.x;
    DeltaWalk w;
    auto cut = [&](int seg) {
        w.first = seg * x.segment;
        w.last = w.first + x.segment;
    };
    if (cta >= ends && cta < 2 * ends) {                     // back: behind segments .. 1, 0
        cta -= ends;
        const int i = cta / walks + last;
        w = whole_walk(f, DK, cta % walks, false);
        if (last) w.from = x.back + ((size_t)(i - 1) * bhs + w.bh) * ssize;
        else w.to = x.back + ((size_t)i * bhs + w.bh) * ssize;
        w.keep = last || i == 0;
        cut(x.segments - 1 - i);
        reverse_walk<DK>(tm_k, tm_do, tm_dv, r, w);
        return;
    }
    if (cta < ends) {
        const int seg = cta / walks + last;
        w = whole_walk(f, DK, cta % walks, false);
        if (last) w.from = x.starts + ((size_t)(seg - 1) * bhs + w.bh) * ssize;
        else w.to = x.starts + ((size_t)seg * bhs + w.bh) * ssize;
        w.keep = last || seg == 0;
        cut(seg);
    } else {                                                 // M
        cta -= 2 * ends;
        const int seg = 1 + cta / bhs;
        w.bh = cta % bhs;
        w.v0 = 0;
        w.width = DK;
        w.from = nullptr;
        w.to = x.units + ((size_t)(seg - 1) * bhs + w.bh) * DK * DK;
        w.out = w.keep = false;
        w.unit = true;
        cut(seg);
    }
    forward_walk<DK, false, false, true, false>(tm_k, tm_v, f, w);
}

// ------------------------------------------------------------------ gradients
// dq, dk, dg and dbeta of a chunk from what the two walks left: X^T and S^T
// (the state before the chunk), dV and D^T (the gradient of the state behind
// it).  With dV = T^^T dX, which is b r of the float32 form (delta_simt.cu):
//   A_ij = scale (do_i . x_j) e^{G_i - G_j}, i >= j;   B_ij = -(dv_i . x_j) e^{G_i - G_j}, i > j
//   dq = scale e^G (dO S^T) + A K
//   dk = -e^G (dV S^T) + e^{G_L - G} (X D^T) + A^T Q + (B + B^T) K
//   dbeta = (dv . x) / b^2;  dg as in delta_simt.cu.
// Of a token that writes nothing x is 0 and dV the gradient of x, r, which B
// and dk leave out (b r is 0); dbeta = r . (v - k S before it), of which
// r . k S are that row's sums of E and of k (r S^T) (S.none), and dv is 0.
// X comes in two parts, A and B are made two; dV is read as it left and, for
// dbeta, with its second part (dot products by the row warps: there is no room
// for another tile).  E, from which dg is summed, takes A and B in float32.
// A chunk's 64 rows fill half of a tcgen05 tile, so two operands share one:
// rows 0-63 belong to the queries (dO, Q, A), rows 64-127 to the keys
// (dV, K, B), and a thread of the epilogue owns a row of dq or of dk:
//   pair columns  [dO; dV] X^T and [Q; K] K^T        (64 each; X, A, B by parts)
//   C1 = [dO; dV] S^T,  C2 = [*; X] D^T              (summed over v, 64 at a time)
//   C3 = [A; B] K,      C4 = [*; A^T] Q + [*; B^T] K (C4 where the pairs were)
// (*: whatever precedes the operand in shared memory; those rows are not read.)
// Persistent, a CTA an SM: the copies of the next chunk run beside the pairs
// and the epilogue of this one (a CTA a chunk, 2048 chunks of 128 x 128: 175
// us, persistent 100; 131 with the second parts: A's and B's 13, X's 11, dV's 5).
constexpr int kGradTcThreads = 352;        // warps 0-7 rows, 8 copies, 9 MMAs, 10 gates and sums

struct DeltaGradTcBars {
    uint64_t full[2], lo_full[2], empty[2], keys[2], keys_free[2], gates[2], done[2];
    uint64_t pair_full, ab_ready, ablo_ready, c_full, acc_free, drain;
    uint32_t tmem_slot;
    int abort_flag;
    // By turns of two items, so that warp 10 prepares the one after next and
    // closes the last one while the row warps work.
    struct Gates {
        DecaySums G;
        float beta[kC], rest[kC], e[kC], since[kC];        // e^{G_L - G}, e^G, e^{G_i - G_r}
        float across[3][kC];                               // as in the prep
    } gate[2];
    struct Sums {
        float row[2][2][kC];               // of E: [queries, keys][column half]
        float col[8][32];                  // by warp: its column half
        float inter[2][2][kC], ahead[2][kC], db[kC], sd[8];
        float none[2][kC];                 // [column half]: - r . k S, where nothing is written
        float lo[2][kC];                   // [channel half]: dV's second part . x
    } sum[2];
};
template <int DK>
struct DeltaGradTcSmem {
    static constexpr uint32_t kKB = DK / 64;
    // two buffers of keys: a Q and a K box by turns ([Q; K] is 128 rows of one
    // operand, and each alone has its column blocks two boxes apart; dq and dk
    // leave from where a thread read its row of them), then the tiles A, B;
    // the second parts of X by stages while A and B are not yet formed
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kBox64;
    static constexpr uint32_t kKeyStep = 2 * kBox64;
    static constexpr uint32_t kKeys = 2 * kKB * kBox64;
    static constexpr uint32_t kA = 2 * kKeys;
    static constexpr uint32_t kB = kA + kBox64;
    static constexpr uint32_t kStage0 = kB + kBox64;
    // a stage of 64 v channels: dO, dV, X^T, S^T, D^T
    static constexpr uint32_t kDo = 0, kDv = kBox64, kX = 2 * kBox64, kS = 3 * kBox64;
    static constexpr uint32_t kD = kS + kKB * kBox64;
    static constexpr uint32_t kStage = kD + kKB * kBox64;
    // float decay[64][65] = e^{G_i - G_j}, i >= j; the second parts of A and B
    // once they have been formed with it
    static constexpr uint32_t kDecay = kStage0 + 2 * kStage;
    static constexpr uint32_t kBars = kDecay + 16640;
    static constexpr uint32_t kBytes = kBars + ((sizeof(DeltaGradTcBars) + 127) & ~127u);
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct DeltaGradTcArgs {
    const __nv_bfloat16 *v, *g, *beta;
    const __nv_bfloat16 *x, *s, *d, *v_lo;                 // X^T (two parts), S^T, D^T, dV^T's second part
    const int *lengths;
    __nv_bfloat16 *dq, *dk_, *dv_, *dg, *dbeta;
    float *dq_wide, *dk_wide;
    float scale;
    int heads, key_heads, tokens, nc, dv, items;
    unsigned *err;
};

template <int DK>
__global__ void __launch_bounds__(kGradTcThreads, 1)
delta_grad_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_dv,
                     const __grid_constant__ CUtensorMap tm_dq,
                     const __grid_constant__ CUtensorMap tm_dk, DeltaGradTcArgs a) {
    using Smem = DeltaGradTcSmem<DK>;
    constexpr int kKB = DK / 64;
    constexpr uint32_t kPd = 0, kPk = 64, kC4 = 0, kC1 = 128, kC2 = kC1 + DK, kC3 = kC2 + DK;
    extern __shared__ __align__(1024) uint8_t smem[];
    DeltaGradTcBars &m = *reinterpret_cast<DeltaGradTcBars *>(smem + Smem::kBars);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
    const bool shared_keys = a.heads != a.key_heads;
    const int nv = a.dv / 64;
    unsigned *err = a.err;
    int *abort_flag = &m.abort_flag;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.full[s], 1);
            mbar_init(&m.lo_full[s], 1);
            mbar_init(&m.empty[s], 9);                     // the MMAs and 8 warps
            mbar_init(&m.keys[s], 1);
            mbar_init(&m.keys_free[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.gates[s], 1);
            mbar_init(&m.done[s], 8);
        }
        mbar_init(&m.pair_full, 1);
        mbar_init(&m.ab_ready, 8);
        mbar_init(&m.ablo_ready, 8);
        mbar_init(&m.c_full, 1);
        mbar_init(&m.acc_free, 8);
        mbar_init(&m.drain, 1);
        m.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&m.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                           // all 512 columns, as above
    grid_dependency_wait();

    // the chunk of an item, and how many of its tokens belong to the sequence
    struct Item {
        int bh, b, h, kh, t0, cnt;
    };
    auto item_of = [&](int i) {
        Item w;
        w.bh = i / a.nc;
        w.b = w.bh / a.heads;
        w.h = w.bh % a.heads;
        w.kh = w.h / (a.heads / a.key_heads);
        w.t0 = (i % a.nc) * kC;
        w.cnt = min(kC, delta_tokens_of(a.lengths, w.b, a.tokens) - w.t0);
        return w;
    };

    float (*decay)[kC + 1] = reinterpret_cast<float (*)[kC + 1]>(smem + Smem::kDecay);
    int it = 0, kit = 0, lit = 0;                          // stages, keys and second parts issued
    if (warp == 8) {
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
            const Item w = item_of(i);
            if (w.cnt <= 0) continue;
            const int kb = kit & 1;
            if (kit >= 2) ok = warp_spin_wait(&m.keys_free[kb], ((kit >> 1) - 1) & 1, abort_flag, err);
            if (!ok) break;
            if (elect_one()) {
                uint8_t *ks = smem + kb * Smem::kKeys;
                mbar_expect_tx(&m.keys[kb], Smem::kKeys);
#pragma unroll
                for (int x = 0; x < kKB; ++x) {
                    tma_load_4d(ks + Smem::kQ + x * Smem::kKeyStep, &tm_q, &m.keys[kb], 64 * x, w.kh, w.t0, w.b);
                    tma_load_4d(ks + Smem::kK + x * Smem::kKeyStep, &tm_k, &m.keys[kb], 64 * x, w.kh, w.t0, w.b);
                }
            }
            __syncwarp();
            ++kit;
            const size_t first = (size_t)i * nv;           // block of 64 channels
            for (int u = 0; u < nv; ++u, ++it) {
                const int s = it & 1;
                if (it >= 2) ok = warp_spin_wait(&m.empty[s], ((it >> 1) - 1) & 1, abort_flag, err);
                if (!ok) break;
                if (hook_skips(blockIdx.x == 0, it)) continue;
                uint8_t *st = smem + Smem::kStage0 + s * Smem::kStage;
                if (elect_one()) {
                    mbar_expect_tx(&m.full[s], Smem::kStage);
                    tma_load_4d(st + Smem::kDo, &tm_do, &m.full[s], 64 * u, w.h, w.t0, w.b);
                    tma_load_4d(st + Smem::kDv, &tm_dv, &m.full[s], 64 * u, w.h, w.t0, w.b);
                    bulk_load(st + Smem::kX, a.x + (first + u) * (2 * 64 * kC), kBox64, &m.full[s]);
                    bulk_load(st + Smem::kS, a.s + (first + u) * (64 * DK), kKB * kBox64, &m.full[s]);
                    bulk_load(st + Smem::kD, a.d + (first + u) * (64 * DK), kKB * kBox64, &m.full[s]);
                }
                __syncwarp();
                // X's second parts of an item's first stages go where A and B
                // of the last item were, once they have been read
                if (u < min(nv, 2) - 1) continue;
                if (u < 2 && kit > 1) ok = warp_spin_wait(&m.c_full, kit & 1, abort_flag, err);
                if (!ok) break;
                for (; lit <= it; ++lit)
                    if (elect_one()) {
                        uint64_t *bar = &m.lo_full[lit & 1];
                        mbar_expect_tx(bar, kBox64);
                        bulk_load(smem + Smem::kA + (lit & 1) * kBox64,
                                  a.x + ((first + u - (it - lit)) * 2 + 1) * (64 * kC), kBox64, bar);
                    }
                __syncwarp();
            }
        }
    } else if (warp == 9) {
        constexpr uint32_t id_kk = idesc_bf16(128, 64, 0, 0);
        constexpr uint32_t id_px = idesc_bf16(128, 64, 0, 1);
        constexpr uint32_t id_c1 = idesc_bf16(128, DK, 0, 1);
        constexpr uint32_t id_c2 = idesc_bf16(128, DK, 1, 1);
        const uint32_t base = smem_u32(smem);
        const uint64_t plain = smem_desc_plain(base, 128, 1024);   // X^T, S^T, D^T blocks
        const uint64_t akm = smem_desc_sw128(base, 16, 1024), amn = smem_desc_sw128(base, kBox64, 1024);
        int g = 0, n = 0;                                  // stages and items so far
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
            const Item w = item_of(i);
            if (w.cnt <= 0) continue;
            const uint32_t ko = (n & 1) * Smem::kKeys;
            const uint64_t kmaj = akm + (ko >> 4);
            const uint64_t keymn = smem_desc_sw128(base + ko, Smem::kKeyStep, 1024);
            ok = warp_spin_wait(&m.keys[n & 1], (n >> 1) & 1, abort_flag, err);
            if (ok && w.cnt < kC) clear_rows(smem + ko + Smem::kQ, 2 * kKB, w.cnt, lane);
            if (ok && n > 0) ok = warp_spin_wait(&m.acc_free, (n - 1) & 1, abort_flag, err);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int x = 0; x < kKB; ++x)
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        const uint32_t o = x * Smem::kKeyStep + k4 * 32;
                        mma_bf16(tmem + kPk, kmaj + ((Smem::kQ + o) >> 4), kmaj + ((Smem::kK + o) >> 4),
                                 id_kk, x + k4 > 0);
                    }
            }
            __syncwarp();
            for (int u = 0; u < nv; ++u, ++g) {
                const int s = g & 1;
                const uint32_t so = (Smem::kStage0 + s * Smem::kStage) >> 4;
                const uint64_t kst = akm + so, kept = plain + so;
                const uint64_t xlo = plain + ((Smem::kA + s * kBox64) >> 4);
                ok = warp_spin_wait(&m.full[s], (g >> 1) & 1, abort_flag, err) &&
                     warp_spin_wait(&m.lo_full[s], (g >> 1) & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t dd = kst + ((Smem::kDo + ks * 32) >> 4);
                        mma_bf16(tmem + kPd, dd, kept + ((Smem::kX + ks * 256) >> 4), id_px, u + ks > 0);
                        mma_bf16(tmem + kPd, dd, xlo + ((ks * 256) >> 4), id_px, 1);
                    }
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)         // the box in front fills the rows that are not read
                        mma_bf16(tmem + kC2, xlo - (kBox64 >> 4) + ((ks * 256) >> 4),
                                 kept + ((Smem::kD + ks * 256) >> 4), id_c2, u + ks > 0);
                    if (u == nv - 1) mma_commit(&m.pair_full);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(tmem + kC1, kst + ((Smem::kDo + ks * 32) >> 4),
                                 kept + ((Smem::kS + ks * 256) >> 4), id_c1, u + ks > 0);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)         // dV fills the rows that are not read
                        mma_bf16(tmem + kC2, kept + ((Smem::kDv + ks * 256) >> 4),
                                 kept + ((Smem::kD + ks * 256) >> 4), id_c2, 1);
                    mma_commit(&m.empty[s]);
                }
                __syncwarp();
            }
            ok = ok && warp_spin_wait(&m.ab_ready, n & 1, abort_flag, err);
            if (!ok) break;
            tc_fence_after();
            // first and second parts of A and B; the box in front of A (of B)
            // fills the rows that are not read
            auto chunk_products = [&](uint32_t tiles, bool first) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t qb = keymn + ((Smem::kQ + ks * 2048) >> 4);
                    const uint64_t kb = keymn + ((Smem::kK + ks * 2048) >> 4);
                    mma_bf16(tmem + kC3, akm + ((tiles + ks * 32) >> 4), kb, id_c1, !first || ks > 0);
                    mma_bf16(tmem + kC4, amn + ((tiles - kBox64 + ks * 2048) >> 4), qb, id_c2, !first || ks > 0);
                    mma_bf16(tmem + kC4, amn + ((tiles + ks * 2048) >> 4), kb, id_c2, 1);
                }
            };
            if (elect_one()) chunk_products(Smem::kA, true);
            __syncwarp();
            ok = warp_spin_wait(&m.ablo_ready, n & 1, abort_flag, err);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                chunk_products(Smem::kDecay, false);
                mma_commit(&m.c_full);
            }
            __syncwarp();
            ++n;
        }
    } else if (warp == 10) {
        // gates of the items ahead; rows without a sequence; dq and dk out, dg
        // and dbeta of the items behind
        int ahead_i = blockIdx.x, ahead_n = 0;
        auto prepare = [&]() {
            for (; ahead_i < a.items; ahead_i += gridDim.x) {
                const Item w = item_of(ahead_i);
                const int room = min(kC, a.tokens - w.t0);
                const size_t row0 = (size_t)w.b * a.tokens + w.t0;
                if (w.cnt <= 0) {                          // no gradients here
                    for (int r1 = 0; r1 < room; ++r1) {
                        const size_t r = (row0 + r1) * a.heads + w.h;
                        for (int j = lane; j < a.dv; j += 32) a.dv_[r * a.dv + j] = from_f32<__nv_bfloat16>(0.f);
                        for (int j = lane; j < DK; j += 32) {
                            if (shared_keys) {
                                a.dq_wide[r * DK + j] = 0.f;
                                a.dk_wide[r * DK + j] = 0.f;
                            } else {
                                a.dq[r * DK + j] = from_f32<__nv_bfloat16>(0.f);
                                a.dk_[r * DK + j] = from_f32<__nv_bfloat16>(0.f);
                            }
                        }
                        if (lane == 0) {
                            a.dg[r] = from_f32<__nv_bfloat16>(0.f);
                            a.dbeta[r] = from_f32<__nv_bfloat16>(0.f);
                        }
                    }
                    continue;
                }
                DeltaGradTcBars::Gates &G = m.gate[ahead_n & 1];
                const size_t at = row0 * a.heads + w.h;
                float g[2], bt[2];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int t = lane + 32 * v;
                    g[v] = t < w.cnt ? log_decay(to_f32(a.g[at + (size_t)t * a.heads])) : 0.f;
                    bt[v] = t < w.cnt ? to_f32(a.beta[at + (size_t)t * a.heads]) : 1.f;
                    if (writes_nothing(bt[v])) bt[v] = 0.f;
                }
                sum_decays(G.G, lane, g[0], g[1]);
                __syncwarp();
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int t = lane + 32 * v;
                    G.beta[t] = bt[v];
                    G.rest[t] = expf(G.G.until(t, 3));
                    G.e[t] = expf(G.G.since_start(t));
                    G.since[t] = expf(G.G.in[t].x + G.G.in[t].y);
#pragma unroll
                    for (int r = 1; r < 4; ++r)
                        if (t < 16 * r) G.across[r - 1][t] = expf(G.G.until(t, r - 1));
                }
                warp_arrive(&m.gates[ahead_n & 1]);
                ++ahead_n;
                ahead_i += gridDim.x;
                return;
            }
        };
        prepare();
        prepare();
        int n = 0;
        for (int i = blockIdx.x; i < a.items; i += gridDim.x) {
            const Item w = item_of(i);
            if (w.cnt <= 0) continue;
            if (!warp_spin_wait(&m.done[n & 1], (n >> 1) & 1, abort_flag, err)) break;
            const int room = min(kC, a.tokens - w.t0);
            const size_t row0 = (size_t)w.b * a.tokens + w.t0;
            uint8_t *ks = smem + (n & 1) * Smem::kKeys;
            if (!shared_keys && elect_one()) {
#pragma unroll
                for (int x = 0; x < kKB; ++x) {
                    tma_store_4d(&tm_dq, ks + Smem::kQ + x * Smem::kKeyStep, 64 * x, w.kh, w.t0, w.b);
                    tma_store_4d(&tm_dk, ks + Smem::kK + x * Smem::kKeyStep, 64 * x, w.kh, w.t0, w.b);
                }
                tma_store_commit();
            }
            __syncwarp();
            // dg: what leaves S and the pairs from a token on, what reaches D
            // from before it, <S, D>
            const DeltaGradTcBars::Sums &S = m.sum[n & 1];
            const DeltaGradTcBars::Gates &G = m.gate[n & 1];
            float back[2], front[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int t = lane + 32 * v;
                float x = S.inter[0][0][t] + S.inter[0][1][t] + S.inter[1][0][t] + S.inter[1][1][t];
                x += S.row[0][0][t] + S.row[0][1][t] + S.row[1][0][t] + S.row[1][1][t];
#pragma unroll
                for (int q = 0; q < 4; ++q) x -= S.col[4 * v + q][lane];
                back[v] = x;
                front[v] = S.ahead[0][t] + S.ahead[1][t];
            }
            const float own[2] = {front[0], front[1]};
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const float d = __shfl_down_sync(0xffffffffu, back[v], o);
                    const float u = __shfl_up_sync(0xffffffffu, front[v], o);
                    if (lane + o < 32) back[v] += d;
                    if (lane >= o) front[v] += u;
                }
            back[0] += __shfl_sync(0xffffffffu, back[1], 0);
            front[1] += __shfl_sync(0xffffffffu, front[0], 31);
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < 8; ++v) s += S.sd[v];
            s *= G.e[kC - 1];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int t = lane + 32 * v;
                if (t < room) {
                    const size_t r = (row0 + t) * a.heads + w.h;
                    const float dg = s + back[v] + (front[v] - own[v]);
                    a.dg[r] = from_f32<__nv_bfloat16>(t < w.cnt ? dg : 0.f);
                    if (G.beta[t] != 0.f)
                        a.dbeta[r] = from_f32<__nv_bfloat16>(t < w.cnt ? (S.db[t] + (S.lo[0][t] + S.lo[1][t])) / (G.beta[t] * G.beta[t]) : 0.f);
                }
            }
            // tokens that write nothing: r lies in dV, which only this CTA has read
#pragma unroll
            for (int v = 0; v < 2; ++v)
                for (unsigned left = __ballot_sync(0xffffffffu, G.beta[lane + 32 * v] == 0.f); left; left &= left - 1) {
                    const int t = 32 * v + __ffs(left) - 1;
                    const size_t r = (row0 + t) * a.heads + w.h;
                    __nv_bfloat16 *dv = a.dv_ + r * a.dv;
                    float d = 0.f;
                    for (int j = lane; j < a.dv; j += 32) {
                        d = fmaf(to_f32(dv[j]), to_f32(a.v[r * a.dv + j]), d);
                        dv[j] = from_f32<__nv_bfloat16>(0.f);
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    if (lane == 0) a.dbeta[r] = from_f32<__nv_bfloat16>(d + (S.none[0][t] + S.none[1][t]));
                }
            __syncwarp();
            prepare();                                     // this item's turn is free
            if (elect_one()) {
                tma_store_wait_read();
                mbar_arrive(&m.keys_free[n & 1]);
            }
            __syncwarp();
            ++n;
        }
    } else {
        const bool key = (warp & 2) != 0;                  // rows 64-127
        const int hf = warp / 4, i = 32 * (warp & 1) + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
        int g = 0, n = 0;
        for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
            const Item w = item_of(item);
            if (w.cnt <= 0) continue;
            const int cnt = w.cnt, room = min(kC, a.tokens - w.t0);
            const size_t row0 = (size_t)w.b * a.tokens + w.t0;
            const bool in = i < cnt;
            const DeltaGradTcBars::Gates &G = m.gate[n & 1];
            DeltaGradTcBars::Sums &S = m.sum[n & 1];
            uint8_t *ks = smem + (n & 1) * Smem::kKeys;
            bool ok = warp_spin_wait(&m.gates[n & 1], (n >> 1) & 1, abort_flag, err);
            {   // the decays between tokens, 16 x 16 at a time (a thread an element)
                const int r = tid / 16, q = tid % 16;
#pragma unroll
                for (int rb = 0; rb < 4; ++rb) {
                    const int t = 16 * rb + r;
                    const float f = G.since[t];
#pragma unroll
                    for (int cb = 0; cb < rb; ++cb)
                        decay[t][16 * cb + q] = f * G.across[rb - 1][16 * cb + q];
                    decay[t][16 * rb + q] = r >= q ? expf(G.G.within(t, 16 * rb + q)) : 0.f;
#pragma unroll
                    for (int cb = rb + 1; cb < 4; ++cb) decay[t][16 * cb + q] = 0.f;
                }
            }
            if (named_barrier_or(1, 256, !ok)) break;      // all eight warps
            // this thread's part of <S, D>: of the last two stages beside the
            // MMAs on A and B, of those before them at once, for the pairs
            // wait for all
            float2 sd = both(0.f);
            // dV's second part times x, 8 tokens of a channel twice a stage: of
            // the last two stages read while A and B are on their way
            int stage = 0;
            uint4 vl[2][2];
            auto get_lo = [&](uint4 (&to)[2], int u) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    to[e] = reinterpret_cast<const uint4 *>(a.v_lo)[((size_t)item * nv + u) * (64 * kC / 8) + tid + 256 * e];
            };
            if (tid < 64 * nv)                             // 128 bytes each, the item's
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a.v_lo + (size_t)item * nv * (64 * kC) + tid * 64));
            auto dot_states = [&](const uint4 (&vl)[2]) {
                const int s = g & 1;
                ok = ok && warp_spin_wait(&m.full[s], (g >> 1) & 1, abort_flag, err);
                ++g;
                if (!ok) return;
                const uint8_t *st = smem + Smem::kStage0 + s * Smem::kStage;
#pragma unroll
                for (int e = 0; e < 2 * kKB; ++e) {
                    const int o = (tid + 256 * e) * 16;    // both tiles have one layout
                    const uint4 x = *reinterpret_cast<const uint4 *>(st + Smem::kS + o);
                    const uint4 y = *reinterpret_cast<const uint4 *>(st + Smem::kD + o);
                    sd = fma2(as_pair(x.x << 16, x.x & 0xffff0000u), as_pair(y.x << 16, y.x & 0xffff0000u), sd);
                    sd = fma2(as_pair(x.y << 16, x.y & 0xffff0000u), as_pair(y.y << 16, y.y & 0xffff0000u), sd);
                    sd = fma2(as_pair(x.z << 16, x.z & 0xffff0000u), as_pair(y.z << 16, y.z & 0xffff0000u), sd);
                    sd = fma2(as_pair(x.w << 16, x.w & 0xffff0000u), as_pair(y.w << 16, y.w & 0xffff0000u), sd);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(st + Smem::kX + (tid + 256 * e) * 16);
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, lw[4] = {vl[e].x, vl[e].y, vl[e].z, vl[e].w};
                    float p[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 t = mul2(as_pair(xw[j] << 16, xw[j] & 0xffff0000u),
                                              as_pair(lw[j] << 16, lw[j] & 0xffff0000u));
                        p[2 * j] = t.x;
                        p[2 * j + 1] = t.y;
                    }
                    // summed over the warp's 32 channels, as the columns of E below
#pragma unroll
                    for (int o = 4; o; o >>= 1)
#pragma unroll
                        for (int j = 0; j < o; ++j) {
                            const float give = lane & (4 * o) ? p[j] : p[j + o];
                            const float keep = lane & (4 * o) ? p[j + o] : p[j];
                            p[j] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * o);
                        }
                    p[0] += __shfl_xor_sync(0xffffffffu, p[0], 2);
                    p[0] += __shfl_xor_sync(0xffffffffu, p[0], 1);
                    if ((lane & 3) == 0) {
                        float &sum = S.lo[warp & 1][8 * (warp / 2 + 4 * e) + lane / 4];
                        sum = stage ? sum + p[0] : p[0];
                    }
                }
                ++stage;
                warp_arrive(&m.empty[s]);
            };
            for (int u = 0; u < nv - 2; ++u) {
                get_lo(vl[0], u);
                dot_states(vl[0]);
            }
            ok = ok && warp_spin_wait(&m.keys[n & 1], (n >> 1) & 1, abort_flag, err) &&
                 warp_spin_wait(&m.pair_full, n & 1, abort_flag, err);
            float e[32], rs = 0.f, mid = 0.f;
            uint32_t low[16];                              // A's, B's second parts
            const bool none = key && G.beta[i] == 0.f;
            if (ok) {                                      // A, B, and the terms of E
                tc_fence_after();
                uint32_t pd[32], pk[32];
                tmem_ld32(tl + kPd + 32 * hf, pd);
                tmem_ld32(tl + kPk + 32 * hf, pk);
                tmem_wait_ld();
                const float f = key ? -1.f : a.scale;
                uint8_t *tile = smem + (key ? Smem::kB : Smem::kA);
#pragma unroll
                for (int j8 = 0; j8 < 4; ++j8) {
                    float w8[8];
                    uint32_t hi[4];
#pragma unroll
                    for (int jj = 0; jj < 8; ++jj) {
                        const int jl = 8 * j8 + jj, j = 32 * hf + jl;
                        const bool diag = i == j;
                        // a row behind the sequence may be NaN: chosen, not multiplied
                        const float p = in ? __uint_as_float(pd[jl]) : 0.f;
                        if (diag) mid = p;
                        w8[jj] = diag && key ? 0.f : f * p * decay[i][j];
                        e[jl] = diag ? 0.f : w8[jj] * __uint_as_float(pk[jl]);
                        rs += e[jl];
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) split_pair(w8[2 * q], w8[2 * q + 1], hi[q], low[4 * j8 + q]);
                    *reinterpret_cast<uint4 *>(tile + tile_off(i, 32 * hf + 8 * j8)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                }
                if (none) {
                    S.none[hf][i] = rs;
                    rs = 0.f;
#pragma unroll
                    for (int j8 = 0; j8 < 4; ++j8)
                        *reinterpret_cast<uint4 *>(tile + tile_off(i, 32 * hf + 8 * j8)) = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 16; ++j) low[j] = 0u;
#pragma unroll
                    for (int j = 0; j < 32; ++j) e[j] = 0.f;
                }
                fence_async_shared();
                tc_fence_before();
                warp_arrive(&m.ab_ready);
            }
            if (named_barrier_or(2, 256, !ok)) break;      // the decays have been read
            {
                uint8_t *tile = smem + Smem::kDecay + (key ? kBox64 : 0);
#pragma unroll
                for (int j8 = 0; j8 < 4; ++j8)
                    *reinterpret_cast<uint4 *>(tile + tile_off(i, 32 * hf + 8 * j8)) =
                        make_uint4(low[4 * j8], low[4 * j8 + 1], low[4 * j8 + 2], low[4 * j8 + 3]);
                fence_async_shared();
                warp_arrive(&m.ablo_ready);
                get_lo(vl[0], max(0, nv - 2));
                if (nv > 1) get_lo(vl[1], nv - 1);
                if (key && (warp & 1) == hf) S.db[i] = mid;
                S.row[key][hf][i] = rs;
                // column sums over the warp's rows: halves swapped and added
                // until a lane holds one column
#pragma unroll
                for (int o = 16; o; o >>= 1)
#pragma unroll
                    for (int j = 0; j < o; ++j) {
                        const float give = lane & o ? e[j] : e[j + o];
                        const float keep = lane & o ? e[j + o] : e[j];
                        e[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                S.col[warp][lane] = e[0];
            }
            dot_states(vl[0]);
            if (nv > 1) dot_states(vl[1]);
            float sd1 = sd.x + sd.y;
#pragma unroll
            for (int o = 16; o; o >>= 1) sd1 += __shfl_xor_sync(0xffffffffu, sd1, o);
            if (lane == 0) S.sd[warp] = sd1;
            ok = ok && warp_spin_wait(&m.c_full, n & 1, abort_flag, err);
            if (ok) {
                tc_fence_after();
                const float f0 = key ? -G.e[i] : a.scale * G.e[i], f1 = none ? 0.f : f0, f2 = G.rest[i];
                uint8_t *mine = ks + (key ? Smem::kK : Smem::kQ);
                float2 inter = both(0.f), ahead = both(0.f);
                float *wide = (key ? a.dk_wide : a.dq_wide) + ((row0 + i) * a.heads + w.h) * (size_t)DK;
#pragma unroll
                for (int p = 0; p < kKB; ++p) {            // 32 of this half's columns
                    const int col = hf * (DK / 2) + 32 * p;
                    uint32_t c1[32], c3[32], c2[32];
                    tmem_ld32(tl + kC1 + col, c1);
                    tmem_ld32(tl + kC3 + col, c3);
                    if (key) tmem_ld32(tl + kC2 + col, c2);
                    tmem_wait_ld();
                    float2 r[16];
#pragma unroll
                    for (int j8 = 0; j8 < 4; ++j8) {
                        const uint4 ov = *reinterpret_cast<const uint4 *>(
                            mine + (col / 64) * Smem::kKeyStep + tile_off(i, (col & 63) + 8 * j8));
                        const uint32_t own[4] = {ov.x, ov.y, ov.z, ov.w};
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj) {
                            const int j = 4 * j8 + jj;
                            const float2 o2 = as_pair(own[jj] << 16, own[jj] & 0xffff0000u);
                            const float2 z = as_pair(c1[2 * j], c1[2 * j + 1]);
                            inter = fma2(o2, z, inter);
                            r[j] = fma2(both(f1), z, as_pair(c3[2 * j], c3[2 * j + 1]));
                            if (key) {
                                const float2 x = mul2(both(f2), as_pair(c2[2 * j], c2[2 * j + 1]));
                                ahead = fma2(o2, x, ahead);
                                r[j] = add2(r[j], x);
                            }
                        }
                    }
                    if (key) {
                        tmem_ld32(tl + kC4 + col, c1);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = add2(r[j], as_pair(c1[2 * j], c1[2 * j + 1]));
                    }
                    if (p == kKB - 1) {                    // the accumulators are read
                        tc_fence_before();
                        warp_arrive(&m.acc_free);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = in ? r[j] : both(0.f);
#pragma unroll
                    for (int j8 = 0; j8 < 4; ++j8) {
                        const float2 *v = &r[4 * j8];
                        if (shared_keys) {
                            if (i < room) {
                                reinterpret_cast<float4 *>(wide + col + 8 * j8)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
                                reinterpret_cast<float4 *>(wide + col + 8 * j8)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
                            }
                        } else {                           // where this thread read its own row
                            *reinterpret_cast<uint4 *>(
                                mine + (col / 64) * Smem::kKeyStep + tile_off(i, (col & 63) + 8 * j8)) =
                                make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                           pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
                        }
                    }
                }
                S.inter[key][hf][i] = in ? f1 * (inter.x + inter.y) : 0.f;
                if (none) S.none[hf][i] += f0 * (inter.x + inter.y);
                if (key) S.ahead[hf][i] = in ? ahead.x + ahead.y : 0.f;
                fence_async_shared();
                warp_arrive(&m.done[n & 1]);
            }
            ++n;                                           // a failed wait shows at the next barrier
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 8 && lane == 0) {           // as in the walks
        for (int j = max(0, kit - 2); j < kit; ++j) mbar_drain(&m.keys[j & 1], (j >> 1) & 1, err);
        for (int j = max(0, it - 2); j < it; ++j)
            if (!hook_skips(blockIdx.x == 0, j)) mbar_drain(&m.full[j & 1], (j >> 1) & 1, err);
        for (int j = max(0, lit - 2); j < lit; ++j) mbar_drain(&m.lo_full[j & 1], (j >> 1) & 1, err);
    }
    if (warp == 9) {
        if (*abort_flag) drain_mmas(&m.drain, err);
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
                                         (int)sizeof(DeltaPrepSmem<DK, kSplit>));
    if (e != cudaSuccess) return e;
    DeltaPrepArgs p = {(const __nv_bfloat16 *)a.q, (const __nv_bfloat16 *)a.k,
                       (const __nv_bfloat16 *)a.g, (const __nv_bfloat16 *)a.beta, a.lengths,
                       blocks, a.scale, a.heads, a.key_heads, a.seqlen, nc, backward ? 1 : 0};
    KernelTimer timer("delta_prep", stream);
    count_launch();
    return launch_overlapped(delta_prep_kernel<DK, kSplit>,
                             dim3((unsigned)((long long)a.batch * a.heads * nc)), dim3(kPrepThreads),
                             sizeof(DeltaPrepSmem<DK, kSplit>), stream, p);
}

// Segments of the walk over nc chunks, and chunks of each: the count with the
// least time, counted in chunks walked behind one another in two parts (a wave
// of 148 CTAs each, first pass and second).  In one part, which is all of it
// without a final state, a chunk takes 0.6 of that (0.72 for dk 64).  The two
// further launches cost 7 (5, 4) and a join of states 1.  Measured, 128 x 128,
// with a final state, a call: 16 heads, 128 chunks: 431 us whole, 231 in 6
// segments; 32 chunks: 114 and 80; 24 heads, 32 chunks: 129 and 107; 32 heads:
// 140 and 136; 64 heads, 128 chunks: 720 and 726 (whole).  Without: 16 heads,
// 128 chunks: 333 and 187; 1 head, 32 chunks: 76 and 48; 32 heads, 64 chunks:
// 206 and 176.
struct DeltaCut {
    int count, chunks;
};
DeltaCut delta_segments(int batch, int heads, int nc, int dk, int dv, bool final_state) {
    const long long units = (long long)batch * heads, walks = units * ((dv + 127) / 128);
    auto waves = [](long long ctas) { return (float)((ctas + 147) / 148); };
    const float coarse = dk == 64 ? 0.72f : 0.6f, fine = final_state ? 1.f : coarse;
    const float fixed = !final_state ? 4.f : dk == 64 ? 5.f : 7.f;
    float best = 0.95f * fine * waves(walks) * nc;
    DeltaCut cut = {1, nc};
    for (int s = 3; s <= 16 && 4 * s <= nc; ++s) {
        // the last segment in two parts as long as the others in one
        const int chunks = (int)ceilf(nc / (s - 1 + coarse / fine)), left = nc - (s - 1) * chunks;
        if (left < 1) continue;
        const float cost = fine * chunks * waves(walks + (s - 2) * (walks + units)) +
                           fmaxf(coarse * chunks, fine * left) * waves(walks * (s - 1)) + fixed + s;
        if (cost < best) {
            best = cost;
            cut = {s, chunks};
        }
    }
    return cut;
}

struct DeltaTcLayout {
    int nc, segments, segment;
    size_t starts, units, total;
};
DeltaTcLayout tc_layout(int batch, int heads, int seqlen, int dk, int dv, bool final_state) {
    DeltaTcLayout l;
    l.nc = (seqlen + kC - 1) / kC;
    const DeltaCut cut = delta_segments(batch, heads, l.nc, dk, dv, final_state);
    l.segments = cut.count;
    l.segment = cut.chunks;
    const size_t bh = (size_t)batch * heads;
    l.starts = bh * l.nc * (dk == 64 ? DeltaBlock<64, true>::kBytes : DeltaBlock<128, true>::kBytes);
    l.units = l.starts + (l.segments > 1 ? (size_t)(l.segments - 1) * bh * dk * dv * 4 : 0);
    l.total = l.units + (l.segments > 1 ? (size_t)(l.segments - 2) * bh * dk * dk * 4 : 0);
    return l;
}

bool scan_maps(const DeltaArgs &a, CUtensorMap *k, CUtensorMap *v) {
    return token_map(k, a.k, a.batch, a.seqlen, a.key_heads, a.dk) &&
           token_map(v, a.v, a.batch, a.seqlen, a.heads, a.dv);
}

template <int DK, bool kSplit>
cudaError_t launch_scan(const DeltaArgs &a, int nc, const uint8_t *blocks, cudaStream_t stream) {
    using Smem = DeltaScanSmem<DK, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(delta_scan_kernel<DK, kSplit>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Smem::kBytes);
    if (e != cudaSuccess) return e;
    CUtensorMap tm_k, tm_v;
    if (!scan_maps(a, &tm_k, &tm_v)) return cudaErrorInvalidValue;
    DeltaScanArgs s = {blocks, a.lengths, a.state_in, a.state_out, (__nv_bfloat16 *)a.out, nullptr,
                       nullptr, a.heads, a.key_heads, a.seqlen, nc, a.dv, device_error_word(),
                       1, nc, nullptr, nullptr};
    const int slabs = (a.dv + 127) / 128;
    KernelTimer timer("delta_scan", stream);
    count_launch();
    return launch_overlapped(delta_scan_kernel<DK, kSplit>,
                             dim3((unsigned)(a.batch * a.heads * slabs)), dim3(kScanThreads),
                             Smem::kBytes, stream, tm_k, tm_v, s);
}

template <int DK, bool kSplit>
cudaError_t launch_segments(const DeltaArgs &a, const DeltaTcLayout &l, uint8_t *ws, cudaStream_t stream) {
    using Smem = DeltaScanSmem<DK, kSplit>;
    CUtensorMap tm_k, tm_v;
    if (!scan_maps(a, &tm_k, &tm_v)) return cudaErrorInvalidValue;
    float *starts = (float *)(ws + l.starts), *units = (float *)(ws + l.units);
    DeltaScanArgs s = {ws, a.lengths, a.state_in, a.state_out, (__nv_bfloat16 *)a.out, nullptr,
                       nullptr, a.heads, a.key_heads, a.seqlen, l.nc, a.dv, device_error_word(),
                       l.segments, l.segment, starts, units};
    const int bhs = a.batch * a.heads, walks = bhs * ((a.dv + 127) / 128);
    auto pass = [&](auto kernel, int ctas, const char *name) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Smem::kBytes);
        if (e != cudaSuccess) return e;
        KernelTimer timer(name, stream);
        count_launch();
        return launch_overlapped(kernel, dim3((unsigned)ctas), dim3(kScanThreads), Smem::kBytes, stream,
                                 tm_k, tm_v, s, bhs);
    };
    cudaError_t e = pass(delta_segments_kernel<DK, kSplit, false>,
                         walks * (l.segments - 1) + bhs * (l.segments - 2), "delta_segments");
    if (e != cudaSuccess) return e;
    e = launch_join<DK>(starts, nullptr, units, bhs, a.dv, l.segments - 2, stream);
    if (e != cudaSuccess) return e;
    return pass(delta_segments_kernel<DK, kSplit, true>, walks * (l.segments - 1), "delta_segments_out");
}

size_t up1k(size_t x) { return (x + 1023) & ~(size_t)1023; }

// Segments of the backward's walks, as delta_segments, in chunks walked back.
// Measured, 128 x 128, a call: 1 head, 128 chunks: 347 us whole, 113 in 12
// segments; 16 heads: 501 and 396 in 4; 24 heads, 64 chunks: 314 and 303 in 3;
// 32 chunks: 177 and 183 (whole); 32 heads, 64 chunks: 359 and 411 (whole).
DeltaCut back_segments(int batch, int heads, int nc, int dv) {
    const long long units = (long long)batch * heads, walks = units * ((dv + 127) / 128);
    auto waves = [](long long ctas) { return (ctas + 147) / 148; };
    float best = 0.95f * (float)(waves(2 * walks) * nc);
    DeltaCut cut = {1, nc};
    for (int s = 3; s <= 16 && 4 * s <= nc; ++s) {
        const int chunks = (nc + s - 1) / s;
        if ((s - 1) * chunks >= nc) continue;
        const float cost = (float)(chunks * (waves(2 * walks * (s - 1) + units * (s - 2)) +
                                             waves(2 * walks * (s - 1)))) + 6.f + s;
        if (cost < best) {
            best = cost;
            cut = {s, chunks};
        }
    }
    return cut;
}

struct DeltaTcGradLayout {
    size_t blocks, x, s, d, vlo, dq, dk, starts, back, units, total;
    DeltaCut cut;
};
DeltaTcGradLayout tc_grad_layout(int batch, int heads, int key_heads, int seqlen, int dk, int dv) {
    const size_t chunks = (size_t)batch * heads * ((seqlen + kC - 1) / kC);
    const size_t wide = heads != key_heads ? up1k((size_t)batch * seqlen * heads * dk * 4) : 0;
    DeltaTcGradLayout l;
    l.blocks = 0;
    l.x = chunks * (dk == 64 ? DeltaBlock<64, false>::kBack : DeltaBlock<128, false>::kBack);
    l.s = l.x + chunks * dv * kC * 4;
    l.d = l.s + chunks * dv * dk * 2;
    l.vlo = l.d + chunks * dv * dk * 2;
    l.dq = l.vlo + chunks * dv * kC * 2;
    l.dk = l.dq + wide;
    l.cut = back_segments(batch, heads, (int)(((size_t)seqlen + kC - 1) / kC), dv);
    const size_t bh = (size_t)batch * heads, between = l.cut.count - 1;
    l.starts = l.dk + wide;
    l.back = l.starts + between * bh * dk * dv * 4;
    l.units = l.back + between * bh * dk * dv * 4;
    l.total = l.units + (between ? between - 1 : 0) * bh * dk * dk * 4;
    return l;
}

template <int DK>
cudaError_t launch_backward(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    const int nc = (a.seqlen + kC - 1) / kC, slabs = (a.dv + 127) / 128;
    const long long bh = (long long)a.batch * a.heads;
    const DeltaTcGradLayout l = tc_grad_layout(a.batch, a.heads, a.key_heads, a.seqlen, a.dk, a.dv);
    uint8_t *ws = (uint8_t *)workspace;
    __nv_bfloat16 *xs = (__nv_bfloat16 *)(ws + l.x), *ss = (__nv_bfloat16 *)(ws + l.s),
                  *ds = (__nv_bfloat16 *)(ws + l.d), *vlo = (__nv_bfloat16 *)(ws + l.vlo);
    float *dq_wide = (float *)(ws + l.dq), *dk_wide = (float *)(ws + l.dk);
    cudaError_t e = launch_prep<DK, false>(a, nc, ws + l.blocks, true, stream);
    if (e != cudaSuccess) return e;
    CUtensorMap tm_q, tm_k, tm_v, tm_do, tm_dv, tm_dq, tm_dk;
    if (!token_map(&tm_q, a.q, a.batch, a.seqlen, a.key_heads, DK) ||
        !token_map(&tm_k, a.k, a.batch, a.seqlen, a.key_heads, DK) ||
        !token_map(&tm_v, a.v, a.batch, a.seqlen, a.heads, a.dv) ||
        !token_map(&tm_do, a.d_out, a.batch, a.seqlen, a.heads, a.dv) ||
        !token_map(&tm_dv, a.dv_grad, a.batch, a.seqlen, a.heads, a.dv) ||
        !token_map(&tm_dq, a.dq, a.batch, a.seqlen, a.key_heads, DK) ||
        !token_map(&tm_dk, a.dk_grad, a.batch, a.seqlen, a.key_heads, DK))
        return cudaErrorInvalidValue;
    {
        using Smem = DeltaReverseSmem<DK>;                 // the larger of the two walks'
        const DeltaScanArgs f = {ws + l.blocks, a.lengths, nullptr, nullptr, nullptr, xs, ss, a.heads,
                                 a.key_heads, a.seqlen, nc, a.dv, device_error_word(), 1, nc, nullptr, nullptr};
        const DeltaReverseArgs r = {ws + l.blocks, a.lengths, ds, vlo, a.heads, a.key_heads, a.seqlen, nc, a.dv,
                                    device_error_word()};
        const int bhs = (int)bh, walks = bhs * slabs;
        auto launch = [&](auto kernel, const char *name, int ctas, auto... rest) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)Smem::kBytes);
            if (e != cudaSuccess) return e;
            KernelTimer timer(name, stream);
            count_launch();
            return launch_overlapped(kernel, dim3((unsigned)ctas), dim3(kScanThreads), Smem::kBytes, stream,
                                     tm_k, tm_v, tm_do, tm_dv, f, r, rest...);
        };
        if (l.cut.count == 1) {
            e = launch(delta_walks_kernel<DK>, "delta_walks", 2 * walks);
        } else {
            const DeltaBackSegments x = {l.cut.count, l.cut.chunks, (float *)(ws + l.starts),
                                         (float *)(ws + l.back), (float *)(ws + l.units)};
            const int ends = 2 * walks * (x.segments - 1);
            e = launch(delta_walks_segments_kernel<DK>, "delta_walks_segments", ends + bhs * (x.segments - 2), x, bhs, 0);
            if (e != cudaSuccess) return e;
            e = launch_join<DK>(x.starts, x.back, x.units, bhs, a.dv, x.segments - 2, stream);
            if (e != cudaSuccess) return e;
            e = launch(delta_walks_segments_kernel<DK>, "delta_walks_segments", ends, x, bhs, 1);
        }
        if (e != cudaSuccess) return e;
    }
    {
        using Smem = DeltaGradTcSmem<DK>;
        e = cudaFuncSetAttribute(delta_grad_tc_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Smem::kBytes);
        if (e != cudaSuccess) return e;
        DeltaGradTcArgs g = {(const __nv_bfloat16 *)a.v, (const __nv_bfloat16 *)a.g, (const __nv_bfloat16 *)a.beta, xs, ss, ds, vlo, a.lengths,
                             (__nv_bfloat16 *)a.dq, (__nv_bfloat16 *)a.dk_grad,
                             (__nv_bfloat16 *)a.dv_grad, (__nv_bfloat16 *)a.dg,
                             (__nv_bfloat16 *)a.dbeta, dq_wide, dk_wide, a.scale, a.heads,
                             a.key_heads, a.seqlen, nc, a.dv, (int)(bh * nc), device_error_word()};
        KernelTimer timer("delta_grad_tc", stream);
        count_launch();
        e = launch_overlapped(delta_grad_tc_kernel<DK>, dim3((unsigned)(bh * nc < 148 ? bh * nc : 148)),
                              dim3(kGradTcThreads), Smem::kBytes, stream, tm_q, tm_k, tm_do, tm_dv,
                              tm_dq, tm_dk, g);
        if (e != cudaSuccess) return e;
    }
    return launch_delta_share(a, dq_wide, dk_wide, stream);
}

template <int DK, bool kSplit>
cudaError_t launch_prefill(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    const DeltaTcLayout l = tc_layout(a.batch, a.heads, a.seqlen, DK, a.dv, kSplit);
    uint8_t *ws = (uint8_t *)workspace;
    const cudaError_t e = launch_prep<DK, kSplit>(a, l.nc, ws, false, stream);
    if (e != cudaSuccess) return e;
    return l.segments > 1 ? launch_segments<DK, kSplit>(a, l, ws, stream)
                          : launch_scan<DK, kSplit>(a, l.nc, ws, stream);
}
// A final state is wanted in float32 precision, and only then operands in two parts.
template <int DK>
cudaError_t launch_forward(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    return a.state_out ? launch_prefill<DK, true>(a, workspace, stream)
                       : launch_prefill<DK, false>(a, workspace, stream);
}

}  // namespace

cudaError_t launch_delta_join(float *starts, float *back, const float *units, int bhs, int dk, int dv,
                              int joins, cudaStream_t stream) {
    return dk == 64 ? launch_join<64>(starts, back, units, bhs, dv, joins, stream)
                    : launch_join<128>(starts, back, units, bhs, dv, joins, stream);
}

size_t delta_backward_tc_workspace(int batch, int heads, int key_heads, int seqlen, int dk, int dv) {
    return tc_grad_layout(batch, heads, key_heads, seqlen, dk, dv).total;
}

cudaError_t launch_delta_backward_tc(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    return a.dk == 64 ? launch_backward<64>(a, workspace, stream)
                      : launch_backward<128>(a, workspace, stream);
}

bool delta_tc_shape_ok(int dk, int dv, retnet_dtype dtype) {
    return dtype == RETNET_BF16 && (dk == 64 || dk == 128) && dv >= 64;
}

size_t delta_tc_workspace(int batch, int heads, int seqlen, int dk, int dv) {
    const size_t with = tc_layout(batch, heads, seqlen, dk, dv, true).total;
    const size_t without = tc_layout(batch, heads, seqlen, dk, dv, false).total;
    return with > without ? with : without;
}

#ifdef RETNET_TEST_HOOKS
cudaError_t set_delta_hooks(unsigned long long wait_limit_ns, int skip_load) {
    const cudaError_t e = cudaMemcpyToSymbol(sm100::g_hook_wait_limit_ns, &wait_limit_ns,
                                             sizeof(wait_limit_ns));
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_hook_skip_second_load, &skip_load, sizeof(int));
}
#endif

cudaError_t launch_delta_tc(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    return a.dk == 64 ? launch_forward<64>(a, workspace, stream)
                      : launch_forward<128>(a, workspace, stream);
}

}  // namespace retnet
