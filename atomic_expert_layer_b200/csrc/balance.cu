// balance.cu -- per-expert counts and the router's balance loss over the
// implicit N_r x N_c grid, with its gradients, on the sm_100a tensor cores.
//
// For tokens t (those with mask 0 left out; n of them counted, n_l in this
// batch), experts e = (i, j) and counts F[i, j] = tasks of expert e:
//   loss = N sum_e f_e P_e,  f_e = F[e] / (K n),
//   P_e  = mean over the kept tokens of exp(p_r[t, i]) exp(p_c[t, j]),
// the product of the shares of the tasks and of the probability that each of
// the N experts gets.  The softmax over the whole grid is the product of the
// row and column softmaxes, so with P_r = exp(p_r), P_c = exp(p_c) [L, N_r],
// [L, N_c] the [L, N] probabilities are never built:
//   U = P_c F^T [L, N_r],  V = P_r F [L, N_c],
//   l_t = sum_i P_r[t, i] U[t, i] = sum_j P_c[t, j] V[t, j],
//   loss = N / (K n n_l) sum_t l_t.
// The counts carry no gradient (a selection has none); through the
// LogSoftmax of the logits, with c = dloss N / (K n n_l),
//   ds_r[t, i] = c P_r[t, i] (U[t, i] - l_t),  ds_c[t, j] = c P_c[t, j] (V[t, j] - l_t),
//   dx = ds_r W_r + ds_c W_c,  dW_r += ds_r^T x,  dW_c += ds_c^T x.
//
// All products run as tcgen05 tile GEMMs with fp32 accumulation.  An operand
// that is fp32 by nature enters as the sum of two 16-bit values, hi + lo,
// against one that 16 bits hold exactly; both halves meet the same B tile, so
// it is loaded once.
//   U, V: fp16.  2^14 P keeps 22 bits (or 2^-39 of P, whichever is coarser)
//     and 2^-16 F holds counts up to 2048 exactly.  U - l_t cancels when the
//     experts are nearly even or when the router has collapsed; bf16 halves
//     (16 bits) left ds of a collapsed router off by 4e-3 where these leave
//     what fp32 arithmetic does.  When some count exceeds 2048, what its
//     rounding to fp16 leaves is a second matrix F_lo, and hi * F_lo is added
//     (22 bits of a count).
//   dx, dW: bf16, the type of W and x.  ds is off by at most 2^-16 of itself
//     (one bf16 would lose 2^-8).
//
// Masked rows of p are never read as numbers: their P and ds are zero.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "omni_common.cuh"
#include "omni_internal.h"
#include "tcgen05.cuh"

namespace omni {
namespace {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float bf16_of(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// 8 values as hi and lo bf16 vectors
__device__ __forceinline__ void split8(const float *v, uint4 *hi, uint4 *lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        const float ah = bf16_of(a), bh = bf16_of(b);
        h[i] = pack_bf16(ah, bh);
        l[i] = pack_bf16(a - ah, b - bh);
    }
    *hi = make_uint4(h[0], h[1], h[2], h[3]);
    *lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The scales at which P and the counts are held in fp16.
constexpr float kScaleP = 16384.f;              // 2^14
constexpr float kScaleF = 1.f / 65536.f;        // 2^-16: counts up to 2^31 stay below fp16's largest
constexpr float kUnscale = 4.f;                 // 1 / (kScaleP kScaleF)
constexpr int kExactCount = 2048;               // counts up to this need no F_lo

__device__ __forceinline__ float f16_of(float v) { return __half2float(__float2half_rn(v)); }
__device__ __forceinline__ uint16_t f16_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ void split8_f16(const float *v, uint4 *hi, uint4 *lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 a = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(a);
        const __half2 b = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
        h[i] = *reinterpret_cast<const uint32_t *>(&a);
        l[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *hi = make_uint4(h[0], h[1], h[2], h[3]);
    *lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// ----------------------------------------------------------------- counts
__global__ void counts_clear_kernel(int32_t *__restrict__ counts, int64_t N,
                                    int32_t *__restrict__ n_tokens) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = at; i < N; i += (int64_t)gridDim.x * blockDim.x) counts[i] = 0;
    if (at == 0) *n_tokens = 0;
}

// One thread per task; integer atomics, so the counts do not depend on the
// order.  The thread of a kept token's first task counts the token.
__global__ void __launch_bounds__(256)
counts_kernel(const int32_t *__restrict__ idx, const uint8_t *__restrict__ mask, int64_t M, int K,
              int64_t N, int32_t *__restrict__ counts, int32_t *__restrict__ n_tokens, int *status) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t m = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    bool first = false;
    if (m < M) {
        const int64_t t = m / K;
        if (!mask || mask[t]) {
            const int e = idx[m];
            if (e < 0 || e >= N) set_status(status, OMNI_DEV_BAD_EXPERT);
            else atomicAdd(&counts[e], 1);
            first = m == t * K;
        }
    }
    const unsigned votes = __ballot_sync(0xffffffffu, first);
    if (votes && lane_id() == 0) atomicAdd(n_tokens, __popc(votes));
}

// -------------------------------------------------------------- operands
struct BalPrep {
    const float *p_r, *p_c;
    const int32_t *counts;
    const uint8_t *mask;
    const uint16_t *x;            // masked copy wanted when xs is not null
    int L, N_r, N_c, d;
    int seg_r, ld;                // columns of the row segment, and of P (0: only the column axis)
    int pc, pr;                   // padded N_c, N_r
    uint16_t *P_hi, *P_lo, *F_hi, *F_lo, *T_hi, *T_lo, *xs;
    int *big;                     // set when a count exceeds kExactCount
    int *n_local;                 // kept tokens of this batch
};

__device__ __forceinline__ void prep_probs(const BalPrep &p, int64_t unit) {
    const int per = p.ld >> 3;
    const int64_t t = unit / per;
    const int c0 = (int)(unit % per) * 8;
    const bool rows = c0 < p.seg_r;
    const int col = rows ? c0 : c0 - p.seg_r;
    const int n = rows ? p.N_r : p.N_c;
    const float *src = (rows ? p.p_r : p.p_c) + t * n + col;
    float v[8];
    const bool keep = !p.mask || p.mask[t];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = keep && col + i < n ? kScaleP * expf(src[i]) : 0.f;
    uint4 hi, lo;
    split8_f16(v, &hi, &lo);
    *reinterpret_cast<uint4 *>(p.P_hi + t * p.ld + c0) = hi;
    *reinterpret_cast<uint4 *>(p.P_lo + t * p.ld + c0) = lo;
}

constexpr int kPrepThreads = 256;

// Work units of a CTA: first the 32 x 32 tiles of the counts (F and its
// transpose, padded with zeros), then 8-value pieces of P, then of x.
__global__ void __launch_bounds__(kPrepThreads) balance_prep_kernel(const BalPrep p) {
    __shared__ float tile[32][33];
    grid_dependency_wait();
    grid_dependents_launch();
    const int tr = p.pr / 32, tc = p.pc / 32;
    bool big = false;
    for (int u = blockIdx.x; u < tr * tc; u += gridDim.x) {
        const int i0 = (u / tc) * 32, j0 = (u % tc) * 32;
        const int a = (int)threadIdx.x >> 5, l = (int)threadIdx.x & 31;
        __syncthreads();
        for (int r = a; r < 32; r += 8) {
            const int i = i0 + r, j = j0 + l;
            const int c = i < p.N_r && j < p.N_c ? p.counts[(int64_t)i * p.N_c + j] : 0;
            big |= c > kExactCount;
            const float f = (float)c * kScaleF;
            tile[r][l] = f;
            if (i < p.N_r) {
                p.F_hi[(int64_t)i * p.pc + j] = f16_bits(f);
                p.F_lo[(int64_t)i * p.pc + j] = f16_bits(f - f16_of(f));
            }
        }
        if (p.T_hi) {
            __syncthreads();
            for (int r = a; r < 32; r += 8) {
                const int j = j0 + r, i = i0 + l;
                const float f = tile[l][r];
                if (j < p.N_c) {
                    p.T_hi[(int64_t)j * p.pr + i] = f16_bits(f);
                    p.T_lo[(int64_t)j * p.pr + i] = f16_bits(f - f16_of(f));
                }
            }
        }
    }
    if (__syncthreads_or(big) && threadIdx.x == 0) atomicOr(p.big, 1);

    const int64_t step = (int64_t)gridDim.x * kPrepThreads;
    const int64_t at = (int64_t)blockIdx.x * kPrepThreads + threadIdx.x;
    const int64_t units = (int64_t)p.L * (p.ld >> 3);
    for (int64_t u = at; u < units; u += step) prep_probs(p, u);
    if (p.xs) {
        const int64_t n = (int64_t)p.L * (p.d >> 3);
        for (int64_t u = at; u < n; u += step) {
            const int64_t t = u / (p.d >> 3);
            reinterpret_cast<uint4 *>(p.xs)[u] =
                p.mask[t] ? reinterpret_cast<const uint4 *>(p.x)[u] : make_uint4(0, 0, 0, 0);
        }
    }
    int kept = 0;
    for (int64_t t = at; t < p.L; t += step) kept += !p.mask || p.mask[t];
    kept = warp_isum(kept);
    if (kept && lane_id() == 0) atomicAdd(p.n_local, kept);
}

// -------------------------------------------------------------- tile GEMM
// C[M, N] = (A_hi + A_lo) B over a K axis of 64-element steps, tiles of 128 x
// bn.  An operand is K-major (its K axis contiguous in memory) or MN-major
// (its M or N axis contiguous); either way a TMA box is 64 elements (128
// bytes, one swizzle atom) wide along the contiguous axis.
constexpr int BM = 128, BN = 256, BK = kSwK, STAGES = 3;
constexpr int kBytesA = BM * BK * 2;             // 16 KB, each of hi and lo
constexpr int kBytesB = BN * BK * 2;             // 32 KB at most
constexpr int kBlockMN = 64 * BK * 2;            // an MN-major box: 64 K rows of 128 bytes
constexpr uint32_t kTmemCols = 2 * BN;
constexpr int kEpiWarps = 8;
constexpr int kEpiBlocks = BN / 64;              // 32-column blocks of a tile for one of them
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kIdescBf16 = umma_idesc_bf16(BM, 0);        // the tile width is added per problem
constexpr uint32_t kIdescF16 = kIdescBf16 & ~((1u << 7) | (1u << 10));   // A and B fp16 (formats 0)
constexpr int kMaxProbs = 3, kMaxMaps = 9;
// K steps that are summed in TMEM before the epilogue warps add them to their
// registers.  The tensor core cuts off what falls below its accumulator at
// every instruction (8 of them in a step), always towards zero: over the 512
// instructions of a dW tile at L = 4096 that took 1.1e-5 off the result, and
// it grows with L; over 32 it is below 1e-6, and the additions in registers
// round to nearest.  Draining is hidden behind the next steps' products.
constexpr int kChunk = 4;

struct __align__(1024) GemmSmem {
    uint8_t a[STAGES][2 * kBytesA];
    uint8_t b[STAGES][kBytesB];
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint32_t tmem_base;
    int abort;
};

struct GemmProb {
    int M, N;                     // rows and columns of C
    int bn, tiles_n, tiles;       // tile width (a multiple of 32), tiles in N, tiles in all
    int nk;                       // 64-element steps of the K axis
    int a_hi, a_lo;               // tensor maps of A
    int a_c0;                     // first column of A's segment in its matrix
    int b, b2;                    // maps of B; b2: the remainder F_lo, or B past step nk1
    int nk1;                      // MN-major B: steps taken from b (the rest from b2)
    float *out;                   // C in fp32 (products with W and x)
    int ld_out, accumulate;
    const float *p;               // log-probabilities beside this C (products with F)
    uint16_t *ds_hi, *ds_lo;      // their gradient, column 0 of this segment
    int seg;                      // columns of the segment (N padded to 64; the pad gets zeros)
};

struct GemmArgs {
    GemmProb prob[kMaxProbs];
    int nprob, tiles;
    const int *big;               // counts above kExactCount: also multiply by F_lo
    const uint8_t *mask;
    float *part;                  // forward: sums over a tile's columns [tiles_n * 2, L]
    const float *token_loss;      // backward
    const int32_t *n_tokens, *n_local;
    float factor;                 // dloss N / K
    int *status;
};
struct GemmMaps { CUtensorMap m[kMaxMaps]; };

// what a launch computes: U with the forward's sums; U and V with ds; dx, dW_r, dW_c
enum : int { kFwd = 0, kGrid = 1, kGrads = 2 };

// Tiles are dealt out back and forth over the CTAs, longest first, so that
// the CTAs with a long first tile get the last of the short ones.
__device__ __forceinline__ int tile_of(int turn, int tiles) {
    const int c = (turn & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x;
    const int64_t i = (int64_t)turn * gridDim.x + c;
    return i < tiles ? (int)i : -1;
}

__device__ __forceinline__ int find_prob(const GemmArgs &g, int *tile) {
    int k = 0;
    while (k + 1 < g.nprob && *tile >= g.prob[k].tiles) *tile -= g.prob[k++].tiles;
    return k;
}

// Descriptor of an MN-major tile: 64-element blocks of the M or N axis
// kBlockMN apart (leading byte offset), groups of 8 K rows 1024 bytes apart
// (stride byte offset), 128-byte swizzle.
__device__ __forceinline__ uint64_t sw128_desc_mn(const void *tile) {
    uint64_t d = sw128_desc(tile) & ~((uint64_t)0x3FFF << 16);
    return d | (uint64_t)(kBlockMN >> 4) << 16;
}

template <int MODE>
__device__ __forceinline__ int steps_of(const GemmProb &p, bool big) {
    return MODE != kGrads && big ? 2 * p.nk : p.nk;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
balance_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs g) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    GemmSmem &sm = *reinterpret_cast<GemmSmem *>(smem_raw + pad);
    const int warp = threadIdx.x >> 5;
    const unsigned lane = lane_id();
    int *status = g.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.tfull[b], 1);
            mbar_init(&sm.tempty[b], kEpiWarps);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&sm.tmem_base)), "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    grid_dependency_wait();
    grid_dependents_launch();
    const bool big = MODE != kGrads && *g.big != 0;


    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer
            int it = 0, issued_from = 0;
            for (int turn = 0; !sm.abort; ++turn) {
                int tile = tile_of(turn, g.tiles);
                if ((int64_t)turn * gridDim.x >= g.tiles) break;
                if (tile < 0) continue;
                const int pk = find_prob(g, &tile);
                const GemmProb &p = g.prob[pk];
                const int m0 = (tile / p.tiles_n) * BM, n0 = (tile % p.tiles_n) * p.bn;
                const int steps = steps_of<MODE>(p, big);
                const bool a_mn = MODE == kGrads && pk < g.nprob - 1;   // dW: A is ds^T
                for (int st = 0; st < steps; ++st, ++it) {
                    const int s = it % STAGES;
                    if (it >= STAGES &&
                        !mbar_wait(&sm.empty[s], (uint32_t)(((it / STAGES) - 1) & 1), status)) {
                        sm.abort = 1;
                        break;
                    }
                    const bool rest = MODE != kGrads && st >= p.nk;      // hi times F_lo
                    const int kb = rest ? st - p.nk : st;
                    mbar_arrive_expect_tx(&sm.full[s],
                                          (uint32_t)((rest ? 1 : 2) * kBytesA + p.bn * BK * 2));
                    uint8_t *a = sm.a[s], *b = sm.b[s];
                    if (a_mn) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            tma_load_2d(a + i * kBlockMN, &maps.m[p.a_hi], p.a_c0 + m0 + 64 * i,
                                        kb * BK, &sm.full[s]);
                            tma_load_2d(a + kBytesA + i * kBlockMN, &maps.m[p.a_lo],
                                        p.a_c0 + m0 + 64 * i, kb * BK, &sm.full[s]);
                        }
                    } else {
                        tma_load_2d(a, &maps.m[p.a_hi], p.a_c0 + kb * BK, m0, &sm.full[s]);
                        if (!rest)
                            tma_load_2d(a + kBytesA, &maps.m[p.a_lo], p.a_c0 + kb * BK, m0,
                                        &sm.full[s]);
                    }
                    if (MODE == kGrads) {
                        const bool second = kb >= p.nk1;
                        const CUtensorMap *tm = &maps.m[second ? p.b2 : p.b];
                        const int k0 = (second ? kb - p.nk1 : kb) * BK;
                        for (int j = 0; j < p.bn / 64; ++j)
                            tma_load_2d(b + j * kBlockMN, tm, n0 + 64 * j, k0, &sm.full[s]);
                    } else {
                        tma_load_2d(b, &maps.m[rest ? p.b2 : p.b], kb * BK, n0, &sm.full[s]);
                    }
                    issued_from = it + 1 > STAGES ? it + 1 - STAGES : 0;
                }
            }
            if (sm.abort)
                for (int k = issued_from; k < it; ++k)
                    mbar_wait(&sm.full[k % STAGES], (uint32_t)((k / STAGES) & 1), status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // ---- MMA issuer
            int it = 0, lt = 0;
            bool ok = true;
            for (int turn = 0; ok; ++turn) {
                int tile = tile_of(turn, g.tiles);
                if ((int64_t)turn * gridDim.x >= g.tiles) break;
                if (tile < 0) continue;
                const int pk = find_prob(g, &tile);
                const GemmProb &p = g.prob[pk];
                const int steps = steps_of<MODE>(p, big);
                const bool a_mn = MODE == kGrads && pk < g.nprob - 1;
                // bits 15 and 16 of the instruction descriptor: A, B are MN-major
                const uint32_t idesc = (MODE == kGrads ? kIdescBf16 | 1u << 16 : kIdescF16) |
                                       ((uint32_t)(p.bn >> 3) << 17) | (a_mn ? 1u << 15 : 0u);
                // a 16-deep slice: 32 bytes along a K-major atom, or 16 K rows
                const uint64_t a_step = (a_mn ? 16 * 128 : 32) >> 4;
                const uint64_t b_step = (MODE == kGrads ? 16 * 128 : 32) >> 4;
                uint32_t acc = 0;
                for (int st = 0; st < steps; ++st, ++it) {
                    const int s = it % STAGES;
                    const bool first = st % kChunk == 0;
                    if (first) {                              // the next accumulator
                        if (lt >= 2 &&
                            !mbar_wait(&sm.tempty[lt & 1], (uint32_t)(((lt >> 1) - 1) & 1), status)) {
                            ok = false;
                            break;
                        }
                        acc = tmem + (uint32_t)((lt & 1) * BN);
                    }
                    if (!mbar_wait(&sm.full[s], (uint32_t)((it / STAGES) & 1), status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ah = a_mn ? sw128_desc_mn(sm.a[s]) : sw128_desc(sm.a[s]);
                    const uint64_t bd = MODE == kGrads ? sw128_desc_mn(sm.b[s]) : sw128_desc(sm.b[s]);
                    const bool rest = MODE != kGrads && st >= p.nk;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        umma_bf16(acc, ah + k * a_step, bd + k * b_step, idesc,
                                  (!first || k > 0) ? 1u : 0u);
                    if (!rest) {
                        const uint64_t al = ah + (kBytesA >> 4);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            umma_bf16(acc, al + k * a_step, bd + k * b_step, idesc, 1u);
                    }
                    umma_commit(&sm.empty[s]);
                    if (st % kChunk == kChunk - 1 || st == steps - 1) {
                        umma_commit(&sm.tfull[lt & 1]);
                        ++lt;
                    }
                }
            }
            if (!ok) sm.abort = 1;
        }
        __syncwarp();
    } else {
        // ---- epilogue: warp w reads TMEM lanes 32*(w % 4) .. +31 (tile rows)
        // and every second block of 32 columns
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        float c = 0.f;
        if (MODE == kGrid) {
            const int n = *g.n_tokens, nl = *g.n_local;
            c = n > 0 && nl > 0 ? g.factor / (float)n / (float)nl : 0.f;
        }
        int lt = 0;
        bool ok = true;
        for (int turn = 0; ok; ++turn) {
            int tile = tile_of(turn, g.tiles);
            if ((int64_t)turn * gridDim.x >= g.tiles) break;
            if (tile < 0) continue;
            const GemmProb &p = g.prob[find_prob(g, &tile)];
            const int m0 = (tile / p.tiles_n) * BM, tn = tile % p.tiles_n, n0 = tn * p.bn;
            const int steps = steps_of<MODE>(p, big), blocks = p.bn / 32;
            float sum[kEpiBlocks][32];
#pragma unroll
            for (int q = 0; q < kEpiBlocks; ++q)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[q][j] = 0.f;
            for (int st = 0; st < steps; st += kChunk, ++lt) {
                if (!mbar_wait(&sm.tfull[lt & 1], (uint32_t)((lt >> 1) & 1), status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)((lt & 1) * BN);
#pragma unroll
                for (int q = 0; q < kEpiBlocks; ++q) {
                    if (half + 2 * q < blocks) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[16];
                            tmem_ld16(tb + (uint32_t)(32 * (half + 2 * q) + 16 * h), r);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[q][16 * h + j] += __uint_as_float(r[j]);
                        }
                    }
                }
                // this accumulator may be overwritten once every epilogue warp is done
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.tempty[lt & 1]);
            }
            if (!ok) break;
            const int row = m0 + quarter * 32 + (int)lane;
            const bool in = row < p.M;
            const bool keep = MODE != kGrads && in && (!g.mask || g.mask[row]);
            const float lt_loss = MODE == kGrid && keep ? g.token_loss[row] : 0.f;
            float part = 0.f;
#pragma unroll
            for (int q = 0; q < kEpiBlocks; ++q) {
                if (half + 2 * q >= blocks) continue;
                const float (&r)[32] = sum[q];
                const int col = n0 + 32 * (half + 2 * q);
                if (MODE == kFwd) {
                    if (keep) {
                        const float *src = p.p + (int64_t)row * p.N + col;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < p.N) part = fmaf(expf(src[j]), kUnscale * r[j], part);
                    }
                } else if (MODE == kGrid) {
                    if (in && col < p.seg) {
                        const float *src = p.p + (int64_t)row * p.N + col;
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            float v[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int k = 8 * o + j;
                                v[j] = keep && col + k < p.N
                                           ? c * expf(src[k]) * (kUnscale * r[k] - lt_loss) : 0.f;
                            }
                            uint4 hi, lo;
                            split8(v, &hi, &lo);
                            const int64_t at = (int64_t)row * p.ld_out + col + 8 * o;
                            *reinterpret_cast<uint4 *>(p.ds_hi + at) = hi;
                            *reinterpret_cast<uint4 *>(p.ds_lo + at) = lo;
                        }
                    }
                } else if (in) {
                    float4 *dst = reinterpret_cast<float4 *>(p.out + (int64_t)row * p.ld_out + col);
#pragma unroll
                    for (int o = 0; o < 8; ++o) {
                        if (col + 4 * o < p.N) {
                            float4 v = make_float4(r[4 * o], r[4 * o + 1], r[4 * o + 2], r[4 * o + 3]);
                            if (p.accumulate) {
                                const float4 prev = dst[o];
                                v.x += prev.x;
                                v.y += prev.y;
                                v.z += prev.z;
                                v.w += prev.w;
                            }
                            dst[o] = v;
                        }
                    }
                }
            }
            if (MODE == kFwd && in) g.part[(int64_t)(2 * tn + half) * p.M + row] = part;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     ::"r"(tmem), "r"(kTmemCols));
    }
}

// l_t from the tiles' sums, and the loss: each CTA sums its tokens in 64 bits,
// the last one to finish adds the CTAs' sums in their order.
constexpr int kLossThreads = 256;
__global__ void __launch_bounds__(kLossThreads)
balance_loss_kernel(const float *__restrict__ part, int nparts, int L, float *__restrict__ token_loss,
                    double *__restrict__ block_sum, int *__restrict__ done, double factor,
                    const int32_t *__restrict__ n_tokens, const int *__restrict__ n_local,
                    float *__restrict__ loss) {
    __shared__ double sm[kLossThreads / 32];
    __shared__ int last;
    grid_dependency_wait();
    grid_dependents_launch();
    double s = 0.0;
    const int64_t t = (int64_t)blockIdx.x * kLossThreads + threadIdx.x;
    if (t < L) {
        float v = 0.f;
        for (int k = 0; k < nparts; ++k) v += part[(int64_t)k * L + t];
        token_loss[t] = v;
        s = v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane_id() == 0) sm[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kLossThreads / 32; ++k) s += sm[k];
        block_sum[blockIdx.x] = s;
        __threadfence();
        last = atomicAdd(done, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    s = 0.0;
    for (int k = (int)threadIdx.x; k < (int)gridDim.x; k += kLossThreads)
        s += *(volatile double *)(block_sum + k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (lane_id() == 0) sm[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kLossThreads / 32; ++k) s += sm[k];
        const double n = *n_tokens, nl = *n_local;
        *loss = n > 0 && nl > 0 ? (float)(factor / (n * nl) * s) : 0.f;
    }
}

inline int pad64(int n) { return (n + 63) / 64 * 64; }

// tile width: the fewest tiles of at most 256 columns, evened out to `unit`
inline int tile_width(int n, int unit) {
    const int tiles = (n + BN - 1) / BN;
    const int each = (n + tiles - 1) / tiles;
    return (each + unit - 1) / unit * unit;
}

template <int MODE>
cudaError_t launch_gemm(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    const int smem = (int)sizeof(GemmSmem) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(balance_gemm_kernel<MODE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    return launch(balance_gemm_kernel<MODE>, dim3((unsigned)(g.tiles < sms ? g.tiles : sms)),
                  dim3(kThreads), (size_t)smem, st, maps, g);
}

void set_tiles(GemmProb *p, int unit) {
    p->bn = tile_width(p->N, unit);
    p->tiles_n = (p->N + p->bn - 1) / p->bn;
    p->tiles = ((p->M + BM - 1) / BM) * p->tiles_n;
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

BalanceWs balance_ws(int L, int d, int N_r, int N_c, bool backward) {
    BalanceWs w = {};
    const int pr = pad64(N_r), pc = pad64(N_c);
    w.ld = backward ? pr + pc : pc;
    size_t o = sizeof(WsHeader);
    auto take = [&](size_t bytes) { const size_t at = o; o = align256(o + bytes); return at; };
    const size_t P = 2 * (size_t)L * w.ld;
    w.P_hi = take(P);
    w.P_lo = take(P);
    w.F_hi = take(2 * (size_t)N_r * pc);
    w.F_lo = take(2 * (size_t)N_r * pc);
    if (backward) {
        w.T_hi = take(2 * (size_t)N_c * pr);
        w.T_lo = take(2 * (size_t)N_c * pr);
        w.ds_hi = take(P);
        w.ds_lo = take(P);
        w.xs = take(2 * (size_t)L * d);
    } else {
        const int bn = tile_width(N_r, 32);
        w.parts = 2 * ((N_r + bn - 1) / bn);
        w.part = take(4 * (size_t)w.parts * L);
        w.blocks = take(8 * (size_t)((L + kLossThreads - 1) / kLossThreads));
    }
    w.total = o;
    return w;
}

cudaError_t launch_counts(const int32_t *idx, const uint8_t *mask, int64_t M, int K, int64_t N,
                          int32_t *counts, int32_t *n_tokens, int *status, cudaStream_t st) {
    const int64_t want = (N + 1023) / 1024, most = (int64_t)device_sm_count() * 8;
    cudaError_t e = launch(counts_clear_kernel, dim3((unsigned)(want < most ? want : most)),
                           dim3(256), 0, st, counts, N, n_tokens);
    if (e != cudaSuccess) return e;
    return launch(counts_kernel, dim3((unsigned)((M + 255) / 256)), dim3(256), 0, st, idx, mask, M,
                  K, N, counts, n_tokens, status);
}

namespace {
// word 1 of the header: some count above kExactCount; 2: kept tokens; 3: CTAs done
cudaError_t launch_prep(BalPrep &p, void *ws, const BalanceWs &w, cudaStream_t st) {
    p.ld = w.ld;
    p.pr = pad64(p.N_r);
    p.pc = pad64(p.N_c);
    p.seg_r = w.ld - p.pc;
    p.P_hi = ws_at<uint16_t>(ws, w.P_hi);
    p.P_lo = ws_at<uint16_t>(ws, w.P_lo);
    p.F_hi = ws_at<uint16_t>(ws, w.F_hi);
    p.F_lo = ws_at<uint16_t>(ws, w.F_lo);
    p.big = ws_at<int>(ws, 4);
    p.n_local = ws_at<int>(ws, 8);
    const int64_t units = (int64_t)p.L * (p.ld / 8), tiles = (int64_t)(p.pr / 32) * (p.pc / 32);
    int64_t want = (units + kPrepThreads - 1) / kPrepThreads;
    if (want < tiles) want = tiles;
    const int64_t most = (int64_t)device_sm_count() * 8;
    return launch(balance_prep_kernel, dim3((unsigned)(want < most ? want : most)),
                  dim3(kPrepThreads), 0, st, p);
}
}  // namespace

cudaError_t launch_balance_fwd(const float *p_r, const float *p_c, const int32_t *counts,
                               const int32_t *n_tokens, const uint8_t *mask, int L, int N_r,
                               int N_c, int K, float *loss, float *token_loss, void *ws,
                               cudaStream_t st) {
    const BalanceWs w = balance_ws(L, 0, N_r, N_c, false);
    BalPrep pp = {};
    pp.p_r = p_r; pp.p_c = p_c; pp.counts = counts; pp.mask = mask;
    pp.L = L; pp.N_r = N_r; pp.N_c = N_c;
    cudaError_t e = launch_prep(pp, ws, w, st);
    if (e != cudaSuccess) return e;
    GemmArgs g = {};
    GemmProb &p = g.prob[0];
    p.M = L; p.N = N_r; p.nk = pp.pc / BK; p.a_hi = 0; p.a_lo = 1; p.b = 2; p.b2 = 3; p.p = p_r;
    set_tiles(&p, 32);
    g.nprob = 1; g.tiles = p.tiles; g.big = pp.big; g.mask = mask;
    g.part = ws_at<float>(ws, w.part);
    g.status = ws_at<int>(ws, 0);
    GemmMaps maps;
    if (!make_sw128_map(&maps.m[0], pp.P_hi, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[1], pp.P_lo, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[2], pp.F_hi, N_r, pp.pc, p.bn) ||
        !make_sw128_map(&maps.m[3], pp.F_lo, N_r, pp.pc, p.bn))
        return cudaErrorInvalidValue;
    if ((e = launch_gemm<kFwd>(maps, g, st)) != cudaSuccess) return e;
    return launch(balance_loss_kernel, dim3((unsigned)((L + kLossThreads - 1) / kLossThreads)),
                  dim3(kLossThreads), 0, st, (const float *)g.part, w.parts, L, token_loss,
                  ws_at<double>(ws, w.blocks), ws_at<int>(ws, 12),
                  (double)N_r * (double)N_c / (double)K, n_tokens, (const int *)pp.n_local, loss);
}

cudaError_t launch_balance_bwd(const uint16_t *x, const uint16_t *W_r, const uint16_t *W_c,
                               const float *p_r, const float *p_c, const int32_t *counts,
                               const int32_t *n_tokens, const uint8_t *mask,
                               const float *token_loss, int L, int d, int N_r, int N_c, int K,
                               float dloss, float *dx, bool accumulate, float *dW_r, float *dW_c,
                               void *ws, cudaStream_t st) {
    const BalanceWs w = balance_ws(L, d, N_r, N_c, true);
    BalPrep pp = {};
    pp.p_r = p_r; pp.p_c = p_c; pp.counts = counts; pp.mask = mask;
    pp.L = L; pp.N_r = N_r; pp.N_c = N_c; pp.d = d; pp.x = x;
    pp.T_hi = ws_at<uint16_t>(ws, w.T_hi);
    pp.T_lo = ws_at<uint16_t>(ws, w.T_lo);
    // what masked rows of x hold must not meet a zero gradient as NaN
    pp.xs = mask ? ws_at<uint16_t>(ws, w.xs) : nullptr;
    cudaError_t e = launch_prep(pp, ws, w, st);
    if (e != cudaSuccess) return e;
    uint16_t *ds_hi = ws_at<uint16_t>(ws, w.ds_hi), *ds_lo = ws_at<uint16_t>(ws, w.ds_lo);

    GemmArgs g = {};
    g.mask = mask; g.big = pp.big; g.token_loss = token_loss;
    g.n_tokens = n_tokens; g.n_local = pp.n_local;
    g.factor = (float)((double)dloss * N_r * N_c / K);
    g.status = ws_at<int>(ws, 0);
    g.nprob = 2;
    for (int a = 0; a < 2; ++a) {                    // U with ds_r, V with ds_c
        GemmProb &p = g.prob[a];
        p.M = L; p.N = a == 0 ? N_r : N_c;
        p.nk = (a == 0 ? pp.pc : pp.pr) / BK;
        p.a_hi = 0; p.a_lo = 1; p.a_c0 = a == 0 ? pp.pr : 0;
        p.b = 2 + 2 * a; p.b2 = 3 + 2 * a;
        p.p = a == 0 ? p_r : p_c;
        p.seg = a == 0 ? pp.pr : pp.pc;
        p.ds_hi = ds_hi + (a == 0 ? 0 : pp.pr);
        p.ds_lo = ds_lo + (a == 0 ? 0 : pp.pr);
        p.ld_out = w.ld;
        // the pad columns belong to the tiles too: they must be written as zeros
        p.N = p.seg;
        set_tiles(&p, 32);
        p.N = a == 0 ? N_r : N_c;
        g.tiles += p.tiles;
    }
    GemmMaps maps;
    if (!make_sw128_map(&maps.m[0], pp.P_hi, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[1], pp.P_lo, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[2], pp.F_hi, N_r, pp.pc, g.prob[0].bn) ||
        !make_sw128_map(&maps.m[3], pp.F_lo, N_r, pp.pc, g.prob[0].bn) ||
        !make_sw128_map(&maps.m[4], pp.T_hi, N_c, pp.pr, g.prob[1].bn) ||
        !make_sw128_map(&maps.m[5], pp.T_lo, N_c, pp.pr, g.prob[1].bn))
        return cudaErrorInvalidValue;
    if ((e = launch_gemm<kGrid>(maps, g, st)) != cudaSuccess) return e;

    GemmArgs h = {};
    h.status = g.status;
    h.nprob = 3;
    for (int a = 0; a < 2; ++a) {                    // dW_r, dW_c: A is ds^T, K the tokens
        GemmProb &p = h.prob[a];
        p.M = a == 0 ? N_r : N_c; p.N = d;
        p.nk = p.nk1 = (L + BK - 1) / BK;
        p.a_hi = 2; p.a_lo = 3; p.a_c0 = a == 0 ? 0 : pp.pr;
        p.b = p.b2 = 4;
        p.out = a == 0 ? dW_r : dW_c; p.ld_out = d; p.accumulate = 1;
    }
    GemmProb &p = h.prob[2];                         // dx: B is W_r, then W_c
    p.M = L; p.N = d; p.nk = w.ld / BK; p.nk1 = pp.pr / BK;
    p.a_hi = 0; p.a_lo = 1; p.b = 5; p.b2 = 6;
    p.out = dx; p.ld_out = d; p.accumulate = accumulate ? 1 : 0;
    for (int a = 0; a < 3; ++a) {
        set_tiles(&h.prob[a], 64);
        h.tiles += h.prob[a].tiles;
    }
    if (!make_sw128_map(&maps.m[0], ds_hi, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[1], ds_lo, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[2], ds_hi, L, w.ld, 64) ||
        !make_sw128_map(&maps.m[3], ds_lo, L, w.ld, 64) ||
        !make_sw128_map(&maps.m[4], pp.xs ? pp.xs : x, L, d, 64) ||
        !make_sw128_map(&maps.m[5], W_r, N_r, d, 64) ||
        !make_sw128_map(&maps.m[6], W_c, N_c, d, 64))
        return cudaErrorInvalidValue;
    return launch_gemm<kGrads>(maps, h, st);
}

}  // namespace omni
