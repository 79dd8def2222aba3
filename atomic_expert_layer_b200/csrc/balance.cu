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
// All products run as fp16 tcgen05 tile GEMMs with fp32 accumulation on CTA
// pairs.  An operand that is fp32 by nature (P, ds) enters as the sum of two
// fp16 values, hi + lo (22 bits), against one that fp16 holds exactly; both
// halves meet the same B tile, so it is loaded once.  Powers of two keep the
// operands inside fp16's range, and come out again in the epilogue:
//   P by 2^14 (22 bits, or 2^-39 of 1 where that is coarser);
//   counts by 2^-16: exact up to 2048.  When some count is larger, what its
//     rounding leaves is a second matrix F_lo, and hi * F_lo is added;
//   ds / c = P (U - l): a token's by the power of two that takes its l, which
//     bounds them, to 2^13 to 2^14.  dx gets it out again row by row; for dW,
//     which sums over tokens, the token's row of x carries it;
//   x (with the token's power) and W, bf16: so that their largest finite
//     magnitude becomes 2^14 to 2^15.  fp16 then holds every bf16 value down to
//     2^-32 of it exactly.
// bf16 halves (16 bits) need no scales, but left dx and dW off by 2.9e-6 of
// themselves, and by 4e-3 for a collapsed router, where U - l_t cancels.  A
// scale of ds by the largest count left 6e-5 at 1304 x 1304 and 1e-2 at 8192 x
// 8192 where spread probabilities meet tasks on one expert.  With these, and
// with what kChunk below says, the gradients' errors against 64 bits are 0.4 to
// 1.6 times those of torch in fp32: headline 5.6e-7 and 1.2e-6, skewed layer
// 1.3e-6 to 2.3e-6 and 1.8e-6 to 2.7e-6 (five seeds).  The losses' are up to 2.6
// times (8e-8 and 3e-8), and the gradients' twice torch's where U and l agree in
// all but their last bits (counts of millions on every expert: 3.5e-5 and
// 1.7e-5), since both are cut off towards zero, by different amounts.
//
// Bounds and measurements, headline layer (L = 4096, d = 1024, 1304 x 1304
// grid, one B200, clocks under load): the products are 28 GFLOP forward, 56 +
// 87 GFLOP backward, twice the definition's because of the halves, against
// 1407 TFLOP/s sustained.  Forward 41 us (20 at that rate), U and V with ds 71
// us (40), dW and dx 87 us (62).  What is above goes to the tiles' output,
// which two accumulators do not cover (U and V without it: 48 us), to handing
// accumulators over every second K step, to the rounds that do not fill 74
// pairs (192 tiles of 256 x 224; 44 tiles of 64 and 64 of 42 K steps).
// Preparing the operands takes 41 us for the two calls (173 MB).
//
// Masked rows of p are never read as numbers: their P and ds are zero.
#include <cuda_fp16.h>

#include "omni_common.cuh"
#include "omni_internal.h"
#include "tcgen05.cuh"

namespace omni {
namespace {

// The scales at which P and the counts are held in fp16.
constexpr float kScaleP = 16384.f;              // 2^14
constexpr float kScaleF = 1.f / 65536.f;        // 2^-16: counts up to 2^31 stay below fp16's largest
constexpr float kUnscale = 4.f;                 // 1 / (kScaleP kScaleF)
constexpr int kExactCount = 2048;               // counts up to this need no F_lo

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

// Words of the workspace header after the status (all zero when a call starts).
struct BalHeader {
    int status;
    int most;            // largest count
    int kept;            // tokens of this batch with mask != 0
    int done;            // CTAs that have finished (forward)
    int x_top;           // largest exponent of the kept rows of x, each with its token's
                         // (kNoExp more; 0: no value but zeros)
    int w_top;           // ... of W_r and W_c
};
constexpr int kNoExp = 512;
// Exponent of a finite magnitude, from its bits as fp32 (subnormals as 2^-126).
__device__ __forceinline__ int exp_of(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127;
    return e < -126 ? -126 : e;
}
// Exponent by which a token's ds is scaled, from its loss: P U and P l are at
// most l, since all terms of l = sum P U are positive and P <= 1, so no |P (U - l)|
// is above it, and the largest is near it where the token's loss lies on few
// experts.  (P may be up to 3.99 where it is not normalised: ds then stays below
// 2^16 x 0.998, which fp16 holds.)  Below 2^-60 some P is under 2^-30 and has lost
// its last bits already; counts below 2^31 give no finite l above 2^40.
__device__ __forceinline__ int token_exp(float l) {
    const int e = exp_of(__float_as_uint(l) & 0x7fffffffu);
    return e < -60 ? -60 : e > 40 ? 40 : e;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// 2^e as two factors, since fp32 holds powers from 2^-126 to 2^127 only.
// Between them a product is never above both its value and its result, and
// below fp32's normal range only where the result is too.
struct Pow2 {
    float a, b;
    __device__ explicit Pow2(int e) {
        e = e < -252 ? -252 : e > 252 ? 252 : e;
        a = pow2f(e >> 1);
        b = pow2f(e - (e >> 1));
    }
};

// ----------------------------------------------------------------- counts
__global__ void counts_clear_kernel(int32_t *__restrict__ counts, int64_t N,
                                    int32_t *__restrict__ n_tokens, int *status) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
#pragma unroll 4
    for (int64_t i = at; i < N; i += (int64_t)gridDim.x * blockDim.x) counts[i] = 0;
    if (at == 0) {
        *n_tokens = 0;
        *status = OMNI_DEV_OK;
    }
}

constexpr int kCountSpan = 4096;        // mask bytes that a CTA counts at a time

// Kept tokens, counted from the mask, 4096 by a CTA: an atomic per token, all
// on one address, took 60 us of 67 at 16384 tokens.
__device__ __forceinline__ void count_tokens(const uint8_t *mask, int L, int32_t *n_tokens) {
    if (!mask) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *n_tokens = L;
        return;
    }
    int kept = 0;
    for (int64_t t = (int64_t)blockIdx.x * kCountSpan; t < L; t += (int64_t)gridDim.x * kCountSpan)
        for (int i = (int)threadIdx.x; i < kCountSpan && t + i < L; i += (int)blockDim.x)
            kept += mask[t + i] != 0;
    kept = warp_isum(kept);
    if (kept && lane_id() == 0) atomicAdd(n_tokens, kept);
}

// One thread per task; integer atomics, so the counts do not depend on the
// order.
__global__ void __launch_bounds__(256)
counts_kernel(const int32_t *__restrict__ idx, const uint8_t *__restrict__ mask, int M, int K, int N,
              int32_t *__restrict__ counts, int32_t *__restrict__ n_tokens, int *status) {
    grid_dependency_wait();
    grid_dependents_launch();
    const unsigned at = blockIdx.x * 256 + threadIdx.x;       // M < 2^31: no wrap
    if (at < (unsigned)M && (!mask || mask[at / (unsigned)K])) {
        const int e = idx[at];
        if (e >= 0 && e < N) atomicAdd(&counts[e], 1);
        else set_status(status, OMNI_DEV_BAD_EXPERT);
    }
    count_tokens(mask, M / K, n_tokens);
}

// The same for crowded experts, whose atomics would wait for one another (2 to
// 4 ns each on one address): a CTA first counts its tasks in a table in shared
// memory, one expert to a slot; a task whose slot another expert holds goes to
// memory by itself.
constexpr int kCrowdThreads = 512, kCrowdTasks = 8192, kCrowdSlots = 4096;
__global__ void __launch_bounds__(kCrowdThreads)
counts_crowded_kernel(const int32_t *__restrict__ idx, const uint8_t *__restrict__ mask, int M, int K,
                      int N, int32_t *__restrict__ counts, int32_t *__restrict__ n_tokens, int *status) {
    __shared__ int key[kCrowdSlots], hits[kCrowdSlots];
    for (int i = (int)threadIdx.x; i < kCrowdSlots; i += kCrowdThreads) {
        key[i] = -1;
        hits[i] = 0;
    }
    grid_dependency_wait();
    grid_dependents_launch();
    __syncthreads();
    const unsigned first = blockIdx.x * (unsigned)kCrowdTasks;
#pragma unroll 4
    for (unsigned i = threadIdx.x; i < (unsigned)kCrowdTasks; i += kCrowdThreads) {
        const unsigned at = first + i;                        // M < 2^31: no wrap
        if (at >= (unsigned)M || (mask && !mask[at / (unsigned)K])) continue;
        const int e = idx[at];
        if (e < 0 || e >= N) {
            set_status(status, OMNI_DEV_BAD_EXPERT);
            continue;
        }
        const unsigned slot = (unsigned)e * 2654435761u >> 20;
        const int held = atomicCAS(&key[slot], -1, e);
        if (held == -1 || held == e) atomicAdd(&hits[slot], 1);
        else atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int i = (int)threadIdx.x; i < kCrowdSlots; i += kCrowdThreads)
        if (hits[i]) atomicAdd(&counts[key[i]], hits[i]);
    count_tokens(mask, M / K, n_tokens);
}

// -------------------------------------------------------------- operands
struct BalPrep {
    const float *p_r, *p_c;
    const int32_t *counts;
    const uint8_t *mask;
    const uint16_t *x, *W_r, *W_c;   // backward (else null): their largest magnitudes are wanted
    const float *token_loss;      // ..., beside x's
    int L, N_r, N_c, d;
    int seg_r, ld;                // columns of the row segment, and of P (0: only the column axis)
    int pc, pr;                   // padded N_c, N_r
    uint16_t *P_hi, *P_lo, *F_hi, *F_lo, *T_hi, *T_lo;
    BalHeader *hdr;
};

// Whether 16-byte pieces at 16-byte boundaries that hold a value of row t of
// p [L, N] lie within p: they reach at most 3 values past the row.
__device__ __forceinline__ bool whole_pieces(const float *p, int64_t t, int64_t L, int N) {
    const int beside = N >= 3 ? 1 : 3;
    return ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (N & 3) == 0) ||
           (t >= beside && t < L - beside);
}

// 8 log-probabilities of a row with whole_pieces, from `at` on, of which `valid`
// exist (the others read as -inf).  A row starts at any multiple of 4 bytes, so
// they come as the 2 or 3 pieces that hold at least one of them, shifted into
// place; what else a piece holds is dropped.  At 6001 tokens and 1101 x 1303 the
// U product takes 47 us so (58 with 4-byte loads) and the preparation 52 (58); at
// 4096 tokens and 1304 x 1304 they take 40 and 42.5 us (41 and 41.5 with a branch
// of its own for aligned rows).
__device__ __forceinline__ void load_logp8(const float *at, int valid, float *v) {
    const int m = (int)(reinterpret_cast<uintptr_t>(at) >> 2) & 3;
    const float4 *piece = reinterpret_cast<const float4 *>(at - m);
    float w[12];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (4 * k - m < valid && (k < 2 || m > 0)) c = piece[k];
        w[4 * k] = c.x, w[4 * k + 1] = c.y, w[4 * k + 2] = c.z, w[4 * k + 3] = c.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = m < 2 ? (m == 0 ? w[i] : w[i + 1]) : (m == 2 ? w[i + 2] : w[i + 3]);
        if (i >= valid) v[i] = -INFINITY;
    }
}

// A warp's 256 columns of a row of P: both segments, the padding as zeros.
__device__ __forceinline__ void prep_probs(const BalPrep &p, int64_t t, int c0) {
    c0 += 8 * (int)lane_id();
    if (c0 >= p.ld) return;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (!p.mask || p.mask[t]) {
        const bool rows = c0 < p.seg_r;
        const int col = rows ? c0 : c0 - p.seg_r, n = rows ? p.N_r : p.N_c;
        const float *src = rows ? p.p_r : p.p_c;
        const float *at = src + t * n + col;
        if (whole_pieces(src, t, p.L, n)) {
            load_logp8(at, n - col, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = col + i < n ? at[i] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = kScaleP * expf(v[i]);
    }
    uint4 hi, lo;
    split8_f16(v, &hi, &lo);
    *reinterpret_cast<uint4 *>(p.P_hi + t * p.ld + c0) = hi;
    *reinterpret_cast<uint4 *>(p.P_lo + t * p.ld + c0) = lo;
}

// The pieces (row, part) that a warp takes, `warps` apart in row-major order.
struct Pieces {
    int64_t row, drow;
    int part, dpart, parts;
    __device__ Pieces(int64_t first, int64_t warps, int n) : parts(n) {
        row = first / n;
        part = (int)(first % n);
        drow = warps / n;
        dpart = (int)(warps % n);
    }
    __device__ void next() {
        row += drow;
        part += dpart;
        if (part >= parts) {
            part -= parts;
            ++row;
        }
    }
};

constexpr int kPrepThreads = 256, kPrepPerSm = 8;     // all of the grid resident: 32 registers

// Largest finite magnitude of 8 bf16 values, as fp32 bits.
__device__ __forceinline__ uint32_t top8(const uint4 &u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = (w[i] << 16) & 0x7fff0000u, b = w[i] & 0x7fff0000u;
        if (a < 0x7f800000u) m = max(m, a);
        if (b < 0x7f800000u) m = max(m, b);
    }
    return m;
}
// ... of a warp's 1024 columns of a row of d8 vectors, four loads at a time
__device__ __forceinline__ uint32_t top_row(const uint16_t *row, int part, int d8) {
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = part * 128 + 32 * i + (int)lane_id();
        u[i] = c < d8 ? reinterpret_cast<const uint4 *>(row)[c] : make_uint4(0, 0, 0, 0);
    }
    return max(max(top8(u[0]), top8(u[1])), max(top8(u[2]), top8(u[3])));
}

// Largest value of the CTA's threads into *out, with an atomic only where it is
// larger than what is there: atomics on one address take 2 to 4 ns each, one
// after another, so one per warp (9472 of them) cost more than the reading.
template <typename T>
__device__ __forceinline__ void cta_max(T m, T *out) {
    __shared__ T best;
    __syncthreads();
    if (threadIdx.x == 0) best = 0;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, m);
    if (m && lane_id() == 0) atomicMax(&best, m);
    __syncthreads();
    if (threadIdx.x == 0 && best > *reinterpret_cast<volatile T *>(out)) atomicMax(out, best);
}

// Two values at `at` as hi and lo.
__device__ __forceinline__ void store_pair(uint16_t *hi, uint16_t *lo, int64_t at, float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    *reinterpret_cast<__half2 *>(hi + at) = h;
    *reinterpret_cast<__half2 *>(lo + at) = __floats2half2_rn(a - f.x, b - f.y);
}

// Work of a CTA: the 64 x 64 tiles of the counts (F and its transpose, padded
// with zeros), then rows of P and the magnitudes of x and W.
__global__ void __launch_bounds__(kPrepThreads, kPrepPerSm) balance_prep_kernel(const BalPrep p) {
    __shared__ float tile[64][65];
    grid_dependency_wait();
    grid_dependents_launch();
    const int tr = p.pr / 64, tc = p.pc / 64;
    const bool even = (p.N_c & 1) == 0 && (reinterpret_cast<uintptr_t>(p.counts) & 7u) == 0;
    int most = 0;
    for (int u = blockIdx.x; u < tr * tc; u += gridDim.x) {
        const int i0 = (u / tc) * 64, j0 = (u % tc) * 64;
        const int a = (int)threadIdx.x >> 5, l2 = 2 * ((int)threadIdx.x & 31);
        int2 c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + a + 8 * k, j = j0 + l2;
            const int32_t *src = p.counts + (int64_t)i * p.N_c + j;
            c[k] = make_int2(0, 0);
            if (i < p.N_r) {
                if (even && j < p.N_c) c[k] = *reinterpret_cast<const int2 *>(src);
                if (!even && j < p.N_c) c[k].x = src[0];
                if (!even && j + 1 < p.N_c) c[k].y = src[1];
            }
        }
        __syncthreads();                             // the tile is free again
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = a + 8 * k, i = i0 + r;
            most = max(most, max(c[k].x, c[k].y));
            const float f[2] = {(float)c[k].x * kScaleF, (float)c[k].y * kScaleF};
            tile[r][l2] = f[0];
            tile[r][l2 + 1] = f[1];
            if (i < p.N_r) store_pair(p.F_hi, p.F_lo, (int64_t)i * p.pc + j0 + l2, f[0], f[1]);
        }
        __syncthreads();
        if (p.T_hi) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = a + 8 * k, j = j0 + r;
                if (j < p.N_c)
                    store_pair(p.T_hi, p.T_lo, (int64_t)j * p.pr + i0 + l2, tile[l2][r], tile[l2 + 1][r]);
            }
        }
    }
    cta_max(most, &p.hdr->most);

    // one warp per 256 columns of a row from here on
    const int64_t warps = (int64_t)gridDim.x * (kPrepThreads / 32);
    const int64_t w0 = (int64_t)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    for (Pieces u(w0, warps, (p.ld + 255) / 256); u.row < p.L; u.next())
        prep_probs(p, u.row, u.part * 256);
    if (p.x) {
        const int d8 = p.d >> 3, dp = (d8 + 127) / 128;
        int top = 0;
        for (Pieces u(w0, warps, dp); u.row < p.L; u.next()) {
            if (p.mask && !p.mask[u.row]) continue;
            const uint32_t m = top_row(p.x + u.row * p.d, u.part, d8);
            if (m) top = max(top, kNoExp + exp_of(m) + token_exp(p.token_loss[u.row]));
        }
        cta_max(top, &p.hdr->x_top);
        uint32_t w_top = 0;
        for (Pieces u(w0, warps, dp); u.row < p.N_r + p.N_c; u.next())
            w_top = max(w_top, top_row(u.row < p.N_r ? p.W_r + u.row * p.d
                                                     : p.W_c + (u.row - p.N_r) * p.d, u.part, d8));
        cta_max(w_top ? kNoExp + exp_of(w_top) : 0, &p.hdr->w_top);
    }
    if (!p.mask) {
        if (blockIdx.x == 0 && threadIdx.x == 0) p.hdr->kept = p.L;
    } else {
        // a few CTAs count, with one atomic each
        int kept = 0;
        for (int64_t t = (int64_t)blockIdx.x * kCountSpan; t < p.L; t += (int64_t)gridDim.x * kCountSpan)
            for (int i = (int)threadIdx.x; i < kCountSpan && t + i < p.L; i += kPrepThreads)
                kept += p.mask[t + i] != 0;
        kept = warp_isum(kept);
        if (kept && lane_id() == 0) atomicAdd(&p.hdr->kept, kept);
    }
}

// x and W in fp16, scaled: each row of x also by its token's power of two, which
// its ds lacks; masked rows of x as zeros (what they hold must not meet a zero
// gradient as NaN), W_r and W_c one under the other with zero rows between, as
// the columns of ds lie.
struct BalCast {
    const uint16_t *x, *W_r, *W_c;
    const uint8_t *mask;
    const float *token_loss;
    int L, N_r, N_c, d, pr, ld;
    uint16_t *x16, *w16;
    const BalHeader *hdr;
};
__global__ void __launch_bounds__(kPrepThreads) balance_cast_kernel(const BalCast p) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int x_exp = 14 + kNoExp - p.hdr->x_top, w_exp = 14 + kNoExp - p.hdr->w_top;
    const int d8 = p.d >> 3;
    const int64_t warps = (int64_t)gridDim.x * (kPrepThreads / 32);
    for (int64_t row = (int64_t)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
         row < (int64_t)p.L + p.ld; row += warps) {
        const bool w = row >= p.L;
        const int64_t r = w ? row - p.L : row;
        const uint16_t *src = nullptr;
        if (!w) {
            if (!p.mask || p.mask[r]) src = p.x + r * p.d;
        } else if (r < p.pr) {
            if (r < p.N_r) src = p.W_r + r * p.d;
        } else if (r - p.pr < p.N_c) {
            src = p.W_c + (r - p.pr) * p.d;
        }
        uint4 *dst = reinterpret_cast<uint4 *>((w ? p.w16 : p.x16) + r * p.d);
        const Pow2 s(w ? w_exp : x_exp + (src ? token_exp(p.token_loss[r]) : 0));
        for (int c = (int)lane_id(); c < d8; c += 32) {
            uint4 o = make_uint4(0, 0, 0, 0);
            if (src) {
                const uint4 in = reinterpret_cast<const uint4 *>(src)[c];
                const uint32_t a[4] = {in.x, in.y, in.z, in.w};
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 b = __floats2half2_rn(__uint_as_float(a[i] << 16) * s.a * s.b,
                                                        __uint_as_float(a[i] & 0xffff0000u) * s.a * s.b);
                    h[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
                o = make_uint4(h[0], h[1], h[2], h[3]);
            }
            dst[c] = o;
        }
    }
}

// -------------------------------------------------------------- tile GEMM
// C[M, N] = (A_hi + A_lo) B over a K axis of 64-element steps, tiles of 256 x
// bn, each computed by a pair of CTAs (a cluster of 2, cta_group::2): CTA r
// holds rows 128 r .. + 127 of A (hi and lo) and half of the B tile in its
// shared memory, the pair's first CTA issues the MMAs, and each CTA's TMEM
// receives its 128 rows of C.  With both halves of A in shared memory a CTA
// of its own (128 x 256 tiles) would read 96 and fill 64 bytes of it per
// clock, against 128; the pair's halves of B make that 64 and 47.
// An operand is K-major (its K axis contiguous in memory: the products with
// F) or MN-major (its M or N axis contiguous: W and x, and ds as ds^T); either
// way a TMA box is 64 elements (128 bytes, one swizzle atom) wide along the
// contiguous axis.
constexpr int BM = 128, BN = 256, BK = kSwK, STAGES = 4;     // BM: rows of one CTA
constexpr int kBytesA = BM * BK * 2;             // 16 KB, each of hi and lo
constexpr int kBytesB = BN / 2 * BK * 2;         // 16 KB at most: half of the B tile
constexpr int kBlockMN = 64 * BK * 2;            // an MN-major box: 64 K rows of 128 bytes
// All of TMEM: three accumulators for tiles of up to 160 columns (forward at the
// headline: 41.7 us, with two 43.1), two for wider ones.
constexpr uint32_t kTmemCols = 2 * BN;
inline int accumulators(int bn) { return bn <= 160 ? 3 : 2; }
__device__ __forceinline__ uint32_t acc_column(int accs, int buf) {
    return (uint32_t)buf * (accs == 3 ? 160u : (uint32_t)BN);
}
constexpr int kEpiWarps = 8;                     // two per TMEM lane quarter
constexpr int kEpiBlocks = BN / 64;              // 32-column blocks of a tile for one of them
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kIdescF16 =                   // A and B fp16 (formats 0); the width is added
    umma_idesc_bf16(2 * BM, 0) & ~((1u << 7) | (1u << 10));
constexpr int kMaxProbs = 2, kMaxMaps = 6;
// K steps that are summed in TMEM before the epilogue warps add them to their
// registers.  The tensor core cuts off what falls below its accumulator at
// every instruction, always towards zero: over the 512 instructions of a dW
// tile at L = 4096 that took 1.1e-5 off the result, and it grows with L.  Here
// an accumulator takes the 8 instructions of two lo halves first, while it is
// small, then the 8 of the hi halves; the additions in registers round to
// nearest.  Headline step, and largest error against 64 bits there and at the
// skewed layer: 2 steps 266 us, 5e-7, 1.3e-6; 4 steps 248 us, 7e-7, 2.9e-6; 8
// steps, halves together, 227 us, 2e-6, 5.6e-6 (torch in fp32: 1.2e-6, 1.8e-6
// to 2.7e-6 by the seed).
// A backward tile's first two accumulators take up to kMaxLead steps (a fifth
// of them at most): they are computed while the warps that would drain them
// still write the last tile (headline step 265 -> 258 us; with 8 steps and a
// quarter 250, but 2e-6 at the skewed layer).
constexpr int kChunk = 2, kMaxLead = 4;

struct __align__(1024) GemmSmem {
    uint8_t a[STAGES][2 * kBytesA];
    uint8_t b[STAGES][kBytesB];
    float turn[kEpiWarps][32 * 32];              // an epilogue warp's 32 x 32 block, between its layouts
    uint64_t full[STAGES];                       // used in the pair's first CTA
    uint64_t empty[STAGES];
    uint64_t tfull[3];                           // accumulator ready for the epilogue
    uint64_t tempty[3];                          // accumulator drained (first CTA: both CTAs' warps)
    uint32_t tmem_base;
    int abort;
};

struct GemmProb {
    int M, N;                     // rows and columns of C
    int bn, tiles_n, tiles;       // tile width, tiles in N, tiles in all
    int nk;                       // 64-element steps of the K axis
    int lead;                     // steps of a tile's first two accumulators
    int a_mn;                     // A is MN-major (ds^T, for dW)
    int a_hi, a_lo;               // tensor maps of A
    int a_c0;                     // first column of A's segment in its matrix
    int b, b_lo;                  // maps of B, and of the remainder F_lo
    const float *p;               // forward: log-probabilities beside this C
    const uint16_t *P_hi, *P_lo;  // backward: P beside this C, column 0 of its segment
    uint16_t *ds_hi, *ds_lo;      // their gradient, column 0 of this segment
    int seg;                      // columns of the segment (N padded to 64; the pad gets zeros)
    float *out, *out2;            // C in fp32: rows below `split`, and from `split` on
    int split, rows1, rows2;      // rows of out and of out2 (the others are padding)
    int accumulate;
};

struct GemmArgs {
    GemmProb prob[kMaxProbs];     // the one with the longer K axis first
    int nprob, tiles;
    int accs;                     // accumulators in TMEM
    int ld;                       // columns of ds
    const uint8_t *mask;
    float *part;                  // forward: sums over a tile's columns [tiles_n * 2, L]
    const float *token_loss;      // backward
    const int32_t *n_tokens;
    double factor;                // dloss N / K
    BalHeader *hdr;
};
struct GemmMaps { CUtensorMap m[kMaxMaps]; };

// what a launch computes: U with the forward's sums; U and V with ds; dW and dx
enum : int { kFwd = 0, kGrid = 1, kGrads = 2 };

// Tiles are dealt out back and forth over the pairs, longest first, so that
// the pairs with a long first tile get the last of the short ones.
__device__ __forceinline__ int tile_of(int turn, int tiles) {
    const int pairs = (int)(gridDim.x >> 1), pair = (int)(blockIdx.x >> 1);
    const int64_t i = (int64_t)turn * pairs + ((turn & 1) ? pairs - 1 - pair : pair);
    return i < tiles ? (int)i : -1;
}
__device__ __forceinline__ bool turns_left(int turn, int tiles) {
    return (int64_t)turn * (gridDim.x >> 1) < tiles;
}

__device__ __forceinline__ int find_prob(const GemmArgs &g, int *tile) {
    if (g.nprob == 1 || *tile < g.prob[0].tiles) return 0;
    *tile -= g.prob[0].tiles;
    return 1;
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

// K steps of the accumulator that begins at step st.
template <int MODE>
__device__ __forceinline__ int chunk_steps(const GemmProb &p, int st, int steps) {
    const int n = MODE != kFwd && st < 2 * p.lead ? p.lead : kChunk;
    return min(n, steps - st);
}

// Arrive on the pair's first CTA's barrier.  What it orders are TMEM reads,
// which have completed (tcgen05.wait::ld, then the fence before thread
// synchronisation; the issuer fences after its wait); no other memory that one
// CTA writes is read by the other.  At cluster scope (and with acquires at
// cluster scope on the other side) each arrive would also wait for the warp's
// global stores, and each wait drop the SM's L1.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *at) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// Word of element (r, c) of a warp's 32 x 32 block: rows and columns are both
// read and written without bank conflicts.
__device__ __forceinline__ int turned(int r, int c) { return r * 32 + (c ^ r); }

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
balance_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs g) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    GemmSmem &sm = *reinterpret_cast<GemmSmem *>(smem_raw + pad);
    const int warp = threadIdx.x >> 5;
    const unsigned lane = lane_id();
    const uint32_t rank = cluster_ctarank();         // 0: issues the MMAs
    int *status = &g.hdr->status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 3; ++b) {
            mbar_init(&sm.tfull[b], 1);
            mbar_init(&sm.tempty[b], 2 * kEpiWarps);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&sm.tmem_base)), "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                  // both CTAs' barriers exist
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    grid_dependency_wait();
    grid_dependents_launch();
    const bool big = MODE != kGrads && g.hdr->most > kExactCount;

    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer (both CTAs): completion counted on the first CTA's barrier
            int it = 0, issued_from = 0;
            for (int turn = 0; !sm.abort && turns_left(turn, g.tiles); ++turn) {
                int tile = tile_of(turn, g.tiles);
                if (tile < 0) continue;
                const GemmProb &p = g.prob[find_prob(g, &tile)];
                const int m0 = (tile / p.tiles_n) * 2 * BM + (int)rank * BM;
                const int n0 = (tile % p.tiles_n) * p.bn + (int)rank * (p.bn / 2);
                const int steps = steps_of<MODE>(p, big);
                const bool a_mn = MODE == kGrads && p.a_mn;
                for (int st = 0; st < steps; ++st, ++it) {
                    const int s = it % STAGES;
                    if (it >= STAGES &&
                        !mbar_wait(&sm.empty[s], (uint32_t)(((it / STAGES) - 1) & 1), status)) {
                        sm.abort = 1;
                        break;
                    }
                    const bool rest = MODE != kGrads && st >= p.nk;      // hi times F_lo
                    const int kb = rest ? st - p.nk : st;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&sm.full[s],
                                              (uint32_t)(2 * (rest ? 1 : 2) * kBytesA + p.bn * BK * 2));
                    const uint32_t fb = smem_in_cta(&sm.full[s], 0);
                    uint8_t *a = sm.a[s], *b = sm.b[s];
                    if (a_mn) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            tma_load_2d_pair(a + i * kBlockMN, &maps.m[p.a_hi], m0 + 64 * i, kb * BK, fb);
                            tma_load_2d_pair(a + kBytesA + i * kBlockMN, &maps.m[p.a_lo], m0 + 64 * i,
                                             kb * BK, fb);
                        }
                    } else {
                        tma_load_2d_pair(a, &maps.m[p.a_hi], p.a_c0 + kb * BK, m0, fb);
                        if (!rest)
                            tma_load_2d_pair(a + kBytesA, &maps.m[p.a_lo], p.a_c0 + kb * BK, m0, fb);
                    }
                    if (MODE == kGrads) {
                        for (int j = 0; j < p.bn / 128; ++j)
                            tma_load_2d_pair(b + j * kBlockMN, &maps.m[p.b], n0 + 64 * j, kb * BK, fb);
                    } else {
                        tma_load_2d_pair(b, &maps.m[rest ? p.b_lo : p.b], kb * BK, n0, fb);
                    }
                    issued_from = it + 1 > STAGES ? it + 1 - STAGES : 0;
                }
            }
            if (sm.abort && rank == 0) {
                // let the loads already issued land before the CTA can exit
                for (int k = issued_from; k < it; ++k)
                    mbar_wait(&sm.full[k % STAGES], (uint32_t)((k / STAGES) & 1), status);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---- MMA issuer (the pair's first CTA)
            int it = 0, buf = 0, wrap = 0;
            bool ok = true;
            for (int turn = 0; ok && turns_left(turn, g.tiles); ++turn) {
                int tile = tile_of(turn, g.tiles);
                if (tile < 0) continue;
                const GemmProb &p = g.prob[find_prob(g, &tile)];
                const int steps = steps_of<MODE>(p, big);
                const bool a_mn = MODE == kGrads && p.a_mn;
                // bits 15 and 16 of the instruction descriptor: A, B are MN-major
                const uint32_t idesc = kIdescF16 | ((uint32_t)(p.bn >> 3) << 17) |
                                       (a_mn ? 1u << 15 : 0u) | (MODE == kGrads ? 1u << 16 : 0u);
                // a 16-deep slice: 32 bytes along a K-major atom, or 16 K rows
                const uint64_t a_step = (a_mn ? 16 * 128 : 32) >> 4;
                constexpr uint64_t b_step = (MODE == kGrads ? 16 * 128 : 32) >> 4;
                const uint64_t a0 = a_mn ? sw128_desc_mn(sm.a[0]) : sw128_desc(sm.a[0]);
                const uint64_t b0 = MODE == kGrads ? sw128_desc_mn(sm.b[0]) : sw128_desc(sm.b[0]);
                // one half of A (hi: 0, lo: kBytesA) of stage s times its B
                const auto products = [&](uint32_t acc, int s, int half, uint32_t started) {
                    uint64_t ad = a0 + (uint64_t)((s * 2 * kBytesA + half) >> 4);
                    uint64_t bd = b0 + (uint64_t)((s * kBytesB) >> 4);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        umma_bf16_pair(acc, ad, bd, idesc, k > 0 ? 1u : started);
                        ad += a_step;
                        bd += b_step;
                    }
                };
                for (int st = 0, n; st < steps; st += n) {
                    n = chunk_steps<MODE>(p, st, steps);
                    if (wrap > 0 && !mbar_wait(&sm.tempty[buf], (uint32_t)((wrap - 1) & 1), status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t acc = tmem + acc_column(g.accs, buf);
                    uint32_t started = 0;
                    // step i's lo half goes before step i - 1's hi half
                    for (int i = 0; i <= n; ++i) {
                        if (i < n) {
                            const int s = (it + i) % STAGES;
                            if (!mbar_wait(&sm.full[s], (uint32_t)(((it + i) / STAGES) & 1), status)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (MODE == kGrads || st + i < p.nk) {    // (hi only times F_lo)
                                products(acc, s, kBytesA, started);
                                started = 1;
                            }
                        }
                        if (i > 0) {
                            const int s = (it + i - 1) % STAGES;
                            products(acc, s, 0, started);
                            started = 1;
                            umma_commit_pair(&sm.empty[s]);           // frees stage s in both CTAs
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair(&sm.tfull[buf]);         // both CTAs' epilogues may read
                    it += n;
                    if (++buf == g.accs) {
                        buf = 0;
                        ++wrap;
                    }
                }
            }
            if (!ok) sm.abort = 1;
        }
        __syncwarp();
    } else {
        // ---- epilogue: warp w reads TMEM lanes 32*(w % 4) .. +31 (this CTA's
        // rows of the tile) and every second block of 32 columns
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const uint32_t tempty = smem_in_cta(&sm.tempty[0], 0);
        float *turn_buf = sm.turn[warp - 2];
        // kGrads: c, as a number of magnitude 1 to 2 and an exponent that the scales join
        float coef = 0.f;
        int coef_exp = 0;
        if (MODE == kGrads) {
            const int n = *g.n_tokens, kept = g.hdr->kept;
            if (n > 0 && kept > 0) {
                const double c = g.factor / n / kept;
                if (c != 0.0 && isfinite(c)) coef_exp = ilogb(c);
                coef = (float)scalbn(c, -coef_exp);
            }
        }
        int buf = 0, wrap = 0;
        bool ok = true;
        for (int turn = 0; ok && turns_left(turn, g.tiles); ++turn) {
            int tile = tile_of(turn, g.tiles);
            if (tile < 0) continue;
            const GemmProb &p = g.prob[find_prob(g, &tile)];
            const int row0 = (tile / p.tiles_n) * 2 * BM + (int)rank * BM + quarter * 32;
            const int tn = tile % p.tiles_n, n0 = tn * p.bn;
            const int steps = steps_of<MODE>(p, big), blocks = p.bn / 32;
            const int row = row0 + (int)lane;
            // what the tile's end will read of this lane's row is asked of L2 now
            if (row < p.M) {
                for (int q = half; q < blocks; q += 2) {
                    const int col = n0 + 32 * q;
                    if (MODE == kFwd && col < p.N) prefetch_l2(p.p + (int64_t)row * p.N + col);
                    if (MODE == kGrid && col < p.seg) {
                        prefetch_l2(p.P_hi + (int64_t)row * g.ld + col);
                        prefetch_l2(p.P_lo + (int64_t)row * g.ld + col);
                    }
                    if (MODE == kGrads && p.accumulate && col < p.N) {
                        const bool second = row >= p.split;
                        const int m = second ? row - p.split : row;
                        if (m < (second ? p.rows2 : p.rows1))
                            prefetch_l2((second ? p.out2 : p.out) + (int64_t)m * p.N + col);
                    }
                }
            }
            float sum[kEpiBlocks][32];
#pragma unroll
            for (int q = 0; q < kEpiBlocks; ++q)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[q][j] = 0.f;
            for (int st = 0; st < steps; st += chunk_steps<MODE>(p, st, steps)) {
                // the warp gives up as one: its lanes meet again below
                const bool got = mbar_wait(&sm.tfull[buf], (uint32_t)(wrap & 1), status);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + acc_column(g.accs, buf);
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
                // this accumulator may be overwritten once every epilogue warp of
                // both CTAs is done (the first CTA's barrier counts all 16)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(tempty + 8u * (uint32_t)buf);
                if (++buf == g.accs) {
                    buf = 0;
                    ++wrap;
                }
            }
            if (!ok) break;
            // a masked row has P = 0, its sums are finite and its token_loss is not used
            const bool keep = MODE != kGrads && row < p.M && (!g.mask || g.mask[row]);
            const bool whole = MODE == kFwd && whole_pieces(p.p, row, p.M, p.N);
            const uint32_t apart = MODE == kFwd ? __ballot_sync(0xffffffffu, keep && !whole) : 0u;
            const float l_t = MODE == kGrid && keep ? g.token_loss[row] : 0.f;
            // kGrid: ds / c to 2^14 at most, P's 2^14 out.  kGrads: the scales of ds
            // (2^(13 - token_exp)) and of the other operand out again
            const float row_scale = MODE == kGrid ? pow2f(-1 - token_exp(l_t)) : 1.f;
            int out_exp = 0;
            if (MODE == kGrads) {
                out_exp = coef_exp - 27 - kNoExp + (p.a_mn ? g.hdr->x_top : g.hdr->w_top);
                if (!p.a_mn && row < p.M) out_exp += token_exp(g.token_loss[row]);
            }
            const Pow2 out_scale(out_exp);
            float part = 0.f;
#pragma unroll
            for (int q = 0; q < kEpiBlocks; ++q) {
                const int col0 = n0 + 32 * (half + 2 * q);
                if (half + 2 * q >= blocks || col0 >= (MODE == kGrid ? p.seg : p.N)) break;
                if constexpr (MODE == kFwd) {
                    // each lane its own row: the sums stay where they are.  Rows at the
                    // array's ends come through shared memory.
                    for (uint32_t m = apart; m != 0; m &= m - 1) {
                        const int r = __ffs((int)m) - 1, col = col0 + (int)lane;
                        if (col < p.N) turn_buf[32 * r + (int)lane] = p.p[(int64_t)(row0 + r) * p.N + col];
                    }
                    __syncwarp();
                    if (keep) {
                        const float *src = whole ? p.p + (int64_t)row * p.N + col0 : turn_buf + 32 * (int)lane;
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            float v[8];
                            load_logp8(src + j, p.N - col0 - j, v);
#pragma unroll
                            for (int k = 0; k < 8; ++k) part = fmaf(expf(v[k]), sum[q][j + k], part);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        turn_buf[turned((int)lane, j)] = MODE == kGrads
                            ? sum[q][j] * coef * out_scale.a * out_scale.b
                            : (kUnscale * sum[q][j] - l_t) * row_scale;
                    __syncwarp();
                }
                if constexpr (MODE == kGrid) {
                    // eight rows at a time, eight columns to a lane; P as the operand holds it
                    const int c = 8 * ((int)lane & 3), r0 = (int)lane >> 2;
                    const int64_t at = (int64_t)(row0 + r0) * g.ld + col0 + c;
#pragma unroll 1
                    for (int i2 = 0; i2 < 4; i2 += 2) {
                        uint4 hi[2], lo[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int64_t o = at + 8 * (i2 + i) * g.ld;
                            const bool in = row0 + r0 + 8 * (i2 + i) < p.M;
                            hi[i] = in ? __ldg(reinterpret_cast<const uint4 *>(p.P_hi + o)) : make_uint4(0, 0, 0, 0);
                            lo[i] = in ? __ldg(reinterpret_cast<const uint4 *>(p.P_lo + o)) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = r0 + 8 * (i2 + i);
                            const uint4 h4 = hi[i], l4 = lo[i];
                            const uint32_t wh[4] = {h4.x, h4.y, h4.z, h4.w}, wl[4] = {l4.x, l4.y, l4.z, l4.w};
                            uint32_t oh[4], ol[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 ph = __half22float2(*reinterpret_cast<const __half2 *>(&wh[k]));
                                const float2 pl = __half22float2(*reinterpret_cast<const __half2 *>(&wl[k]));
                                const float a = (ph.x + pl.x) * turn_buf[turned(r, c + 2 * k)];
                                const float b = (ph.y + pl.y) * turn_buf[turned(r, c + 2 * k + 1)];
                                const __half2 h = __floats2half2_rn(a, b);
                                const float2 f = __half22float2(h);
                                const __half2 o = __floats2half2_rn(a - f.x, b - f.y);
                                oh[k] = *reinterpret_cast<const uint32_t *>(&h);
                                ol[k] = *reinterpret_cast<const uint32_t *>(&o);
                            }
                            if (row0 + r < p.M) {
                                const int64_t o = at + 8 * (i2 + i) * g.ld;
                                *reinterpret_cast<uint4 *>(p.ds_hi + o) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                                *reinterpret_cast<uint4 *>(p.ds_lo + o) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                            }
                        }
                    }
                } else if constexpr (MODE == kGrads) {
                    // four rows at a time, four columns to a lane
                    const int c = 4 * ((int)lane & 7), col = col0 + c, r0 = (int)lane >> 3;
                    // a block lies on one side of the split (both are multiples of 32)
                    const bool second = row0 >= p.split;
                    const int m0 = row0 - (second ? p.split : 0) + r0;
                    const int rows = col < p.N ? (second ? p.rows2 : p.rows1) : 0;
                    float *out = (second ? p.out2 : p.out) + (int64_t)m0 * p.N + col;
#pragma unroll 1
                    for (int i4 = 0; i4 < 8; i4 += 4) {
                        float4 prev[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            prev[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (p.accumulate && m0 + 4 * (i4 + i) < rows)
                                prev[i] = *reinterpret_cast<const float4 *>(out + (int64_t)4 * (i4 + i) * p.N);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = r0 + 4 * (i4 + i);
                            float4 v;
                            v.x = turn_buf[turned(r, c)];
                            v.y = turn_buf[turned(r, c + 1)];
                            v.z = turn_buf[turned(r, c + 2)];
                            v.w = turn_buf[turned(r, c + 3)];
                            if (p.accumulate) {
                                v.x += prev[i].x;
                                v.y += prev[i].y;
                                v.z += prev[i].z;
                                v.w += prev[i].w;
                            }
                            if (m0 + 4 * (i4 + i) < rows)
                                *reinterpret_cast<float4 *>(out + (int64_t)4 * (i4 + i) * p.N) = v;
                        }
                    }
                }
                __syncwarp();
            }
            if (MODE == kFwd && row < p.M) g.part[(int64_t)(2 * tn + half) * p.M + row] = kUnscale * part;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                  // the pair is done with both TMEMs
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     ::"r"(tmem), "r"(kTmemCols));
    }
}

// l_t from the tiles' sums, and the loss: each CTA sums its tokens in 64 bits,
// the last one to finish adds the CTAs' sums in their order.
constexpr int kLossThreads = 256;
__global__ void __launch_bounds__(kLossThreads)
balance_loss_kernel(const float *__restrict__ part, int nparts, int L, float *__restrict__ token_loss,
                    double *__restrict__ block_sum, BalHeader *hdr, double factor,
                    const int32_t *__restrict__ n_tokens, float *__restrict__ loss) {
    __shared__ double sm[kLossThreads / 32];
    __shared__ int last;
    grid_dependency_wait();
    grid_dependents_launch();
    double s = 0.0;
    const int64_t t = (int64_t)blockIdx.x * kLossThreads + threadIdx.x;
    if (t < L) {
        float v = 0.f;
#pragma unroll 8
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
        last = atomicAdd(&hdr->done, 1) == (int)gridDim.x - 1;
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
        const double n = *n_tokens, nl = hdr->kept;
        *loss = n > 0 && nl > 0 ? (float)(factor / (n * nl) * s) : 0.f;
    }
}

inline int pad64(int n) { return (n + 63) / 64 * 64; }

// Clocks of a K step of a tile bn columns wide: its 8 MMAs take 4 per column;
// its shared-memory traffic (operands read and filled) is 64 KB and 192 bytes
// per column at 128 bytes a clock, which is more for narrow tiles.
inline int step_clocks(int bn) {
    const int mma = 4 * bn, smem = 512 + bn * 3 / 2;
    return mma > smem ? mma : smem;
}

// Width of the tiles of a launch whose problems have n[i] columns and as many
// 256-row tiles: the one that takes the least time in whole rounds of the
// pairs.
int pick_width(const int *n, int probs, int mtiles, int pairs) {
    int best = 0;
    int64_t best_cost = 0;
    for (int bn = BN; bn >= 64; bn -= 32) {
        int64_t tiles = 0;
        for (int i = 0; i < probs; ++i) tiles += (int64_t)mtiles * ((n[i] + bn - 1) / bn);
        const int64_t cost = (tiles + pairs - 1) / pairs * step_clocks(bn);
        if (best == 0 || cost < best_cost) {
            best = bn;
            best_cost = cost;
        }
    }
    return best;
}

void set_tiles(GemmProb *p, int cols, int bn) {
    const int fifth = p->nk / 5;
    p->lead = fifth < kChunk ? kChunk : fifth > kMaxLead ? kMaxLead : fifth;
    p->bn = bn;
    p->tiles_n = (cols + bn - 1) / bn;
    p->tiles = ((p->M + 2 * BM - 1) / (2 * BM)) * p->tiles_n;
}

// Widths of dW's and dx's tiles, 128 or 256 (whole 64-element boxes in each
// CTA): 256, unless narrower ones of one of them or both still make one round
// of the pairs and a shorter one.
void set_grad_tiles(GemmProb *p, int d, int pairs) {
    int64_t best = 0;
    int width[2] = {256, 256};
    for (int k = 0; k < 4; ++k) {
        const int w[2] = {k & 1 ? 128 : 256, k & 2 ? 128 : 256};
        set_tiles(&p[0], d, w[0]);
        set_tiles(&p[1], d, w[1]);
        const int64_t a = (int64_t)p[0].nk * step_clocks(w[0]), b = (int64_t)p[1].nk * step_clocks(w[1]);
        const int64_t cost = a > b ? a : b;
        if (k == 0 || ((int64_t)p[0].tiles + p[1].tiles <= pairs && cost < best)) {
            best = cost;
            width[0] = w[0];
            width[1] = w[1];
        }
    }
    set_tiles(&p[0], d, width[0]);
    set_tiles(&p[1], d, width[1]);
}

template <int MODE>
cudaError_t launch_gemm(const GemmMaps &maps, GemmArgs &g, cudaStream_t st) {
    const int smem = (int)sizeof(GemmSmem) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(balance_gemm_kernel<MODE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int most = device_sm_count() / 2, pairs = g.tiles < most ? g.tiles : most;
    int bn = 0;
    for (int k = 0; k < g.nprob; ++k) bn = g.prob[k].bn > bn ? g.prob[k].bn : bn;
    g.accs = accumulators(bn);
    return launch(balance_gemm_kernel<MODE>, dim3((unsigned)(2 * pairs)), dim3(kThreads),
                  (size_t)smem, st, maps, g);
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

inline int fwd_width(int L, int N_r) {
    const int n[1] = {N_r};
    return pick_width(n, 1, (L + 2 * BM - 1) / (2 * BM), device_sm_count() / 2);
}

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
        w.x16 = take(2 * (size_t)L * d);
        w.w16 = take(2 * (size_t)w.ld * d);
    } else {
        const int bn = fwd_width(L, N_r);
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
                           dim3(256), 0, st, counts, N, n_tokens, status);
    if (e != cudaSuccess) return e;
    // crowded: as many tasks as experts or more, and enough of them for a CTA
    // on every SM (skewed layer, M = 2 N = 2^21: 17 against 61 us; with M = N =
    // 2^18, 10 against 3).  The sizes stand for what decides, how many tasks meet
    // on one expert, and are not always right.  In the table against one by one:
    // even tasks, M = N = 2^20, 9.2 against 7.0 us, and M = 2 N, 12.9 against
    // 11.6 (the table is taken); collapsed on 64 of 1304 x 1304 experts, 2^18
    // tasks 6.0 against 11.1, 2^20 tasks 6.1 against 41, and 2^19 even tasks on
    // 64 experts 7.3 against 133 (it is not).
    if (M >= N && M >= (int64_t)1 << 20)
        return launch(counts_crowded_kernel, dim3((unsigned)((M + kCrowdTasks - 1) / kCrowdTasks)),
                      dim3(kCrowdThreads), 0, st, idx, mask, (int)M, K, (int)N, counts, n_tokens, status);
    return launch(counts_kernel, dim3((unsigned)((M + 255) / 256)), dim3(256), 0, st, idx, mask,
                  (int)M, K, (int)N, counts, n_tokens, status);
}

namespace {
unsigned prep_grid(int64_t want) {
    const int64_t most = (int64_t)device_sm_count() * kPrepPerSm;
    return (unsigned)(want < most ? want : most);
}

cudaError_t launch_prep(BalPrep &p, void *ws, const BalanceWs &w, cudaStream_t st) {
    p.ld = w.ld;
    p.pr = pad64(p.N_r);
    p.pc = pad64(p.N_c);
    p.seg_r = w.ld - p.pc;
    p.P_hi = ws_at<uint16_t>(ws, w.P_hi);
    p.P_lo = ws_at<uint16_t>(ws, w.P_lo);
    p.F_hi = ws_at<uint16_t>(ws, w.F_hi);
    p.F_lo = ws_at<uint16_t>(ws, w.F_lo);
    p.hdr = ws_at<BalHeader>(ws, 0);
    const int64_t units =
        ((int64_t)p.L * ((p.ld + 255) / 256) + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
    const int64_t tiles = (int64_t)(p.pr / 64) * (p.pc / 64);
    return launch(balance_prep_kernel, dim3(prep_grid(units > tiles ? units : tiles)),
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
    p.M = L; p.N = N_r; p.nk = pp.pc / BK; p.a_hi = 0; p.a_lo = 1; p.b = 2; p.b_lo = 3; p.p = p_r;
    set_tiles(&p, N_r, fwd_width(L, N_r));
    g.nprob = 1; g.tiles = p.tiles; g.mask = mask; g.hdr = pp.hdr;
    g.part = ws_at<float>(ws, w.part);
    GemmMaps maps;
    if (!make_sw128_map(&maps.m[0], pp.P_hi, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[1], pp.P_lo, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[2], pp.F_hi, N_r, pp.pc, p.bn / 2) ||
        !make_sw128_map(&maps.m[3], pp.F_lo, N_r, pp.pc, p.bn / 2))
        return cudaErrorInvalidValue;
    if ((e = launch_gemm<kFwd>(maps, g, st)) != cudaSuccess) return e;
    return launch(balance_loss_kernel, dim3((unsigned)((L + kLossThreads - 1) / kLossThreads)),
                  dim3(kLossThreads), 0, st, (const float *)g.part, w.parts, L, token_loss,
                  ws_at<double>(ws, w.blocks), pp.hdr, (double)N_r * (double)N_c / (double)K,
                  n_tokens, loss);
}

cudaError_t launch_balance_bwd(const uint16_t *x, const uint16_t *W_r, const uint16_t *W_c,
                               const float *p_r, const float *p_c, const int32_t *counts,
                               const int32_t *n_tokens, const uint8_t *mask,
                               const float *token_loss, int L, int d, int N_r, int N_c, int K,
                               float dloss, float *dx, bool accumulate, float *dW_r, float *dW_c,
                               bool overwrite, void *ws, cudaStream_t st) {
    const BalanceWs w = balance_ws(L, d, N_r, N_c, true);
    BalPrep pp = {};
    pp.p_r = p_r; pp.p_c = p_c; pp.counts = counts; pp.mask = mask;
    pp.L = L; pp.N_r = N_r; pp.N_c = N_c; pp.d = d; pp.x = x; pp.W_r = W_r; pp.W_c = W_c;
    pp.token_loss = token_loss;
    pp.T_hi = ws_at<uint16_t>(ws, w.T_hi);
    pp.T_lo = ws_at<uint16_t>(ws, w.T_lo);
    cudaError_t e = launch_prep(pp, ws, w, st);
    if (e != cudaSuccess) return e;
    BalCast ca = {};
    ca.x = x; ca.W_r = W_r; ca.W_c = W_c; ca.mask = mask; ca.token_loss = token_loss;
    ca.L = L; ca.N_r = N_r; ca.N_c = N_c; ca.d = d; ca.pr = pp.pr; ca.ld = w.ld;
    ca.x16 = ws_at<uint16_t>(ws, w.x16);
    ca.w16 = ws_at<uint16_t>(ws, w.w16);
    ca.hdr = pp.hdr;
    const int64_t rows = (int64_t)L + w.ld;
    e = launch(balance_cast_kernel, dim3(prep_grid((rows + kPrepThreads / 32 - 1) / (kPrepThreads / 32))),
               dim3(kPrepThreads), 0, st, ca);
    if (e != cudaSuccess) return e;
    uint16_t *ds_hi = ws_at<uint16_t>(ws, w.ds_hi), *ds_lo = ws_at<uint16_t>(ws, w.ds_lo);
    const int mtiles = (L + 2 * BM - 1) / (2 * BM);

    GemmArgs g = {};
    g.mask = mask; g.token_loss = token_loss; g.hdr = pp.hdr; g.ld = w.ld;
    g.nprob = 2;
    // the pad columns belong to the tiles too: they must be written as zeros.
    // U's products run over the columns and V's over the rows
    const int segs[2] = {pp.pr, pp.pc};
    const int bn = pick_width(segs, 2, mtiles, device_sm_count() / 2);
    const int longer = segs[1] >= segs[0] ? 0 : 1;
    for (int k = 0; k < 2; ++k) {
        const int a = k ^ longer;                    // 0: U with ds_r, 1: V with ds_c
        GemmProb &p = g.prob[k];
        p.M = L; p.N = a == 0 ? N_r : N_c;
        p.nk = segs[1 - a] / BK;
        p.a_hi = 0; p.a_lo = 1; p.a_c0 = a == 0 ? pp.pr : 0;
        p.b = 2 + 2 * a; p.b_lo = 3 + 2 * a;
        p.P_hi = pp.P_hi + (a == 0 ? 0 : pp.pr);
        p.P_lo = pp.P_lo + (a == 0 ? 0 : pp.pr);
        p.seg = segs[a];
        p.ds_hi = ds_hi + (a == 0 ? 0 : pp.pr);
        p.ds_lo = ds_lo + (a == 0 ? 0 : pp.pr);
        set_tiles(&p, p.seg, bn);
        g.tiles += p.tiles;
    }
    GemmMaps maps;
    if (!make_sw128_map(&maps.m[0], pp.P_hi, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[1], pp.P_lo, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[2], pp.F_hi, N_r, pp.pc, bn / 2) ||
        !make_sw128_map(&maps.m[3], pp.F_lo, N_r, pp.pc, bn / 2) ||
        !make_sw128_map(&maps.m[4], pp.T_hi, N_c, pp.pr, bn / 2) ||
        !make_sw128_map(&maps.m[5], pp.T_lo, N_c, pp.pr, bn / 2))
        return cudaErrorInvalidValue;
    if ((e = launch_gemm<kGrid>(maps, g, st)) != cudaSuccess) return e;

    GemmArgs h = {};
    h.hdr = pp.hdr; h.n_tokens = n_tokens; h.token_loss = token_loss;
    h.factor = (double)dloss * N_r * N_c / K;
    h.nprob = 2;
    const int nk_dw = (L + BK - 1) / BK, nk_dx = w.ld / BK;
    GemmProb &dw = h.prob[nk_dw < nk_dx];            // A is ds^T, K the tokens
    dw.M = w.ld; dw.N = d; dw.nk = nk_dw; dw.a_mn = 1;
    dw.a_hi = 2; dw.a_lo = 3; dw.b = 4;
    dw.out = dW_r; dw.out2 = dW_c; dw.split = pp.pr; dw.rows1 = N_r; dw.rows2 = N_c;
    dw.accumulate = overwrite ? 0 : 1;
    GemmProb &px = h.prob[nk_dw >= nk_dx];
    px.M = L; px.N = d; px.nk = nk_dx;
    px.a_hi = 0; px.a_lo = 1; px.b = 5;
    px.out = dx; px.split = L; px.rows1 = L;
    px.accumulate = accumulate ? 1 : 0;
    set_grad_tiles(h.prob, d, device_sm_count() / 2);
    h.tiles = dw.tiles + px.tiles;
    if (!make_sw128_map(&maps.m[0], ds_hi, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[1], ds_lo, L, w.ld, BM) ||
        !make_sw128_map(&maps.m[2], ds_hi, L, w.ld, 64) ||
        !make_sw128_map(&maps.m[3], ds_lo, L, w.ld, 64) ||
        !make_sw128_map(&maps.m[4], ca.x16, L, d, 64) ||
        !make_sw128_map(&maps.m[5], ca.w16, w.ld, d, 64))
        return cudaErrorInvalidValue;
    return launch_gemm<kGrads>(maps, h, st);
}

}  // namespace omni
