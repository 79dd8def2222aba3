// norm.cu -- layer norm (forward and backward) and 8-bit activation
// checkpoints on sm_100a.
//
// Layer norm of a row x of d values, with weight w and optional bias b:
//   mean = sum(x) / d,  var = sum((x - mean)^2) / d,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b
// and its derivative, with g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw += sum_t dy xh,  db += sum_t dy
//
// A checkpoint holds a row in blocks of 32 values: e4m3 bytes q and one byte
// of scale, value = q 2^(scale - 127), the scale being the smallest power of
// two that lets no value of its block pass 448.  Scaling by a power of two is
// exact, so each value is rounded once (half a step of e4m3: at most 2^-4 of
// the value, or 2^-10 of the scale near zero).  Infinities and NaN are kept as
// NaN and do not take part in the block's scale.
//
// A row stays in registers between its one read and its one write: TPR
// threads share it, each holding VPT vectors of 8 values, so the variance is
// taken about the mean (no cancellation) and x is read once.  Everything is
// bound by HBM (or by launch latency below a few hundred rows).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "omni_common.cuh"
#include "omni_internal.h"

namespace omni {
namespace {

constexpr int kNormThreads = 128;

// ------------------------------------------------------------- 8 values
__device__ __forceinline__ void load8(const uint16_t *p, float *v) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float *v) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// ------------------------------------------------------------ checkpoints
// Scale byte of a block whose largest finite magnitude is amax = 1.m 2^(E - 127):
// 448 = 1.75 2^8, so s = E - 127 - 8, one more when 1.m > 1.75.
__device__ __forceinline__ int ckpt_code(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int code = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return code < 0 ? 0 : code;
}
__device__ __forceinline__ float ckpt_scale(int code) {     // 2^(code - 127)
    return __uint_as_float(code == 0 ? 0x00400000u : (uint32_t)code << 23);
}
__device__ __forceinline__ float finite_or_nan(float v) {
    return fabsf(v) <= 3.402823466e38f ? v : __uint_as_float(0x7fc00000u);
}
// Packs this thread's 8 values; four neighbouring lanes hold one block.
// Every lane of the warp takes part in the shuffles.
__device__ __forceinline__ uint2 ckpt_pack8(const float *v, int *code) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(finite_or_nan(v[i])));   // fmaxf drops NaN
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    *code = ckpt_code(amax);
    const float inv = __uint_as_float((uint32_t)(254 - *code) << 23);              // 2^(127 - code)
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(finite_or_nan(v[2 * i]) * inv,
                                                    finite_or_nan(v[2 * i + 1]) * inv),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ void ckpt_unpack8(uint2 q, int code, float *v) {
    const float s = ckpt_scale(code);
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

// ------------------------------------------------- sums over a row's threads
// TPR = 32: the row belongs to one warp; TPR = kNormThreads: to the CTA.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float *red) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = warp_sum(v[i]);
    if (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = (int)(threadIdx.x >> 5);
        __syncthreads();                                  // red is free again
        if (lane_id() == 0)
            for (int i = 0; i < NV; ++i) red[i * W + warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) v[i] += red[i * W + k];
        }
    }
}

// ---------------------------------------------------------------- forward
template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(kNormThreads)
norm_fwd_kernel(const T *__restrict__ x, const uint16_t *__restrict__ w,
                const uint16_t *__restrict__ b, int L, int d, float eps, uint16_t *__restrict__ y,
                float *__restrict__ mean_out, float *__restrict__ rstd_out,
                uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
    __shared__ float red[8];
    grid_dependency_wait();
    grid_dependents_launch();
    constexpr int RPC = kNormThreads / TPR;               // rows of a CTA
    const int tr = (int)threadIdx.x % TPR;
    const int nvec = d >> 3;
    const float inv_d = 1.f / (float)d;
    // the rows of a CTA take the same number of turns, so its barriers match
    for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < L; r0 += (int64_t)gridDim.x * RPC) {
        const int64_t row = r0 + (int)threadIdx.x / TPR;
        const bool live = row < L;
        float v[VPT][8];
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = tr + k * TPR;
            if (live && c < nvec) {
                load8(x + row * d + 8 * c, v[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] += v[k][i];
            }
        }
        row_sum<TPR, 1>(s, red);
        const float mean = s[0] * inv_d;
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (live && tr + k * TPR < nvec) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[k][i] -= mean;
                    s[0] = fmaf(v[k][i], v[k][i], s[0]);
                }
            }
        }
        row_sum<TPR, 1>(s, red);
        const float rstd = rsqrtf(fmaf(s[0], inv_d, eps));
        if (live && tr == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = tr + k * TPR;
            const bool on = live && c < nvec;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = on ? v[k][i] * rstd : 0.f;
            if (q) {
                int code;
                const uint2 p = ckpt_pack8(v[k], &code);
                if (on) {
                    *reinterpret_cast<uint2 *>(q + row * d + 8 * c) = p;
                    if ((c & 3) == 0) scale[row * (d >> 5) + (c >> 2)] = (uint8_t)code;
                }
            }
            if (on && y) {
                float wf[8], bf[8];
                load8(w + 8 * c, wf);
                if (b) load8(b + 8 * c, bf);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = b ? fmaf(v[k][i], wf[i], bf[i]) : v[k][i] * wf[i];
                store8(y + row * d + 8 * c, v[k]);
            }
        }
    }
}

// --------------------------------------------------------------- backward
// KEPT: 0 = x in T with mean, 1 = checkpoint.  Each CTA adds up dy xh and dy
// over its rows in registers and writes them to part[blockIdx.x * RPC + r][2][d]
// (r: the row slot in the CTA).
template <typename T, bool CKPT, int TPR, int VPT>
__global__ void __launch_bounds__(kNormThreads)
norm_bwd_kernel(const T *__restrict__ x, const float *__restrict__ mean_in,
                const float *__restrict__ rstd_in, const uint8_t *__restrict__ q,
                const uint8_t *__restrict__ scale, const uint16_t *__restrict__ w,
                const float *__restrict__ dy, int L, int d, float *__restrict__ dx,
                int accumulate, float *__restrict__ part) {
    __shared__ float red[2 * kNormThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    constexpr int RPC = kNormThreads / TPR;
    const int tr = (int)threadIdx.x % TPR;
    const int nvec = d >> 3;
    const float inv_d = 1.f / (float)d;
    float aw[VPT][8], ab[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) aw[k][i] = ab[k][i] = 0.f;
    for (int64_t r0 = (int64_t)blockIdx.x * RPC; r0 < L; r0 += (int64_t)gridDim.x * RPC) {
        const int64_t row = r0 + (int)threadIdx.x / TPR;
        const bool live = row < L;
        const float rstd = live ? rstd_in[row] : 0.f;
        const float mean = live && !CKPT ? mean_in[row] : 0.f;
        float h[VPT][8], g[VPT][8];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = tr + k * TPR;
            if (live && c < nvec) {
                if (CKPT) {
                    ckpt_unpack8(*reinterpret_cast<const uint2 *>(q + row * d + 8 * c),
                                 scale[row * (d >> 5) + (c >> 2)], h[k]);
                } else {
                    load8(x + row * d + 8 * c, h[k]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[k][i] = (h[k][i] - mean) * rstd;
                }
                load8(dy + row * d + 8 * c, g[k]);
                float wf[8];
                load8(w + 8 * c, wf);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    aw[k][i] = fmaf(g[k][i], h[k][i], aw[k][i]);
                    ab[k][i] += g[k][i];
                    g[k][i] *= wf[i];
                    s[0] += g[k][i];
                    s[1] = fmaf(g[k][i], h[k][i], s[1]);
                }
            }
        }
        row_sum<TPR, 2>(s, red);
        const float m0 = s[0] * inv_d, m1 = s[1] * inv_d;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = tr + k * TPR;
            if (live && c < nvec) {
                float *out = dx + row * d + 8 * c;
                float o[8];
                if (accumulate) load8(out, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // rounded on its own, so that an addition to dx is one addition
                    const float t = __fmul_rn(rstd, g[k][i] - m0 - h[k][i] * m1);
                    o[i] = accumulate ? o[i] + t : t;
                }
                store8(out, o);
            }
        }
    }
    float *pw = part + ((int64_t)blockIdx.x * RPC + (int)threadIdx.x / TPR) * 2 * d;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = tr + k * TPR;
        if (c < nvec) {
            store8(pw + 8 * c, aw[k]);
            store8(pw + d + 8 * c, ab[k]);
        }
    }
}

// dw += sum of part[i][0], db += sum of part[i][1], in the order of i: one
// column per thread of 32, eight slices of i per column.
__global__ void __launch_bounds__(256)
norm_bwd_sum_kernel(const float *__restrict__ part, int nparts, int d, float *__restrict__ dw,
                    float *__restrict__ db) {
    __shared__ float sm[8][32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int c = blockIdx.x * 32 + (int)(threadIdx.x & 31);
    const int slice = (int)(threadIdx.x >> 5);
    const int cols = db ? 2 * d : d;
    float s = 0.f;
    if (c < cols)
        for (int i = slice; i < nparts; i += 8) s += part[(int64_t)i * 2 * d + c];
    sm[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sm[k][threadIdx.x & 31];
        float *o = c < d ? dw + c : db + (c - d);
        *o += s;
    }
}

// ------------------------------------------------- packing and restoring
template <typename T>
__global__ void __launch_bounds__(256)
ckpt_pack_kernel(const T *__restrict__ x, int64_t nvec, uint8_t *__restrict__ q,
                 uint8_t *__restrict__ scale) {
    grid_dependency_wait();
    grid_dependents_launch();
    // whole warps take each turn (the shuffles need every lane)
    for (int64_t c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) & ~(int64_t)31; c0 < nvec;
         c0 += (int64_t)gridDim.x * blockDim.x) {
        const int64_t c = c0 + lane_id();
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (c < nvec) load8(x + 8 * c, v);
        int code;
        const uint2 p = ckpt_pack8(v, &code);
        if (c < nvec) {
            *reinterpret_cast<uint2 *>(q + 8 * c) = p;
            if ((c & 3) == 0) scale[c >> 2] = (uint8_t)code;
        }
    }
}

__global__ void __launch_bounds__(256)
ckpt_unpack_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale,
                   const uint16_t *__restrict__ w, const uint16_t *__restrict__ b, int64_t nvec,
                   int dvec, uint16_t *__restrict__ x) {
    grid_dependency_wait();
    grid_dependents_launch();
    for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < nvec;
         c += (int64_t)gridDim.x * blockDim.x) {
        float v[8];
        ckpt_unpack8(*reinterpret_cast<const uint2 *>(q + 8 * c), scale[c >> 2], v);
        if (w) {
            const int at = 8 * (int)(c % dvec);
            float wf[8], bf[8];
            load8(w + at, wf);
            if (b) load8(b + at, bf);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = b ? fmaf(v[i], wf[i], bf[i]) : v[i] * wf[i];
        }
        store8(x + 8 * c, v);
    }
}

unsigned blocks_for(int64_t units, int per_block, int per_sm) {
    const int64_t want = (units + per_block - 1) / per_block;
    const int64_t most = (int64_t)device_sm_count() * per_sm;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

// rows of partial sums that the backward writes for these sizes
int norm_bwd_parts(int L, int d) {
    const int rpc = d <= 1024 ? kNormThreads / 32 : 1;
    return (int)blocks_for(L, rpc, 4) * rpc;
}

namespace {

template <typename T>
cudaError_t norm_fwd_t(const T *x, const uint16_t *w, const uint16_t *b, int L, int d, float eps,
                       uint16_t *y, float *mean, float *rstd, uint8_t *q, uint8_t *scale,
                       cudaStream_t st) {
    const int rpc = d <= 1024 ? kNormThreads / 32 : 1;
    const dim3 grid(blocks_for(L, rpc, 8)), block(kNormThreads);
    const int vecs = d <= 1024 ? (d + 255) / 256 : (d + 1023) / 1024;
#define OMNI_NORM(tpr, n) \
    case n: return launch(norm_fwd_kernel<T, tpr, n>, grid, block, 0, st, x, w, b, L, d, eps, y, \
                          mean, rstd, q, scale);
    if (d <= 1024) {
        switch (vecs) { OMNI_NORM(32, 1) OMNI_NORM(32, 2) OMNI_NORM(32, 3) OMNI_NORM(32, 4) }
    } else {
        switch (vecs) {
            OMNI_NORM(kNormThreads, 2) OMNI_NORM(kNormThreads, 3) OMNI_NORM(kNormThreads, 4)
            OMNI_NORM(kNormThreads, 5) OMNI_NORM(kNormThreads, 6) OMNI_NORM(kNormThreads, 7)
            OMNI_NORM(kNormThreads, 8)
        }
    }
#undef OMNI_NORM
    return cudaErrorInvalidValue;
}

template <typename T, bool CKPT>
cudaError_t norm_bwd_t(const T *x, const float *mean, const float *rstd, const uint8_t *q,
                       const uint8_t *scale, const uint16_t *w, const float *dy, int L, int d,
                       float *dx, bool accumulate, float *part, cudaStream_t st) {
    const int rpc = d <= 1024 ? kNormThreads / 32 : 1;
    const dim3 grid((unsigned)(norm_bwd_parts(L, d) / rpc)), block(kNormThreads);
    const int vecs = d <= 1024 ? (d + 255) / 256 : (d + 1023) / 1024;
    const int acc = accumulate ? 1 : 0;
#define OMNI_NORM(tpr, n) \
    case n: return launch(norm_bwd_kernel<T, CKPT, tpr, n>, grid, block, 0, st, x, mean, rstd, q, \
                          scale, w, dy, L, d, dx, acc, part);
    if (d <= 1024) {
        switch (vecs) { OMNI_NORM(32, 1) OMNI_NORM(32, 2) OMNI_NORM(32, 3) OMNI_NORM(32, 4) }
    } else {
        switch (vecs) {
            OMNI_NORM(kNormThreads, 2) OMNI_NORM(kNormThreads, 3) OMNI_NORM(kNormThreads, 4)
            OMNI_NORM(kNormThreads, 5) OMNI_NORM(kNormThreads, 6) OMNI_NORM(kNormThreads, 7)
            OMNI_NORM(kNormThreads, 8)
        }
    }
#undef OMNI_NORM
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_fwd(const void *x, bool x_f32, const uint16_t *w, const uint16_t *b, int L,
                            int d, float eps, uint16_t *y, float *mean, float *rstd, uint8_t *q,
                            uint8_t *scale, cudaStream_t st) {
    if (x_f32)
        return norm_fwd_t(static_cast<const float *>(x), w, b, L, d, eps, y, mean, rstd, q, scale, st);
    return norm_fwd_t(static_cast<const uint16_t *>(x), w, b, L, d, eps, y, mean, rstd, q, scale, st);
}

cudaError_t launch_norm_bwd(const void *x, bool x_f32, const float *mean, const float *rstd,
                            const uint8_t *q, const uint8_t *scale, const uint16_t *w,
                            const float *dy, int L, int d, float *dx, bool accumulate, float *dw,
                            float *db, float *part, cudaStream_t st) {
    cudaError_t e;
    if (q)
        e = norm_bwd_t<uint16_t, true>(nullptr, mean, rstd, q, scale, w, dy, L, d, dx, accumulate,
                                       part, st);
    else if (x_f32)
        e = norm_bwd_t<float, false>(static_cast<const float *>(x), mean, rstd, q, scale, w, dy, L,
                                     d, dx, accumulate, part, st);
    else
        e = norm_bwd_t<uint16_t, false>(static_cast<const uint16_t *>(x), mean, rstd, q, scale, w,
                                        dy, L, d, dx, accumulate, part, st);
    if (e != cudaSuccess) return e;
    const int cols = db ? 2 * d : d;
    return launch(norm_bwd_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st,
                  (const float *)part, norm_bwd_parts(L, d), d, dw, db);
}

cudaError_t launch_ckpt_pack(const void *x, bool x_f32, int L, int d, uint8_t *q, uint8_t *scale,
                             cudaStream_t st) {
    const int64_t nvec = (int64_t)L * (d >> 3);
    const dim3 grid(blocks_for(nvec, 256, 8)), block(256);
    if (x_f32)
        return launch(ckpt_pack_kernel<float>, grid, block, 0, st, static_cast<const float *>(x),
                      nvec, q, scale);
    return launch(ckpt_pack_kernel<uint16_t>, grid, block, 0, st, static_cast<const uint16_t *>(x),
                  nvec, q, scale);
}

cudaError_t launch_ckpt_unpack(const uint8_t *q, const uint8_t *scale, const uint16_t *w,
                               const uint16_t *b, int L, int d, uint16_t *x, cudaStream_t st) {
    const int64_t nvec = (int64_t)L * (d >> 3);
    return launch(ckpt_unpack_kernel, dim3(blocks_for(nvec, 256, 8)), dim3(256), 0, st, q, scale, w,
                  b, nvec, d >> 3, x);
}

}  // namespace omni
