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
// A row stays in registers between its one read and its one write: a group of
// G threads shares it, each holding VPT vectors of 8 values (one, up to d =
// 4096), so the variance is taken about the mean (no cancellation) and x is
// read once.  A CTA's groups take rows side by side, and each loads its next
// row before it reduces the present one.  Everything is bound by HBM (or by
// launch latency below a few hundred rows).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "omni_common.cuh"
#include "omni_internal.h"

namespace omni {
namespace {

// Threads of a CTA whose rows take groups of G, and CTAs of an SM for the
// forward and the backward (VPT vectors a thread): what their registers allow
// without spilling, which mattered more than the number of warps (backward at
// L = 16384, d = 2048 from a checkpoint: 84 us at 64 registers with 120 bytes
// spilled, 55 us at 79 with none).
__host__ __device__ constexpr int cta_threads(int G) { return G > 256 ? G : 256; }
__host__ __device__ constexpr int fwd_ctas(int G, int VPT) { return VPT > 1 ? 1 : G > 256 ? 2 : 4; }
__host__ __device__ constexpr int bwd_ctas(int G, int VPT) { return VPT > 1 || G > 256 ? 1 : 3; }

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
__device__ __forceinline__ float block_max(float m) {        // of four neighbouring lanes
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
// Packs this thread's 8 values; four neighbouring lanes hold one block.
// Every lane of the warp takes part in the shuffles.  NaN needs no care: fmaxf
// drops it and the conversion keeps it.  Infinities are looked for once a
// block (testing every value made the kernel issue-bound: 75 us at L = 65536,
// d = 2048, where 407 MB take 63).
__device__ __forceinline__ uint2 ckpt_pack8(const float *x, int *code) {
    float v[8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = x[i];
        amax = fmaxf(amax, fabsf(v[i]));
    }
    amax = block_max(amax);
    if (__any_sync(0xffffffffu, amax > 3.402823466e38f)) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = finite_or_nan(v[i]);
            amax = fmaxf(amax, fabsf(v[i]));
        }
        amax = block_max(amax);
    }
    *code = ckpt_code(amax);
    const float inv = __uint_as_float((uint32_t)(254 - *code) << 23);              // 2^(127 - code)
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv),
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
// Sums over a group; red: two sets of slots, used in turn, so that one barrier
// a sum is enough (a group cannot be two sums ahead of one of its warps).
template <int G, int NV>
struct GroupSum {
    static constexpr int W = G / 32;
    float *red;
    int turn;
    __device__ GroupSum(float *smem, int group) : red(smem + group * 2 * NV * W), turn(0) {}
    __device__ void operator()(float (&v)[NV], int group) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = warp_sum(v[i]);
        if (G > 32) {
            float *r = red + turn * NV * W;
            turn ^= 1;
            const int warp = (int)(threadIdx.x % G) >> 5;
            if (lane_id() == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) r[i * W + warp] = v[i];
            }
            // barriers 1 to 4: a CTA of 8 groups has warps for groups
            if (G == cta_threads(G)) __syncthreads();
            else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(G) : "memory");
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k) v[i] += r[i * W + k];
            }
        }
    }
};

// A thread's vectors of a row as they lie in memory.
template <typename T, int VPT>
struct RawRow;
template <int VPT>
struct RawRow<float, VPT> {
    float4 a[VPT], b[VPT];
    __device__ void load(const float *row, int c, int step, int nvec) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (c + k * step < nvec) {
                const float4 *p = reinterpret_cast<const float4 *>(row) + 2 * (c + k * step);
                a[k] = p[0];
                b[k] = p[1];
            }
    }
    __device__ void get(int k, float *v) const {
        v[0] = a[k].x; v[1] = a[k].y; v[2] = a[k].z; v[3] = a[k].w;
        v[4] = b[k].x; v[5] = b[k].y; v[6] = b[k].z; v[7] = b[k].w;
    }
};
template <int VPT>
struct RawRow<uint16_t, VPT> {
    uint4 u[VPT];
    __device__ void load(const uint16_t *row, int c, int step, int nvec) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (c + k * step < nvec) u[k] = reinterpret_cast<const uint4 *>(row)[c + k * step];
    }
    __device__ void get(int k, float *v) const {
        const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
// ... of a checkpoint: T is uint8_t, 8 bytes and their block's scale
template <int VPT>
struct RawRow<uint8_t, VPT> {
    uint2 q[VPT];
    uint8_t s[VPT];
    __device__ void load(const uint8_t *row, int c, int step, int nvec, const uint8_t *scale) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (c + k * step < nvec) {
                q[k] = reinterpret_cast<const uint2 *>(row)[c + k * step];
                s[k] = scale[(c + k * step) >> 2];
            }
    }
    __device__ void get(int k, float *v) const { ckpt_unpack8(q[k], s[k], v); }
};

// ---------------------------------------------------------------- forward
// (y may be x, row for row)
template <typename T, int G, int VPT, bool CKPT>
__global__ void __launch_bounds__(cta_threads(G), fwd_ctas(G, VPT))
norm_fwd_kernel(const T *x, const uint16_t *__restrict__ w,
                const uint16_t *__restrict__ b, int L, int d, float eps, uint16_t *y,
                float *__restrict__ mean_out, float *__restrict__ rstd_out,
                uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
    constexpr int GROUPS = cta_threads(G) / G;
    __shared__ float red[2 * cta_threads(G) / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int group = (int)threadIdx.x / G, c = (int)threadIdx.x % G;
    const int nvec = d >> 3;
    const float inv_d = 1.f / (float)d;
    GroupSum<G, 1> sum(red, group);
    RawRow<T, VPT> raw;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + group;
    if (row < L) raw.load(x + row * d, c, G, nvec);
    for (; row < L; row += step) {                       // the same for a whole group
        float v[VPT][8];
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (c + k * G < nvec) {
                raw.get(k, v[k]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] += v[k][i];
            }
        }
        if (row + step < L) raw.load(x + (row + step) * d, c, G, nvec);
        sum(s, group);
        const float mean = s[0] * inv_d;
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (c + k * G < nvec) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[k][i] -= mean;
                    s[0] = fmaf(v[k][i], v[k][i], s[0]);
                }
            }
        }
        sum(s, group);
        const float rstd = __frsqrt_rn(fmaf(s[0], inv_d, eps));
        if (c == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int cc = c + k * G;
            const bool on = cc < nvec;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = on ? v[k][i] * rstd : 0.f;
            if (CKPT) {
                int code;
                const uint2 p = ckpt_pack8(v[k], &code);
                if (on) {
                    *reinterpret_cast<uint2 *>(q + row * d + 8 * cc) = p;
                    if ((cc & 3) == 0) scale[row * (d >> 5) + (cc >> 2)] = (uint8_t)code;
                }
            }
            if (on) {
                float wf[8], bf[8];
                load8(w + 8 * cc, wf);
                if (b) load8(b + 8 * cc, bf);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = b ? fmaf(v[k][i], wf[i], bf[i]) : v[k][i] * wf[i];
                store8(y + row * d + 8 * cc, v[k]);
            }
        }
    }
}

// --------------------------------------------------------------- backward
// T: the kept rows' type, fp32 or bf16 with mean, or uint8_t for a checkpoint.
// A CTA adds up dy xh and dy over its rows in registers, then over its groups
// in shared memory, and writes them to part[blockIdx.x][2][d].  dx may be dy or x,
// row for row.
template <typename T, int G, int VPT>
__global__ void __launch_bounds__(cta_threads(G), bwd_ctas(G, VPT))
norm_bwd_kernel(const T *x, const uint8_t *__restrict__ scale,
                const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                const uint16_t *__restrict__ w, const float *dy, int L, int d, float *dx,
                int accumulate, float *__restrict__ part) {
    constexpr bool CKPT = sizeof(T) == 1;
    constexpr int GROUPS = cta_threads(G) / G;
    __shared__ float red[4 * cta_threads(G) / 32];
    // half of the groups' sums at most: GROUPS / 2 rows of 2 d <= 16 G floats
    __shared__ float4 half_sums[GROUPS > 1 ? cta_threads(G) * 2 : 1];
    grid_dependency_wait();
    grid_dependents_launch();
    const int group = (int)threadIdx.x / G, c = (int)threadIdx.x % G;
    const int nvec = d >> 3;
    const float inv_d = 1.f / (float)d;
    GroupSum<G, 2> sum(red, group);
    float aw[VPT][8], ab[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) aw[k][i] = ab[k][i] = 0.f;
    RawRow<T, VPT> raw;
    RawRow<float, VPT> raw_dy;
    float mean = 0.f, rstd = 0.f;
    const auto load = [&](int64_t r) {
        if constexpr (CKPT) raw.load(x + r * d, c, G, nvec, scale + r * (d >> 5));
        else raw.load(x + r * d, c, G, nvec);
        raw_dy.load(dy + r * d, c, G, nvec);
        rstd = rstd_in[r];
        if (!CKPT) mean = mean_in[r];
    };
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + group;
    if (row < L) load(row);
    for (; row < L; row += step) {                       // the same for a whole group
        float h[VPT][8], g[VPT][8];
        float s[2] = {0.f, 0.f};
        const float rs = rstd;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (c + k * G < nvec) {
                raw.get(k, h[k]);
                raw_dy.get(k, g[k]);
                float wf[8];
                load8(w + 8 * (c + k * G), wf);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!CKPT) h[k][i] = (h[k][i] - mean) * rs;
                    aw[k][i] = fmaf(g[k][i], h[k][i], aw[k][i]);
                    ab[k][i] += g[k][i];
                    g[k][i] *= wf[i];
                    s[0] += g[k][i];
                    s[1] = fmaf(g[k][i], h[k][i], s[1]);
                }
            }
        }
        if (row + step < L) load(row + step);
        sum(s, group);
        const float m0 = s[0] * inv_d, m1 = s[1] * inv_d;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (c + k * G < nvec) {
                float *out = dx + row * d + 8 * (c + k * G);
                float o[8];
                if (accumulate) load8(out, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // rounded on its own, so that an addition to dx is one addition
                    const float t = __fmul_rn(rs, g[k][i] - m0 - h[k][i] * m1);
                    o[i] = accumulate ? o[i] + t : t;
                }
                store8(out, o);
            }
        }
    }
    // groups h .. 2h - 1 hand their sums to groups 0 .. h - 1 (VPT is 1 where
    // there are several groups)
#pragma unroll
    for (int n = GROUPS / 2; n >= 1; n /= 2) {
        float *slot = reinterpret_cast<float *>(half_sums) + ((group % n) * G + c) * 16;
        __syncthreads();
        if (group >= n && group < 2 * n) {
            store8(slot, aw[0]);
            store8(slot + 8, ab[0]);
        }
        __syncthreads();
        if (group < n) {
            float t[16];
            load8(slot, t);
            load8(slot + 8, t + 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                aw[0][i] += t[i];
                ab[0][i] += t[8 + i];
            }
        }
    }
    if (group != 0) return;
    float *pw = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int cc = c + k * G;
        if (cc < nvec) {
            store8(pw + 8 * cc, aw[k]);
            store8(pw + d + 8 * cc, ab[k]);
        }
    }
}

// dw, db += (or =) the sums of part[i][0], part[i][1] in a fixed order: 32
// columns of a CTA, their rows in 32 slices.  Clears the workspace's status word:
// nothing here sets it.
constexpr int kSumSlices = 32;
__global__ void __launch_bounds__(32 * kSumSlices)
norm_bwd_sum_kernel(const float *__restrict__ part, int nparts, int d, float *__restrict__ dw,
                    float *__restrict__ db, int overwrite, int *status) {
    __shared__ float sm[kSumSlices][33];
    grid_dependency_wait();
    grid_dependents_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = OMNI_DEV_OK;
    const int lane = (int)(threadIdx.x & 31), slice = (int)(threadIdx.x >> 5);
    const int c = blockIdx.x * 32 + lane;
    const int cols = db ? 2 * d : d;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int i = slice; i < nparts; i += kSumSlices) s += part[(int64_t)i * 2 * d + c];
    }
    sm[slice][lane] = s;
    __syncthreads();
    // warp w adds up column w
    s = warp_sum(sm[lane][slice]);
    const int col = blockIdx.x * 32 + slice;
    if (lane == 0 && col < cols) {
        float *o = col < d ? dw + col : db + (col - d);
        *o = overwrite ? s : *o + s;
    }
}

// ------------------------------------------------- packing and restoring
// All CTAs of both grids are resident: 32 registers.
constexpr int kCkptThreads = 256, kCkptPerSm = 8;

template <typename T>
__global__ void __launch_bounds__(kCkptThreads, kCkptPerSm)
ckpt_pack_kernel(const T *__restrict__ x, int64_t nvec, uint8_t *__restrict__ q,
                 uint8_t *__restrict__ scale) {
    grid_dependency_wait();
    grid_dependents_launch();
    // whole warps take each turn (the shuffles need every lane)
    for (int64_t c0 = ((int64_t)blockIdx.x * kCkptThreads + threadIdx.x) & ~(int64_t)31; c0 < nvec;
         c0 += (int64_t)gridDim.x * kCkptThreads) {
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

__global__ void __launch_bounds__(kCkptThreads, kCkptPerSm)
ckpt_unpack_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale,
                   const uint16_t *__restrict__ w, const uint16_t *__restrict__ b, int64_t nvec,
                   int dvec, uint16_t *__restrict__ x) {
    grid_dependency_wait();
    grid_dependents_launch();
    for (int64_t c = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x; c < nvec;
         c += (int64_t)gridDim.x * kCkptThreads) {
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

// Threads that share a row: one vector of 8 each, a power of two of them (two
// vectors for d > 4096).
int group_threads(int d) {
    int g = 32;
    while (g < 512 && 8 * g < d) g *= 2;
    return g;
}
unsigned norm_blocks(int L, int d, bool backward) {
    const int g = group_threads(d), vpt = d > 4096 ? 2 : 1;
    return blocks_for(L, cta_threads(g) / g, backward ? bwd_ctas(g, vpt) : fwd_ctas(g, vpt));
}

}  // namespace

int norm_bwd_parts(int L, int d) { return (int)norm_blocks(L, d, true); }

namespace {

template <typename T, bool CKPT>
cudaError_t norm_fwd_t(const T *x, const uint16_t *w, const uint16_t *b, int L, int d, float eps,
                       uint16_t *y, float *mean, float *rstd, uint8_t *q, uint8_t *scale,
                       cudaStream_t st) {
    const int g = group_threads(d);
    const auto go = [&](auto kernel) {
        return launch(kernel, dim3(norm_blocks(L, d, false)), dim3(cta_threads(g)), 0, st, x, w, b, L,
                      d, eps, y, mean, rstd, q, scale);
    };
    if (d > 4096) return go(norm_fwd_kernel<T, 512, 2, CKPT>);
    switch (g) {
        case 32: return go(norm_fwd_kernel<T, 32, 1, CKPT>);
        case 64: return go(norm_fwd_kernel<T, 64, 1, CKPT>);
        case 128: return go(norm_fwd_kernel<T, 128, 1, CKPT>);
        case 256: return go(norm_fwd_kernel<T, 256, 1, CKPT>);
        default: return go(norm_fwd_kernel<T, 512, 1, CKPT>);
    }
}

template <typename T>
cudaError_t norm_bwd_t(const T *x, const uint8_t *scale, const float *mean, const float *rstd,
                       const uint16_t *w, const float *dy, int L, int d, float *dx, bool accumulate,
                       float *part, cudaStream_t st) {
    const int g = group_threads(d);
    const auto go = [&](auto kernel) {
        return launch(kernel, dim3(norm_blocks(L, d, true)), dim3(cta_threads(g)), 0, st, x, scale,
                      mean, rstd, w, dy, L, d, dx, accumulate ? 1 : 0, part);
    };
    if (d > 4096) return go(norm_bwd_kernel<T, 512, 2>);
    switch (g) {
        case 32: return go(norm_bwd_kernel<T, 32, 1>);
        case 64: return go(norm_bwd_kernel<T, 64, 1>);
        case 128: return go(norm_bwd_kernel<T, 128, 1>);
        case 256: return go(norm_bwd_kernel<T, 256, 1>);
        default: return go(norm_bwd_kernel<T, 512, 1>);
    }
}

}  // namespace

cudaError_t launch_norm_fwd(const void *x, bool x_f32, const uint16_t *w, const uint16_t *b, int L,
                            int d, float eps, uint16_t *y, float *mean, float *rstd, uint8_t *q,
                            uint8_t *scale, cudaStream_t st) {
    const auto go = [&](auto *xt) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(xt)>>;
        return q ? norm_fwd_t<T, true>(xt, w, b, L, d, eps, y, mean, rstd, q, scale, st)
                 : norm_fwd_t<T, false>(xt, w, b, L, d, eps, y, mean, rstd, q, scale, st);
    };
    return x_f32 ? go(static_cast<const float *>(x)) : go(static_cast<const uint16_t *>(x));
}

cudaError_t launch_norm_bwd(const void *x, bool x_f32, const float *mean, const float *rstd,
                            const uint8_t *q, const uint8_t *scale, const uint16_t *w,
                            const float *dy, int L, int d, float *dx, bool accumulate, float *dw,
                            float *db, bool overwrite, float *part, int *status, cudaStream_t st) {
    cudaError_t e;
    if (q)
        e = norm_bwd_t(q, scale, mean, rstd, w, dy, L, d, dx, accumulate, part, st);
    else if (x_f32)
        e = norm_bwd_t(static_cast<const float *>(x), scale, mean, rstd, w, dy, L, d, dx,
                       accumulate, part, st);
    else
        e = norm_bwd_t(static_cast<const uint16_t *>(x), scale, mean, rstd, w, dy, L, d, dx,
                       accumulate, part, st);
    if (e != cudaSuccess) return e;
    const int cols = db ? 2 * d : d;
    return launch(norm_bwd_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(32 * kSumSlices), 0,
                  st, (const float *)part, norm_bwd_parts(L, d), d, dw, db, overwrite ? 1 : 0,
                  status);
}

cudaError_t launch_ckpt_pack(const void *x, bool x_f32, int L, int d, uint8_t *q, uint8_t *scale,
                             cudaStream_t st) {
    const int64_t nvec = (int64_t)L * (d >> 3);
    const dim3 grid(blocks_for(nvec, kCkptThreads, kCkptPerSm)), block(kCkptThreads);
    if (x_f32)
        return launch(ckpt_pack_kernel<float>, grid, block, 0, st, static_cast<const float *>(x),
                      nvec, q, scale);
    return launch(ckpt_pack_kernel<uint16_t>, grid, block, 0, st, static_cast<const uint16_t *>(x),
                  nvec, q, scale);
}

cudaError_t launch_ckpt_unpack(const uint8_t *q, const uint8_t *scale, const uint16_t *w,
                               const uint16_t *b, int L, int d, uint16_t *x, cudaStream_t st) {
    const int64_t nvec = (int64_t)L * (d >> 3);
    return launch(ckpt_unpack_kernel, dim3(blocks_for(nvec, kCkptThreads, kCkptPerSm)),
                  dim3(kCkptThreads), 0, st, q, scale, w,
                  b, nvec, d >> 3, x);
}

}  // namespace omni
