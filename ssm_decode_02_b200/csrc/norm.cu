// norm.cu -- the norms around the mixer: rsq_gated_norm and rsq_residual_norm
// with their gradients (sm_100a).
//
// A unit is one group of columns of one row.  Its threads keep the unit in
// registers between the reduction and the output, so that every input is read
// once and every output written once: the forward kernels are bound by HBM.  A
// block walks down the rows with its columns fixed (grid.y = group), a row at a time:
// load, reduce, write; the other blocks of the SM load meanwhile.  In the backward
// pass it adds up the column sums (dw, dscale) of its rows in shared memory; a
// second kernel adds the blocks' partial sums in block order.
//
// With n = u r, r = 1/sqrt(mean(u^2) + eps) and dn the gradient of n:
//     du = r (dn - n mean(dn n)),   mean(dn n) = r mean(dn u)
// so the two sums of a backward row, u^2 and dn u, share one reduction.
//
// Measured: gated norm of 16384 x 5120 bf16 84 to 91 us (5.5 to 6.0 TB/s, 84 to 91% of the
// measured copy rate), residual norm of as many bytes 89 us; gradients 96 us (8192 x 5120,
// 420 MB) and 79 us (8192 x 2560 with a binary32 stream, 378 MB), 67 and 73%, with 20 of
// an SM's 64 warps at 96 registers a thread.  The gated one issues in 64% of its slots, and
// its warps wait for global loads (2.2 of 7.7 cycles an instruction), their turn (1.5) and
// shared memory and the special functions (0.9); the residual one issues in 40%, with 4.1 of
// 12.2 cycles on global loads and 3.6 on the sums and weights in shared memory.
// Rows on their way to shared memory by cp.async (107 to 159 us), paired binary32
// arithmetic (135), one vector a thread (126 to 170) and fewer registers (spills) were
// slower.  A step's few rows are one launch: 3 us in a graph.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "rsq_internal.h"
#include "scan_launch.cuh"

namespace rsq {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kBackwardRegs = 96;
constexpr int kMaxWidth = 16384;
constexpr int kForwardBlocks = 2368;  // over all groups: every thread an SM can hold, and a few rows each

enum Mode { kPlain = 0, kNormGate = 1, kGateNorm = 2, kResidual = 3 };

struct NormParams {
    long long rows;
    int width, group;
    int tpu, upb;                 // threads of a unit, rows a block takes at a time
    float eps;
    long long xs, ss;             // row strides of x and of z / residual
    const void* x;
    const void* side;             // z | residual (forward) / h (backward)
    const float* w;
    const float* scale;
    const void* dy;
    const void* dh;
    void* y;                      // y | dx
    void* out2;                   // h | dz | dresidual
    float* part_w;                // [gridDim.x][width] partial dw, or null
    float* part_s;                // [gridDim.x][width] partial dscale, or null
};

// VEC consecutive elements of type T, as loaded.  load_fixed is for what nothing writes
// while the kernel runs (a read-only load); load for what the call may write in place.
template <class T, int VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void load_fixed(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : (i < 4 ? v.y : (i < 6 ? v.z : v.w));
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <>
struct Raw<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void load_fixed(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float get(int i) const {
        switch (i) {
            case 0: return a.x;
            case 1: return a.y;
            case 2: return a.z;
            case 3: return a.w;
            case 4: return b.x;
            case 5: return b.y;
            case 6: return b.z;
            default: return b.w;
        }
    }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    unsigned short v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const unsigned short*>(p); }
    __device__ __forceinline__ void load_fixed(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const unsigned short*>(p)); }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
};
template <>
struct Raw<float, 1> {
    float v;
    __device__ __forceinline__ void load(const float* p) { v = *p; }
    __device__ __forceinline__ void load_fixed(const float* p) { v = __ldg(p); }
    __device__ __forceinline__ void zero() { v = 0.f; }
    __device__ __forceinline__ float get(int) const { return v; }
};

template <int VEC>
__device__ __forceinline__ void store(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}
template <int VEC>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}

// VEC floats of a per-column vector.
template <int VEC>
__device__ __forceinline__ void load_cols(const float* p, float (&v)[VEC]) {
    Raw<float, VEC> r;
    r.load_fixed(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r.get(i);
}

// 1 / (1 + e^-z): e^-z = inf gives 0.  Flushing subnormals (.ftz) saves the scaling
// around both approximations and changes no result by more than 2^-126.
__device__ __forceinline__ float sigmoid(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// Sums (a, b) over the unit's threads; every thread gets them.  Units of at
// most a warp use shuffles among their lanes; a larger unit is a whole block.
__device__ __forceinline__ float2 unit_sum(float2 s, int tpu, float2* sh) {
    for (int d = min(tpu, 32) / 2; d; d >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
    }
    if (tpu > 32) {  // at most 16 warps: every half-warp adds up their sums
        const int lane = threadIdx.x & 31;
        if (lane == 0) sh[threadIdx.x >> 5] = s;
        __syncthreads();
        s = (lane & 15) < tpu / 32 ? sh[lane & 15] : make_float2(0.f, 0.f);
#pragma unroll
        for (int d = 8; d; d >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
        }
    }
    return s;
}

// A thread's part of one row of one array: K vectors, tpu vectors apart.
template <class T, int VEC, int K>
struct Part {
    Raw<T, VEC> v[K];

    // `mine`: the thread's first vector, the others `apart` elements from one another; zero
    // where not `on`.  `fixed`: no call may write the array in place
    __device__ __forceinline__ void fetch(const T* mine, int apart, const bool (&on)[K], bool row_on, bool fixed) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k].zero();
            if (on[k] && row_on) {
                if (fixed)
                    v[k].load_fixed(mine + k * apart);
                else
                    v[k].load(mine + k * apart);
            }
        }
    }
};

template <int MODE, class TX, class TS, class TY, int VEC, int K>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__(VEC * K <= 16 && VEC == 8 ? 48 : 128)
norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 sh[2][kMaxThreads / 32];
    const int sub = threadIdx.x / p.tpu, t = threadIdx.x - sub * p.tpu;
    const int col = blockIdx.y * p.group + t * VEC, apart = p.tpu * VEC;
    const float inv_n = 1.f / static_cast<float>(p.group);
    bool on[K];
#pragma unroll
    for (int k = 0; k < K; ++k) on[k] = (t + k * p.tpu) * VEC < p.group;
    const TX* x = static_cast<const TX*>(p.x);
    const TS* side = static_cast<const TS*>(p.side);
    int buf = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * p.upb; r0 < p.rows; r0 += static_cast<long long>(gridDim.x) * p.upb, buf ^= 1) {
        const long long row = r0 + sub;
        const bool row_on = row < p.rows;
        Part<TX, VEC, K> xs;
        Part<TS, VEC, K> ss;
        xs.fetch(x + row * p.xs + col, apart, on, row_on, true);
        if constexpr (MODE != kPlain) ss.fetch(side + row * p.ss + col, apart, on, row_on && side, MODE != kResidual);  // h over the residual
        float u[K][VEC];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float sc[VEC];
            if (MODE == kResidual && p.scale) {  // the same columns every row: from L1
#pragma unroll
                for (int i = 0; i < VEC; ++i) sc[i] = 0.f;
                if (on[k]) load_cols<VEC>(p.scale + col + k * apart, sc);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float v = xs.v[k].get(i);
                if constexpr (MODE == kGateNorm) {
                    const float z = ss.v[k].get(i);
                    v *= z * sigmoid(z);
                }
                if constexpr (MODE == kResidual) {
                    v = p.scale ? fmaf(sc[i], v, ss.v[k].get(i)) : v + ss.v[k].get(i);
                    // the norm is that of the residual stream as stored
                    if constexpr (sizeof(TS) == 2) v = __bfloat162float(__float2bfloat16_rn(v));
                }
                u[k][i] = v;
                sum = fmaf(v, v, sum);
            }
        }
        const float r = rsqrtf(fmaf(unit_sum(make_float2(sum, 0.f), p.tpu, sh[buf]).x, inv_n, p.eps));
        if (!row_on) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!on[k]) continue;
            const long long at = row * p.width + col + k * apart;
            if constexpr (MODE == kResidual) store<VEC>(static_cast<TS*>(p.out2) + at, u[k]);
            float o[VEC], w[VEC];
            load_cols<VEC>(p.w + col + k * apart, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                o[i] = u[k][i] * r * w[i];
                if constexpr (MODE == kNormGate) {
                    const float z = ss.v[k].get(i);
                    o[i] *= z * sigmoid(z);
                }
            }
            store<VEC>(static_cast<TY*>(p.y) + at, o);
        }
    }
}

// A thread's own K vectors of a block's shared array, as pieces of four floats (VEC
// = 8) that lie next to those of its neighbours.
template <int VEC>
struct Own {
    float* base;
    __device__ __forceinline__ float* at(int piece) const { return base + (piece * blockDim.x + threadIdx.x) * (VEC == 8 ? 4 : 1); }
    __device__ __forceinline__ void set(int k, const float (&v)[VEC]) const {
        if constexpr (VEC == 8) {
            *reinterpret_cast<float4*>(at(2 * k)) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(at(2 * k + 1)) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *at(k) = v[0];
        }
    }
    __device__ __forceinline__ void get(int k, float (&v)[VEC]) const {
        if constexpr (VEC == 8) {
            const float4 a = *reinterpret_cast<const float4*>(at(2 * k)), b = *reinterpret_cast<const float4*>(at(2 * k + 1));
            v[0] = a.x;
            v[1] = a.y;
            v[2] = a.z;
            v[3] = a.w;
            v[4] = b.x;
            v[5] = b.y;
            v[6] = b.z;
            v[7] = b.w;
        } else {
            v[0] = *at(k);
        }
    }
    __device__ __forceinline__ void add(int k, const float (&v)[VEC]) const {
        float o[VEC];
        get(k, o);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] += v[i];
        set(k, o);
    }
};

// Whether w and scale fit shared memory beside the column sums: up to 8192 columns.
template <int VEC, int K>
constexpr bool kKeepCols = VEC * K <= 16;

// Backward.  Between the loads of a row and its stores lie two passes over its
// elements and one reduction.  For room for more rows in that chain, registers hold
// the row as loaded and its sigmoids alone, and the second pass makes u and dn again;
// w, scale and the column sums lie in shared memory at places of the thread's own.
template <int MODE, class TX, class TS, class TY, int VEC, int K>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__(VEC * K <= 16 && VEC == 8 ? kBackwardRegs : 128)
norm_backward_kernel(const __grid_constant__ NormParams p) {
    let_next();
    constexpr bool GATED = MODE == kNormGate || MODE == kGateNorm;
    constexpr bool KEEP = kKeepCols<VEC, K>;
    extern __shared__ float4 own4[];  // sums of dw, of dscale (if wanted), w, scale: [K][threads] vectors each
    __shared__ float2 sh[2][kMaxThreads / 32];
    const int floats = K * VEC * blockDim.x;
    const Own<VEC> acc{reinterpret_cast<float*>(own4)}, acc_s{acc.base + floats}, ws{acc_s.base + (p.part_s ? floats : 0)},
        scales{ws.base + floats};
    const int sub = threadIdx.x / p.tpu, t = threadIdx.x - sub * p.tpu;
    const int g0 = blockIdx.y * p.group, col = g0 + t * VEC, apart = p.tpu * VEC;
    const float inv_n = 1.f / static_cast<float>(p.group);
    const bool want_s = MODE == kResidual && p.part_s;
    const TX* x = static_cast<const TX*>(p.x);
    const TS* side = static_cast<const TS*>(p.side);
    const TS* dh = static_cast<const TS*>(p.dh);
    bool on[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        on[k] = (t + k * p.tpu) * VEC < p.group;
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.f;
        acc.set(k, v);
        if (want_s) acc_s.set(k, v);
        if constexpr (KEEP) {
            if (on[k]) load_cols<VEC>(p.w + col + k * apart, v);
            ws.set(k, v);
            if (MODE == kResidual && p.scale) {
                if (on[k]) load_cols<VEC>(p.scale + col + k * apart, v);
                scales.set(k, v);
            }
        }
    }
    auto weights = [&](int k, float (&v)[VEC]) {
        if constexpr (KEEP) {
            ws.get(k, v);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = 0.f;
            if (on[k]) load_cols<VEC>(p.w + col + k * apart, v);
        }
    };
    int buf = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * p.upb; r0 < p.rows; r0 += static_cast<long long>(gridDim.x) * p.upb, buf ^= 1) {
        const long long row = r0 + sub, packed = row * p.width + col;
        const bool row_on = row < p.rows;
        Part<TX, VEC, K> xs;
        Part<TS, VEC, K> ss, hs;
        Part<TY, VEC, K> ys;
        ys.fetch(static_cast<const TY*>(p.dy) + packed, apart, on, row_on, true);
        if (MODE != kResidual || want_s) xs.fetch(x + row * p.xs + col, apart, on, row_on, true);
        if constexpr (MODE != kPlain) ss.fetch(side + row * p.ss + col, apart, on, row_on, true);
        if constexpr (MODE == kResidual) hs.fetch(dh + packed, apart, on, row_on && dh, false);  // dresidual over dh

        float sg[K][VEC], w[VEC] = {};
        // u: what is normed; dn: the gradient of n
        auto u_dn = [&](int k, int i, float& u, float& dn) {
            dn = ys.v[k].get(i) * w[i];
            if constexpr (MODE == kResidual)
                u = ss.v[k].get(i);
            else
                u = xs.v[k].get(i);
            if constexpr (MODE == kGateNorm) u *= ss.v[k].get(i) * sg[k][i];
            if constexpr (MODE == kNormGate) dn *= ss.v[k].get(i) * sg[k][i];
        };
        float su = 0.f, sd = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            weights(k, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if constexpr (GATED) sg[k][i] = sigmoid(ss.v[k].get(i));
                float u, dn;
                u_dn(k, i, u, dn);
                su = fmaf(u, u, su);
                sd = fmaf(dn, u, sd);
            }
        }
        const float2 s = unit_sum(make_float2(su, sd), p.tpu, sh[buf]);
        const float r = rsqrtf(fmaf(s.x, inv_n, p.eps));
        if (!row_on) continue;
        const float m = -s.y * r * r * inv_n;  // du = r dn + r m u
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float dx[VEC], d2[VEC], dw[VEC], sc[VEC];
            weights(k, w);
            if (MODE == kResidual && p.scale) {
                if constexpr (KEEP)
                    scales.get(k, sc);
                else if (on[k])
                    load_cols<VEC>(p.scale + col + k * apart, sc);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float u, dn;
                u_dn(k, i, u, dn);
                const float du = r * fmaf(u, m, dn);
                const float gn = ys.v[k].get(i) * u * r;
                dx[i] = du;
                d2[i] = 0.f;
                dw[i] = gn;
                if constexpr (GATED) {
                    const float z = ss.v[k].get(i), gate = z * sg[k][i];
                    const float slope = sg[k][i] * fmaf(z, 1.f - sg[k][i], 1.f);
                    if constexpr (MODE == kGateNorm) {
                        d2[i] = du * xs.v[k].get(i) * slope;
                        dx[i] = du * gate;
                    } else {
                        d2[i] = gn * w[i] * slope;
                        dw[i] = gn * gate;
                    }
                }
                if constexpr (MODE == kResidual) {
                    d2[i] = du + hs.v[k].get(i);
                    dx[i] = p.scale ? d2[i] * sc[i] : d2[i];
                }
            }
            if (!on[k]) continue;
            if (p.y) store<VEC>(static_cast<TX*>(p.y) + packed + k * apart, dx);
            if (MODE != kPlain && p.out2) store<VEC>(static_cast<TS*>(p.out2) + packed + k * apart, d2);
            if (p.part_w) acc.add(k, dw);
            if (want_s) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d2[i] *= xs.v[k].get(i);
                acc_s.add(k, d2);
            }
        }
    }
    // this block's column sums: the sub-units' in order
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
        float* part = which ? p.part_s : p.part_w;
        if (!part || (which && !want_s)) continue;
        const float* a = which ? acc_s.base : acc.base;
        for (int c = threadIdx.x; c < p.group; c += blockDim.x) {
            const int vec = c / VEC, e = c - vec * VEC;
            const int k = vec / p.tpu, tt = vec - k * p.tpu;
            float sum = 0.f;
            for (int q = 0; q < p.upb; ++q) {
                const int thread = q * p.tpu + tt;
                sum += VEC == 8 ? a[((2 * k + (e >> 2)) * blockDim.x + thread) * 4 + (e & 3)] : a[k * blockDim.x + thread];
            }
            part[static_cast<long long>(blockIdx.x) * p.width + g0 + c] = sum;
        }
    }
}

// out[c] = sum over the blocks' partial sums: 32 interleaved runs in block order,
// then the runs in order.  blockIdx.y: dw, dscale.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part_w, const float* part_s, int parts, int width,
                                                          float* out_w, float* out_s) {
    __shared__ float sh[32][33];
    wait_before();
    const float* part = blockIdx.y ? part_s : part_w;
    float* out = blockIdx.y ? out_s : out_w;
    if (!out) return;
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < width)
        for (int i = q; i < parts; i += 32) s += part[static_cast<long long>(i) * width + c];
    sh[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < width) {
        for (int i = 1; i < 32; ++i) s += sh[i][lane];
        out[c] = s;
    }
}

struct Geometry {
    int vec, k, tpu, upb, gx;
};

// Backward blocks of an SM: those that fit at once (registers), four at most.
int blocks_fit(const Geometry& g) { return std::max(1, std::min(4, 65536 / (kBackwardRegs * g.tpu * g.upb))); }

// Whether every row of every array starts on a vector of eight elements (the bases are then
// 16-byte aligned).
bool is_wide(const rsq_norm_config& c) {
    return c.group % 8 == 0 && c.width % 8 == 0 && c.x_stride % 8 == 0 && c.side_stride % 8 == 0;
}

// Vectors of eight elements where rows start on one, else single elements.  Two vectors per thread up to groups of 8192, four above:
// one would leave half the threads of a block of 512 without work at 5120 columns.
Geometry geometry(const rsq_norm_config& c, bool backward) {
    Geometry g;
    const bool wide = is_wide(c);
    g.vec = wide ? 8 : 1;
    const int chunks = c.group / g.vec;
    g.k = wide ? (c.group <= 8192 ? 2 : 4) : (c.group <= 8192 ? 16 : 32);
    const int need = (chunks + g.k - 1) / g.k;
    g.tpu = 1;
    if (need > 32)
        g.tpu = (need + 31) / 32 * 32;
    else
        while (g.tpu < need) g.tpu *= 2;
    g.upb = g.tpu <= 32 ? 128 / g.tpu : 1;
    const int groups = c.width / c.group;
    const long long blocks = (c.rows + g.upb - 1) / g.upb;
    // Backward: the blocks that fit at once, so that none waits with its whole share
    // of rows (4 per SM at most: every block leaves partial column sums behind).
    g.gx = static_cast<int>(std::max<long long>(1, std::min<long long>(blocks, std::max(1, (backward ? 148 * blocks_fit(g) : kForwardBlocks) / groups))));
    return g;
}

template <int MODE, class TX, class TS, class TY, int VEC, int K>
int launch_one(bool backward, const NormParams& p, const Geometry& g, cudaStream_t s) {
    const dim3 grid(g.gx, p.width / p.group), block(g.tpu * g.upb);
    if (!backward) {
        norm_kernel<MODE, TX, TS, TY, VEC, K><<<grid, block, 0, s>>>(p);
        return cudaGetLastError();
    }
    const size_t smem = static_cast<size_t>(K) * block.x * VEC * sizeof(float) *
                        (1 + (p.part_s != nullptr) + (kKeepCols<VEC, K> ? 1 + (MODE == kResidual && p.scale) : 0));
    auto* f = norm_backward_kernel<MODE, TX, TS, TY, VEC, K>;
    if (smem > 40 * 1024) {
        const int err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err) return err;
    }
    f<<<grid, block, smem, s>>>(p);
    return cudaGetLastError();
}

template <int MODE, class TX, class TS, class TY>
int launch_vec(bool backward, const NormParams& p, const Geometry& g, cudaStream_t s) {
    if (g.vec == 8)
        return g.k == 2 ? launch_one<MODE, TX, TS, TY, 8, 2>(backward, p, g, s) : launch_one<MODE, TX, TS, TY, 8, 4>(backward, p, g, s);
    return g.k == 16 ? launch_one<MODE, TX, TS, TY, 1, 16>(backward, p, g, s) : launch_one<MODE, TX, TS, TY, 1, 32>(backward, p, g, s);
}

template <int MODE, class TX, class TS>
int launch_y(bool backward, const rsq_norm_config& c, const NormParams& p, const Geometry& g, cudaStream_t s) {
    return c.y_dtype == RSQ_F32 ? launch_vec<MODE, TX, TS, float>(backward, p, g, s)
                                : launch_vec<MODE, TX, TS, __nv_bfloat16>(backward, p, g, s);
}

template <int MODE>
int launch_types(bool backward, const rsq_norm_config& c, const NormParams& p, const Geometry& g, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (c.x_dtype == RSQ_F32)
        return c.side_dtype == RSQ_F32 ? launch_y<MODE, float, float>(backward, c, p, g, s) : launch_y<MODE, float, B>(backward, c, p, g, s);
    return c.side_dtype == RSQ_F32 ? launch_y<MODE, B, float>(backward, c, p, g, s) : launch_y<MODE, B, B>(backward, c, p, g, s);
}

int launch(int mode, bool backward, const rsq_norm_config& c, const NormParams& p, const Geometry& g, cudaStream_t s) {
    switch (mode) {
        case kPlain: return c.x_dtype == RSQ_F32 ? launch_y<kPlain, float, float>(backward, c, p, g, s)
                                                 : launch_y<kPlain, __nv_bfloat16, float>(backward, c, p, g, s);
        case kNormGate: return launch_types<kNormGate>(backward, c, p, g, s);
        case kGateNorm: return launch_types<kGateNorm>(backward, c, p, g, s);
        default: return launch_types<kResidual>(backward, c, p, g, s);
    }
}

bool misaligned(const void* p, unsigned to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// What the arrays of a call have to be aligned to: whole vectors, or single elements.
unsigned aligned_to(const rsq_norm_config& c, int dtype) { return is_wide(c) ? 16 : (dtype == RSQ_F32 ? 4 : 2); }

struct Array {
    const void* p;
    int dtype;
};
rsq_status check_aligned(const char* who, const rsq_norm_config& c, std::initializer_list<Array> arrays) {
    for (const Array& a : arrays)
        if (misaligned(a.p, aligned_to(c, a.dtype)))
            return set_error(RSQ_E_INVAL, "%s: a buffer is not %u-byte aligned", who, aligned_to(c, a.dtype));
    return RSQ_OK;
}

// Checks a configuration and fills in its defaults.
rsq_status check_config(const char* who, const rsq_norm_config* cfg, bool residual, rsq_norm_config* out) {
    if (!cfg) return set_error(RSQ_E_INVAL, "%s: null config", who);
    rsq_norm_config c = *cfg;
    if (c.rows < 0 || c.rows > (1LL << 40)) return set_error(RSQ_E_INVAL, "%s: rows out of range", who);
    if (c.width < 1) return set_error(RSQ_E_INVAL, "%s: width must be positive", who);
    if (c.width > kMaxWidth) return set_error(RSQ_E_UNSUPPORTED, "%s: width is at most %d (got %d)", who, kMaxWidth, c.width);
    if (c.group == 0) c.group = c.width;
    if (c.group < 1 || c.width % c.group) return set_error(RSQ_E_INVAL, "%s: group must divide width", who);
    if (residual && c.group != c.width) return set_error(RSQ_E_INVAL, "%s: one group per row", who);
    for (int d : {c.x_dtype, c.side_dtype, c.y_dtype})
        if (d != RSQ_F32 && d != RSQ_BF16) return set_error(RSQ_E_INVAL, "%s: bad dtype %d", who, d);
    if (c.order != RSQ_NORM_GATE && c.order != RSQ_GATE_NORM) return set_error(RSQ_E_INVAL, "%s: bad order %d", who, c.order);
    if (!(c.eps > 0.f) || c.eps > 1e30f) return set_error(RSQ_E_INVAL, "%s: eps must be positive and finite", who);
    for (int64_t* s : {&c.x_stride, &c.side_stride}) {
        if (*s == 0) *s = c.width;
        if (*s < c.width || *s > (1LL << 40)) return set_error(RSQ_E_INVAL, "%s: a row stride below the width", who);
    }
    *out = c;
    return RSQ_OK;
}

NormParams params(const rsq_norm_config& c, const Geometry& g) {
    NormParams p{};
    p.rows = c.rows;
    p.width = c.width;
    p.group = c.group;
    p.tpu = g.tpu;
    p.upb = g.upb;
    p.eps = c.eps;
    p.xs = c.x_stride;
    p.ss = c.side_stride;
    return p;
}

size_t workspace_bytes_of(const rsq_norm_config& c) {
    return 2 * sizeof(float) * static_cast<size_t>(geometry(c, true).gx) * static_cast<size_t>((c.width + 3) / 4 * 4);
}

// Launches a backward pass and the sums of its partial column sums.
rsq_status run_backward(const char* who, int mode, const rsq_norm_config& c, NormParams p, float* dw, float* dscale,
                        void* workspace, size_t bytes, void* stream) {
    const Geometry g = geometry(c, true);
    auto s = static_cast<cudaStream_t>(stream);
    if (dw || dscale) {
        if (!workspace || misaligned(workspace)) return set_error(RSQ_E_INVAL, "%s: workspace null or not 16-byte aligned", who);
        if (bytes < workspace_bytes_of(c))
            return set_error(RSQ_E_INVAL, "%s: workspace of %zu bytes, %zu needed", who, bytes, workspace_bytes_of(c));
        p.part_w = dw ? static_cast<float*>(workspace) : nullptr;
        p.part_s = dscale ? static_cast<float*>(workspace) + static_cast<size_t>(g.gx) * ((c.width + 3) / 4 * 4) : nullptr;
    }
    int err = launch(mode, true, c, p, g, s);
    if (!err && (dw || dscale)) {
        err = rsq::launch(column_sum_kernel, dim3((c.width + 31) / 32, dscale ? 2 : 1), 1024, 0, s, false, p.part_w, p.part_s, g.gx, c.width,
                          dw, dscale);
    }
    return err ? set_error(RSQ_E_CUDA, "%s: %s", who, cudaGetErrorString(static_cast<cudaError_t>(err))) : RSQ_OK;
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" {

rsq_status rsq_norm_workspace(const rsq_norm_config* cfg, size_t* bytes) {
    rsq_norm_config c;
    if (!bytes) return set_error(RSQ_E_INVAL, "norm_workspace: null argument");
    const rsq_status st = check_config("norm_workspace", cfg, false, &c);
    if (st) return st;
    *bytes = workspace_bytes_of(c);
    return RSQ_OK;
}

rsq_status rsq_gated_norm(const rsq_norm_config* cfg, const void* x, const void* z, const float* w, void* y, void* stream) {
    rsq_norm_config c;
    rsq_status st = check_config("gated_norm", cfg, false, &c);
    if (st) return st;
    if (!w) return set_error(RSQ_E_INVAL, "gated_norm: null w");
    if ((st = check_aligned("gated_norm", c, {{x, c.x_dtype}, {z, c.side_dtype}, {w, RSQ_F32}, {y, c.y_dtype}}))) return st;
    if (c.rows == 0) return RSQ_OK;
    if (!x || !y) return set_error(RSQ_E_INVAL, "gated_norm: null x or y");
    const Geometry g = geometry(c, false);
    NormParams p = params(c, g);
    p.x = x;
    p.side = z;
    p.w = w;
    p.y = y;
    const int mode = !z ? kPlain : (c.order == RSQ_GATE_NORM ? kGateNorm : kNormGate);
    const int err = launch(mode, false, c, p, g, static_cast<cudaStream_t>(stream));
    return err ? set_error(RSQ_E_CUDA, "gated_norm: %s", cudaGetErrorString(static_cast<cudaError_t>(err))) : RSQ_OK;
}

rsq_status rsq_gated_norm_backward(const rsq_norm_config* cfg, const void* x, const void* z, const float* w,
                                   const void* dy, void* dx, void* dz, float* dw, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    rsq_norm_config c;
    rsq_status st = check_config("gated_norm_backward", cfg, false, &c);
    if (st) return st;
    if (!w) return set_error(RSQ_E_INVAL, "gated_norm_backward: null w");
    if (c.rows && (!x || !dy)) return set_error(RSQ_E_INVAL, "gated_norm_backward: null x or dy");
    if (dz && !z) return set_error(RSQ_E_INVAL, "gated_norm_backward: dz without z");
    if ((st = check_aligned("gated_norm_backward", c, {{x, c.x_dtype}, {z, c.side_dtype}, {w, RSQ_F32}, {dy, c.y_dtype}, {dx, c.x_dtype},
                                                       {dz, c.side_dtype}, {dw, RSQ_F32}})))
        return st;
    NormParams p = params(c, geometry(c, true));
    p.x = x;
    p.side = z;
    p.w = w;
    p.dy = dy;
    p.y = dx;
    p.out2 = dz;
    const int mode = !z ? kPlain : (c.order == RSQ_GATE_NORM ? kGateNorm : kNormGate);
    return run_backward("gated_norm_backward", mode, c, p, dw, nullptr, workspace, workspace_bytes, stream);
}

rsq_status rsq_residual_norm(const rsq_norm_config* cfg, const void* x, const void* residual, const float* scale,
                             const float* w, void* h, void* y, void* stream) {
    rsq_norm_config c;
    rsq_status st = check_config("residual_norm", cfg, true, &c);
    if (st) return st;
    if (!w) return set_error(RSQ_E_INVAL, "residual_norm: null w");
    if ((st = check_aligned("residual_norm", c, {{x, c.x_dtype}, {residual, c.side_dtype}, {scale, RSQ_F32}, {w, RSQ_F32},
                                                 {h, c.side_dtype}, {y, c.y_dtype}})))
        return st;
    if (c.rows == 0) return RSQ_OK;
    if (!x || !h || !y) return set_error(RSQ_E_INVAL, "residual_norm: null x, h or y");
    if (residual == h && c.side_stride != c.width)
        return set_error(RSQ_E_INVAL, "residual_norm: h is packed: in place needs a packed residual");
    const Geometry g = geometry(c, false);
    NormParams p = params(c, g);
    p.x = x;
    p.side = residual;
    p.scale = scale;
    p.w = w;
    p.out2 = h;
    p.y = y;
    const int err = launch(kResidual, false, c, p, g, static_cast<cudaStream_t>(stream));
    return err ? set_error(RSQ_E_CUDA, "residual_norm: %s", cudaGetErrorString(static_cast<cudaError_t>(err))) : RSQ_OK;
}

rsq_status rsq_residual_norm_backward(const rsq_norm_config* cfg, const void* x, const void* h, const float* scale,
                                      const float* w, const void* dy, const void* dh, void* dx, void* dresidual,
                                      float* dscale, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    rsq_norm_config c;
    rsq_status st = check_config("residual_norm_backward", cfg, true, &c);
    if (st) return st;
    c.side_stride = c.width;  // h as the forward pass wrote it
    if (!w) return set_error(RSQ_E_INVAL, "residual_norm_backward: null w");
    if (c.rows && (!h || !dy)) return set_error(RSQ_E_INVAL, "residual_norm_backward: null h or dy");
    if (c.rows && dscale && !x) return set_error(RSQ_E_INVAL, "residual_norm_backward: dscale needs x");
    if ((st = check_aligned("residual_norm_backward", c, {{x, c.x_dtype}, {h, c.side_dtype}, {scale, RSQ_F32}, {w, RSQ_F32}, {dy, c.y_dtype},
                                                          {dh, c.side_dtype}, {dx, c.x_dtype}, {dresidual, c.side_dtype},
                                                          {dscale, RSQ_F32}, {dw, RSQ_F32}})))
        return st;
    NormParams p = params(c, geometry(c, true));
    p.x = x;
    p.side = h;
    p.scale = scale;
    p.w = w;
    p.dy = dy;
    p.dh = dh;
    p.y = dx;
    p.out2 = dresidual;
    return run_backward("residual_norm_backward", kResidual, c, p, dw, dscale, workspace, workspace_bytes, stream);
}

}  // extern "C"
