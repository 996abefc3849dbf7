// norm.cu -- the norms around the mixer: rsq_gated_norm and rsq_residual_norm
// with their gradients (sm_100a).
//
// A unit is one group of columns of one row.  Its threads keep the unit in
// registers between the reduction and the output, so that every input is read
// once and every output written once: the kernels are bound by HBM.  A block
// walks down the rows with its columns fixed (grid.y = group), loads the next
// row's vectors before it reduces the current one, and in the backward pass
// adds up the column sums (dw, dscale) of its rows in shared memory; a second
// kernel adds the blocks' partial sums in block order.
//
// With n = u r, r = 1/sqrt(mean(u^2) + eps) and dn the gradient of n:
//     du = r (dn - n mean(dn n)),   mean(dn n) = r mean(dn u)
// so the two sums of a backward row, u^2 and dn u, share one reduction.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rsq_internal.h"

namespace rsq {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxWidth = 16384;
// Blocks over all groups: four per SM.  More blocks mean more partial sums to
// add up in the backward pass, fewer leave HBM idle while a block reduces.
constexpr int kBlocks = 592;

enum Mode { kPlain = 0, kNormGate = 1, kGateNorm = 2, kResidual = 3 };

struct NormParams {
    long long rows;
    int width, group;
    int tpu, upb;                 // threads of a unit, rows a block takes at a time
    float eps;
    int y_f32;
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

// VEC consecutive elements of type T, as loaded.
template <class T, int VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
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
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const unsigned short*>(p)); }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
};
template <>
struct Raw<float, 1> {
    float v;
    __device__ __forceinline__ void load(const float* p) { v = __ldg(p); }
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
    r.load(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r.get(i);
}

// 1 / (1 + e^-z): e^-z = inf gives 0.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// Sums (a, b) over the unit's threads; every thread gets them.  Units of at
// most a warp use shuffles among their lanes; a larger unit is a whole block.
__device__ __forceinline__ float2 unit_sum(float2 s, int tpu, float2* sh) {
    for (int d = min(tpu, 32) / 2; d; d >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
    }
    if (tpu > 32) {
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
        __syncthreads();
        s = make_float2(0.f, 0.f);
        for (int i = 0; i < tpu / 32; ++i) {
            s.x += sh[i].x;
            s.y += sh[i].y;
        }
    }
    return s;
}

template <class TX, class TS, int VEC, int K>
struct RowRaw {
    Raw<TX, VEC> x[K];
    Raw<TS, VEC> s[K];
};

template <int MODE, class TX, class TS, int VEC, int K>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 sh[2][kMaxThreads / 32];
    const int sub = threadIdx.x / p.tpu, t = threadIdx.x - sub * p.tpu;
    const int g0 = blockIdx.y * p.group;
    const TX* x = static_cast<const TX*>(p.x);
    const TS* side = static_cast<const TS*>(p.side);
    const bool has_side = MODE == kNormGate || MODE == kGateNorm || (MODE == kResidual && side);
    const float inv_n = 1.f / static_cast<float>(p.group);

    // the group's vectors that do not change from row to row
    float w[K][VEC], sc[K][VEC];
    bool on[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (t + k * p.tpu) * VEC;
        on[k] = c < p.group;
        if (on[k]) load_cols<VEC>(p.w + g0 + c, w[k]);
        if constexpr (MODE == kResidual) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) sc[k][i] = 1.f;
            if (on[k] && p.scale) load_cols<VEC>(p.scale + g0 + c, sc[k]);
        }
    }
    auto fetch = [&](long long row, RowRaw<TX, TS, VEC, K>& r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (t + k * p.tpu) * VEC;
            r.x[k].zero();
            r.s[k].zero();
            if (on[k] && row < p.rows) {
                r.x[k].load(x + row * p.xs + g0 + c);
                if (has_side) r.s[k].load(side + row * p.ss + g0 + c);
            }
        }
    };
    const long long step = static_cast<long long>(gridDim.x) * p.upb;
    RowRaw<TX, TS, VEC, K> next;
    fetch(static_cast<long long>(blockIdx.x) * p.upb + sub, next);
    int buf = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * p.upb; r0 < p.rows; r0 += step, buf ^= 1) {
        const long long row = r0 + sub;
        const RowRaw<TX, TS, VEC, K> cur = next;
        fetch(row + step, next);
        float u[K][VEC];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float v = cur.x[k].get(i);
                if constexpr (MODE == kGateNorm) {
                    const float z = cur.s[k].get(i);
                    v *= z * sigmoid(z);
                }
                if constexpr (MODE == kResidual) {
                    v = fmaf(sc[k][i], v, cur.s[k].get(i));
                    // the norm is that of the residual stream as stored
                    if constexpr (sizeof(TS) == 2) v = __bfloat162float(__float2bfloat16_rn(v));
                    if (!on[k]) v = 0.f;
                }
                u[k][i] = v;
                sum = fmaf(v, v, sum);
            }
        }
        const float r = rsqrtf(fmaf(unit_sum(make_float2(sum, 0.f), p.tpu, sh[buf]).x, inv_n, p.eps));
        if (row < p.rows) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!on[k]) continue;
                const long long at = row * p.width + g0 + (t + k * p.tpu) * VEC;
                if constexpr (MODE == kResidual) store<VEC>(static_cast<TS*>(p.out2) + at, u[k]);
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    o[i] = u[k][i] * r * w[k][i];
                    if constexpr (MODE == kNormGate) {
                        const float z = cur.s[k].get(i);
                        o[i] *= z * sigmoid(z);
                    }
                }
                if (p.y_f32)
                    store<VEC>(static_cast<float*>(p.y) + at, o);
                else
                    store<VEC>(static_cast<__nv_bfloat16*>(p.y) + at, o);
            }
        }
    }
}

// Adds VEC values to a thread's own places of the shared column sums.  Sums of
// VEC = 8 lie as two float4 planes so that a warp's accesses do not conflict.
template <int VEC>
__device__ __forceinline__ void add_cols(float* acc, int slot, int slots, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        float4* a = reinterpret_cast<float4*>(acc);
        float4 lo = a[slot], hi = a[slots + slot];
        lo.x += v[0];
        lo.y += v[1];
        lo.z += v[2];
        lo.w += v[3];
        hi.x += v[4];
        hi.y += v[5];
        hi.z += v[6];
        hi.w += v[7];
        a[slot] = lo;
        a[slots + slot] = hi;
    } else {
        acc[slot] += v[0];
    }
}

template <int MODE, class TX, class TS, int VEC, int K>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ float4 acc4[];   // column sums of dw, then of dscale: [K][threads] chunks each
    __shared__ float2 sh[2][kMaxThreads / 32];
    float* acc = reinterpret_cast<float*>(acc4);
    const int slots = K * blockDim.x;
    float* acc_s = acc + slots * VEC;
    const int sub = threadIdx.x / p.tpu, t = threadIdx.x - sub * p.tpu;
    const int g0 = blockIdx.y * p.group;
    const TX* x = static_cast<const TX*>(p.x);
    const TS* side = static_cast<const TS*>(p.side);
    const TS* dh = static_cast<const TS*>(p.dh);
    const float inv_n = 1.f / static_cast<float>(p.group);
    const bool want_s = MODE == kResidual && p.part_s;
    const bool need_x = MODE != kResidual || want_s;

    for (int i = threadIdx.x; i < slots * VEC * (want_s ? 2 : 1); i += blockDim.x) acc[i] = 0.f;
    __syncthreads();

    struct Row {
        Raw<TX, VEC> x[K];
        Raw<TS, VEC> s[K];
        Raw<__nv_bfloat16, VEC> d[K];
        Raw<float, VEC> df[K];
        Raw<TS, VEC> dh[K];
    };
    auto fetch = [&](long long row, Row& r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (t + k * p.tpu) * VEC;
            r.x[k].zero();
            r.s[k].zero();
            r.d[k].zero();
            r.df[k].zero();
            r.dh[k].zero();
            if (c >= p.group || row >= p.rows) continue;
            const long long at = row * p.width + g0 + c;
            if (need_x) r.x[k].load(x + row * p.xs + g0 + c);
            if (MODE != kPlain) r.s[k].load(side + row * p.ss + g0 + c);
            if (p.y_f32)
                r.df[k].load(static_cast<const float*>(p.dy) + at);
            else
                r.d[k].load(static_cast<const __nv_bfloat16*>(p.dy) + at);
            if (MODE == kResidual && dh) r.dh[k].load(dh + at);
        }
    };
    const long long step = static_cast<long long>(gridDim.x) * p.upb;
    Row cur;
    int buf = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * p.upb; r0 < p.rows; r0 += step, buf ^= 1) {
        const long long row = r0 + sub;
        fetch(row, cur);
        // u: what is normed; dn: the gradient of n
        float u[K][VEC], dn[K][VEC];
        float su = 0.f, sd = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (t + k * p.tpu) * VEC;
            float w[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = 0.f;
            if (c < p.group) load_cols<VEC>(p.w + g0 + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float dy = p.y_f32 ? cur.df[k].get(i) : cur.d[k].get(i);
                float v = MODE == kResidual ? cur.s[k].get(i) : cur.x[k].get(i);
                float d = dy * w[i];
                if constexpr (MODE == kNormGate || MODE == kGateNorm) {
                    const float z = cur.s[k].get(i);
                    const float gate = z * sigmoid(z);
                    if constexpr (MODE == kGateNorm) v *= gate;
                    if constexpr (MODE == kNormGate) d *= gate;
                }
                u[k][i] = v;
                dn[k][i] = d;
                su = fmaf(v, v, su);
                sd = fmaf(d, v, sd);
            }
        }
        const float2 s = unit_sum(make_float2(su, sd), p.tpu, sh[buf]);
        const float r = rsqrtf(fmaf(s.x, inv_n, p.eps));
        const float m = s.y * r * inv_n;
        if (row >= p.rows) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (t + k * p.tpu) * VEC;
            if (c >= p.group) continue;
            const long long at = row * p.width + g0 + c;
            float dx[VEC], d2[VEC], dw[VEC], w[VEC];
            load_cols<VEC>((MODE == kResidual && p.scale ? p.scale : p.w) + g0 + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float dy = p.y_f32 ? cur.df[k].get(i) : cur.d[k].get(i);
                const float n = u[k][i] * r;
                const float du = r * fmaf(-n, m, dn[k][i]);
                dx[i] = du;
                d2[i] = 0.f;
                dw[i] = dy * n;
                if constexpr (MODE == kNormGate || MODE == kGateNorm) {
                    const float z = cur.s[k].get(i), sg = sigmoid(z), gate = z * sg;
                    const float slope = sg * fmaf(z, 1.f - sg, 1.f);
                    if constexpr (MODE == kGateNorm) {
                        dx[i] = du * gate;
                        d2[i] = du * cur.x[k].get(i) * slope;
                    } else {
                        d2[i] = dy * n * w[i] * slope;
                        dw[i] *= gate;
                    }
                }
                if constexpr (MODE == kResidual) {
                    d2[i] = du + cur.dh[k].get(i);
                    dx[i] = p.scale ? d2[i] * w[i] : d2[i];
                }
            }
            if (p.y) store<VEC>(static_cast<TX*>(p.y) + at, dx);
            if (MODE != kPlain && p.out2) store<VEC>(static_cast<TS*>(p.out2) + at, d2);
            const int slot = k * blockDim.x + threadIdx.x;
            if (p.part_w) add_cols<VEC>(acc, slot, slots, dw);
            if (want_s) {
                float ds[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) ds[i] = d2[i] * cur.x[k].get(i);
                add_cols<VEC>(acc_s, slot, slots, ds);
            }
        }
    }
    // this block's column sums: the sub-units' in order
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
        float* part = which ? p.part_s : p.part_w;
        if (!part || (which && !want_s)) continue;
        const float* a = which ? acc_s : acc;
        for (int c = threadIdx.x; c < p.group; c += blockDim.x) {
            const int chunk = c / VEC, e = c - chunk * VEC;
            const int k = chunk / p.tpu, tt = chunk - k * p.tpu;
            float sum = 0.f;
            for (int q = 0; q < p.upb; ++q) {
                const int slot = k * blockDim.x + q * p.tpu + tt;
                sum += VEC == 8 ? a[((e >> 2) * slots + slot) * 4 + (e & 3)] : a[slot];
            }
            part[static_cast<long long>(blockIdx.x) * p.width + g0 + c] = sum;
        }
    }
}

// dw[c] = sum over the blocks' partial sums, in block order within each of 8
// interleaved runs, the runs in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* part, int parts, int width, float* out) {
    __shared__ float sh[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;
    float s = 0.f;
    if (c < width)
        for (int i = q; i < parts; i += 8) s += part[static_cast<long long>(i) * width + c];
    sh[q][threadIdx.x & 31] = s;
    __syncthreads();
    if (q == 0 && c < width) {
        for (int i = 1; i < 8; ++i) s += sh[i][threadIdx.x];
        out[c] = s;
    }
}

struct Geometry {
    int vec, k, tpu, upb, gx;
};

// Vectors of eight elements where every row of every array starts on one
// (width, group and strides multiples of 8; the bases are 16-byte aligned),
// else single elements.  Two vectors per thread up to groups of 8192, so that
// a thread has two loads of each input in flight and a backward row stays in
// registers; four above.
Geometry geometry(const rsq_norm_config& c) {
    Geometry g;
    const bool wide = c.group % 8 == 0 && c.width % 8 == 0 && c.x_stride % 8 == 0 && c.side_stride % 8 == 0;
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
    g.gx = static_cast<int>(std::max<long long>(1, std::min<long long>(blocks, std::max(1, kBlocks / groups))));
    return g;
}

template <int MODE, class TX, class TS, int VEC, int K>
int launch_one(bool backward, const NormParams& p, const Geometry& g, cudaStream_t s) {
    const dim3 grid(g.gx, p.width / p.group), block(g.tpu * g.upb);
    if (!backward) {
        norm_kernel<MODE, TX, TS, VEC, K><<<grid, block, 0, s>>>(p);
    } else {
        const size_t smem = static_cast<size_t>(K) * block.x * VEC * sizeof(float) * (MODE == kResidual && p.part_s ? 2 : 1);
        auto* f = norm_backward_kernel<MODE, TX, TS, VEC, K>;
        if (smem > 40 * 1024) {
            const int err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (err) return err;
        }
        f<<<grid, block, smem, s>>>(p);
    }
    return cudaGetLastError();
}

template <int MODE, class TX, class TS>
int launch_vec(bool backward, const NormParams& p, const Geometry& g, cudaStream_t s) {
    if (g.vec == 8) return g.k == 2 ? launch_one<MODE, TX, TS, 8, 2>(backward, p, g, s) : launch_one<MODE, TX, TS, 8, 4>(backward, p, g, s);
    return g.k == 16 ? launch_one<MODE, TX, TS, 1, 16>(backward, p, g, s) : launch_one<MODE, TX, TS, 1, 32>(backward, p, g, s);
}

template <int MODE>
int launch_types(bool backward, const rsq_norm_config& c, const NormParams& p, const Geometry& g, cudaStream_t s) {
    if (c.x_dtype == RSQ_F32)
        return c.side_dtype == RSQ_F32 ? launch_vec<MODE, float, float>(backward, p, g, s)
                                       : launch_vec<MODE, float, __nv_bfloat16>(backward, p, g, s);
    return c.side_dtype == RSQ_F32 ? launch_vec<MODE, __nv_bfloat16, float>(backward, p, g, s)
                                   : launch_vec<MODE, __nv_bfloat16, __nv_bfloat16>(backward, p, g, s);
}

int launch(int mode, bool backward, const rsq_norm_config& c, const NormParams& p, const Geometry& g, cudaStream_t s) {
    switch (mode) {
        case kPlain: return c.x_dtype == RSQ_F32 ? launch_vec<kPlain, float, float>(backward, p, g, s)
                                                 : launch_vec<kPlain, __nv_bfloat16, float>(backward, p, g, s);
        case kNormGate: return launch_types<kNormGate>(backward, c, p, g, s);
        case kGateNorm: return launch_types<kGateNorm>(backward, c, p, g, s);
        default: return launch_types<kResidual>(backward, c, p, g, s);
    }
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

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
    p.y_f32 = c.y_dtype == RSQ_F32;
    p.xs = c.x_stride;
    p.ss = c.side_stride;
    return p;
}

size_t workspace_bytes_of(const rsq_norm_config& c) {
    return 2 * sizeof(float) * static_cast<size_t>(geometry(c).gx) * static_cast<size_t>((c.width + 3) / 4 * 4);
}

// Launches a backward pass and the sums of its partial column sums.
rsq_status run_backward(const char* who, int mode, const rsq_norm_config& c, NormParams p, float* dw, float* dscale,
                        void* workspace, size_t bytes, void* stream) {
    const Geometry g = geometry(c);
    auto s = static_cast<cudaStream_t>(stream);
    if (dw || dscale) {
        if (!workspace || misaligned(workspace)) return set_error(RSQ_E_INVAL, "%s: workspace null or not 16-byte aligned", who);
        if (bytes < workspace_bytes_of(c))
            return set_error(RSQ_E_INVAL, "%s: workspace of %zu bytes, %zu needed", who, bytes, workspace_bytes_of(c));
        p.part_w = dw ? static_cast<float*>(workspace) : nullptr;
        p.part_s = dscale ? static_cast<float*>(workspace) + static_cast<size_t>(g.gx) * ((c.width + 3) / 4 * 4) : nullptr;
    }
    int err = launch(mode, true, c, p, g, s);
    for (int i = 0; i < 2 && !err; ++i) {
        float* out = i ? dscale : dw;
        if (!out) continue;
        column_sum_kernel<<<(c.width + 31) / 32, 256, 0, s>>>(i ? p.part_s : p.part_w, g.gx, c.width, out);
        err = cudaGetLastError();
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
    const rsq_status st = check_config("gated_norm", cfg, false, &c);
    if (st) return st;
    if (!w || misaligned(w)) return set_error(RSQ_E_INVAL, "gated_norm: w null or not 16-byte aligned");
    if (c.rows == 0) return RSQ_OK;
    if (!x || !y) return set_error(RSQ_E_INVAL, "gated_norm: null x or y");
    for (const void* q : {x, z, static_cast<const void*>(y)})
        if (misaligned(q)) return set_error(RSQ_E_INVAL, "gated_norm: a buffer is not 16-byte aligned");
    const Geometry g = geometry(c);
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
    const rsq_status st = check_config("gated_norm_backward", cfg, false, &c);
    if (st) return st;
    if (!w || misaligned(w)) return set_error(RSQ_E_INVAL, "gated_norm_backward: w null or not 16-byte aligned");
    if (c.rows && (!x || !dy)) return set_error(RSQ_E_INVAL, "gated_norm_backward: null x or dy");
    if (dz && !z) return set_error(RSQ_E_INVAL, "gated_norm_backward: dz without z");
    for (const void* q : {x, z, dy, static_cast<const void*>(dx), static_cast<const void*>(dz), static_cast<const void*>(dw)})
        if (misaligned(q)) return set_error(RSQ_E_INVAL, "gated_norm_backward: a buffer is not 16-byte aligned");
    NormParams p = params(c, geometry(c));
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
    const rsq_status st = check_config("residual_norm", cfg, true, &c);
    if (st) return st;
    if (!w || misaligned(w) || misaligned(scale))
        return set_error(RSQ_E_INVAL, "residual_norm: w null, or w or scale not 16-byte aligned");
    if (c.rows == 0) return RSQ_OK;
    if (!x || !h || !y) return set_error(RSQ_E_INVAL, "residual_norm: null x, h or y");
    for (const void* q : {x, residual, static_cast<const void*>(h), static_cast<const void*>(y)})
        if (misaligned(q)) return set_error(RSQ_E_INVAL, "residual_norm: a buffer is not 16-byte aligned");
    if (residual == h && c.side_stride != c.width)
        return set_error(RSQ_E_INVAL, "residual_norm: h is packed: in place needs a packed residual");
    const Geometry g = geometry(c);
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
    const rsq_status st = check_config("residual_norm_backward", cfg, true, &c);
    if (st) return st;
    if (!w || misaligned(w) || misaligned(scale))
        return set_error(RSQ_E_INVAL, "residual_norm_backward: w null, or w or scale not 16-byte aligned");
    if (c.rows && (!h || !dy)) return set_error(RSQ_E_INVAL, "residual_norm_backward: null h or dy");
    if (c.rows && dscale && !x) return set_error(RSQ_E_INVAL, "residual_norm_backward: dscale needs x");
    for (const void* q : {x, h, dy, dh, static_cast<const void*>(dx), static_cast<const void*>(dresidual),
                          static_cast<const void*>(dscale), static_cast<const void*>(dw)})
        if (misaligned(q)) return set_error(RSQ_E_INVAL, "residual_norm_backward: a buffer is not 16-byte aligned");
    c.side_stride = c.width;  // h as the forward pass wrote it
    NormParams p = params(c, geometry(c));
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
