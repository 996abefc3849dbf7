// scan_backward.cu -- the scan's backward pass (sm_100a).  The states before the
// chunks and the gradients of the states behind them come from states_kernel
// (scan_forward.cu); everything here is independent from chunk to chunk.
//
// With Z_ij = L_ij dt_j (C_i.B_j)(dout_i.x_j) for i >= j, and over the chunk
//     in_i  = 2^b_i C_i.(S_0 dout_i)                  what comes in with the state
//     fin_j = 2^(b_end-b_j) B_j.(dS x_j)              what leaves with it
//     m_t   = in_t + sum_{j<t} Z_tj - sum_{i>t} Z_it
// the gradients of the gates are
//     dlog a_t = sum_{t'>=t} m_t' + sum_{j<t} dt_j fin_j + 2^b_end <S_0, dS>
//     ddt_t    = sum_{i>=t} L_it (C_i.B_t)(dout_i.x_t) + fin_t + A dlog a_t
// where sum_{t'>=t} of the Z in m_t' is the sum of Z_ij over i >= t > j, made as such
// (head_gates, scan.cuh).  They are binary32 outputs: Z comes from products of the inputs alone, and the
// two state terms from states in three bf16 terms (split3).
#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

// Rows [r0, r0 + R) of a 64-column binary32 state as bf16: TERMS planes of R rows.
template <int R, int TERMS>
__device__ __forceinline__ void load_state(uint32_t dst, const float* src) {
    for (int i = threadIdx.x; i < R * 8; i += kThreads) {
        const int r = i >> 3, c = i & 7;
        const float4 a = *reinterpret_cast<const float4*>(src + r * kTile + c * 8);
        const float4 b = *(reinterpret_cast<const float4*>(src + r * kTile + c * 8) + 1);
        uint32_t t[3][4];
        split3(a.x, a.y, t[0][0], t[1][0], t[2][0]);
        split3(a.z, a.w, t[0][1], t[1][1], t[2][1]);
        split3(b.x, b.y, t[0][2], t[1][2], t[2][2]);
        split3(b.z, b.w, t[0][3], t[1][3], t[2][3]);
#pragma unroll
        for (int m = 0; m < TERMS; ++m)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + m * R * 128 + tile_at<2 * kTile>(r, c)),
                         "r"(t[m][0]), "r"(t[m][1]), "r"(t[m][2]), "r"(t[m][3])
                         : "memory");
    }
}

__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
// Bytes of row `row`, columns 8 c + 2 q, + 1 of a 64-column tile.
__device__ __forceinline__ uint32_t pair_at(int row, int c, int q) { return tile_at<2 * kTile>(row, c) + 4 * q; }

template <int N>
__device__ __forceinline__ void zero(float (&a)[N][4]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][e] = 0.f;
}

// A diagonal block of 16 x 16 (rows j, columns i > j; else zero): every column t gets,
// in the rows before it, the sum of its row from t on.
__device__ __forceinline__ void around_each(float (&z)[2][4], int g, int q) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float behind = 0.f;             // the columns of the block behind this one
#pragma unroll
        for (int nb = 1; nb >= 0; --nb) {
            float* v = z[nb] + 2 * r;
            const float t = v[0] + v[1], n1 = __shfl_xor_sync(0xffffffffu, t, 1);
            const float two = t + n1, n2 = __shfl_xor_sync(0xffffffffu, two, 2);
            const float rest = ((q & 1) ? 0.f : n1) + (q < 2 ? n2 : 0.f) + behind;
            const int c = nb * 8 + 2 * q, j = g + 8 * r;
            v[0] = c > j ? t + rest : 0.f;
            v[1] = c + 1 > j ? v[1] + rest : 0.f;
            behind += two + n2;
        }
    }
}

// ---------------------------------------------------------------------------
// dx and the gates: a block per (chunk, set of heads of one group).
// ---------------------------------------------------------------------------
template <int N>
struct DxShape {
    static constexpr int kK = kChunk * N * 2;
    static constexpr int kX = kChunk * kTile * 2;
    static constexpr int kRows = N < 128 ? N : 128;             // state rows staged at a time
    static constexpr int kPlanes = 3 * kRows * kTile * 2;
    static constexpr int kSmall = kChunk * (8 + 4) + 16 * kChunk * 4 + 4 * kChunk * 4 + 64;
    static constexpr int kSmem = 2 * kK + 2 * kX + kPlanes + kSmall;
};

template <int N>
__global__ void __launch_bounds__(kThreads, 1) dx_kernel(const __grid_constant__ Params p, int head_set) {
    using Sh = DxShape<N>;
    extern __shared__ __align__(128) uint8_t smem[];
    wait_before();
    const Rows rg = slot_rows(p, blockIdx.x);
    const int sets = (p.per + head_set - 1) / head_set;
    const int group = blockIdx.y / sets, set = blockIdx.y - group * sets;
    const int h0 = group * p.per + set * head_set;
    const int heads = min(head_set, p.per - set * head_set);
    if (!rg.valid) {
        // no rows: this slot adds nothing to the sums over tokens
        for (int i = threadIdx.x; i < heads; i += kThreads) {
            const long long at = static_cast<long long>(blockIdx.x) * p.H + h0 + i;
            p.part[at] = 0.f;
            p.part[static_cast<long long>(p.slots) * p.H + at] = 0.f;
        }
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint32_t sk = smem_u32(smem), sq = sk + Sh::kK, sx = sq + Sh::kK, sy = sx + Sh::kX, sp = sy + Sh::kX;
    float2* b = reinterpret_cast<float2*>(smem + 2 * Sh::kK + 2 * Sh::kX + Sh::kPlanes);
    float* dt = reinterpret_cast<float*>(b + kChunk);
    float* zrow = dt + kChunk;           // [8][kChunk] by the warps of j: sum_j Z_ij; in its own block the pairs around i
    float* zcol = zrow + 8 * kChunk;     // [8][kChunk] sum_{i>j} Z_ij / dt_j by the blocks of 16 i
    float* in_i = zcol + 8 * kChunk;     // 2^b_i C_i.(S_0 dout_i)
    float* own = in_i + kChunk;          // Z_jj / dt_j
    float* fin = own + kChunk;           // 2^(b_end-b_j) B_j.(dS x_j)
    float* row_d = fin + kChunk;         // x_i.dout_i
    float* ends = row_d + kChunk;          // [8] <S_0, dS> by warp
    const int valid = rg.valid;
    const int row0 = warp * 16;
    const bool live = row0 < valid;
    const long long os = static_cast<long long>(p.H) * p.P;

    load_tile<2 * N, kChunk>(sk, p.Bm + rg.first * p.bs + group * N, p.bs, valid, N / 8);
    load_tile<2 * N, kChunk>(sq, p.Cm + rg.first * p.cs + group * N, p.cs, valid, N / 8);
    cp_commit();
    cp_wait<0>();
    __syncthreads();

    // scores B_j.C_i: rows j of this warp, tokens i from its block on
    float sc[16][4];
    zero(sc);
    if (live) {
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) {
            uint32_t a[4];
            frag_a<2 * N>(a, sk, row0, ks, lane);
#pragma unroll
            for (int ib = 0; ib < 8; ++ib) {
                if (ib < warp) continue;
                uint32_t v[4];
                frag_b<2 * N>(v, sq, ib * 16, ks, lane);
                mma(sc[2 * ib], a, v[0], v[1]);
                mma(sc[2 * ib + 1], a, v[2], v[3]);
            }
        }
    }

    for (int hi = 0; hi < heads; ++hi) {
        const int h = h0 + hi;
        const long long gate_at = (static_cast<long long>(blockIdx.x) * p.H + h) * kChunk;
        __syncthreads();  // the head before is done with the shared arrays
        if (threadIdx.x < kChunk) {
            b[threadIdx.x] = p.gb[gate_at + threadIdx.x];
            dt[threadIdx.x] = p.gdt[gate_at + threadIdx.x];
        }
        for (int i = threadIdx.x; i < 16 * kChunk; i += kThreads) zrow[i] = 0.f;  // and zcol
        float in0 = 0.f, in8 = 0.f, own0 = 0.f, own8 = 0.f, fin0 = 0.f, fin8 = 0.f, d0 = 0.f, d8 = 0.f, through = 0.f;
        const float dh = p.D ? __ldg(p.D + h) : 0.f;

        for (int tile = 0; tile < p.tiles; ++tile) {
            const int cols = min(kTile, p.P - tile * kTile);
            const long long cell = ((static_cast<long long>(blockIdx.x) * p.H + h) * p.tiles + tile) * N * kTile;
            __syncthreads();
            load_tile<2 * kTile, kChunk>(sx, p.x + rg.first * p.xs + static_cast<long long>(h) * p.P + tile * kTile, p.xs, valid, cols / 8);
            load_tile<2 * kTile, kChunk>(sy, p.dout + rg.first * os + static_cast<long long>(h) * p.P + tile * kTile, os, valid, cols / 8);
            cp_commit();
            float acc[8][4], st[8][4];
            zero(st);
            // B_j dS
#pragma unroll
            for (int part = 0; part < N / Sh::kRows; ++part) {
                if (part) __syncthreads();
                load_state<Sh::kRows, 3>(sp, p.df + cell + part * Sh::kRows * kTile);
                cp_wait<0>();
                __syncthreads();
                if (live) {
#pragma unroll
                    for (int ks = 0; ks < Sh::kRows / 16; ++ks) {
                        uint32_t a[4];
                        frag_a<2 * N>(a, sk, row0, part * (Sh::kRows / 16) + ks, lane);
#pragma unroll
                        for (int m = 2; m >= 0; --m)
#pragma unroll
                            for (int c2 = 0; c2 < 4; ++c2) {
                                uint32_t v[4];
                                frag_bt<2 * kTile>(v, sp + m * Sh::kRows * 128, c2 * 16, ks, lane);
                                mma(st[2 * c2], a, v[0], v[1]);
                                mma(st[2 * c2 + 1], a, v[2], v[3]);
                            }
                    }
                }
            }
            const float2 b0 = b[row0 + g], b8 = b[row0 + g + 8], be = b[kChunk - 1];
            if (live) {
                const float w0 = ex2_diff(be, b0), w8 = ex2_diff(be, b8);
                float f0 = 0.f, f8 = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t x0 = lds32(sx + pair_at(row0 + g, i, q)), x8 = lds32(sx + pair_at(row0 + g + 8, i, q));
                    const uint32_t y0 = lds32(sy + pair_at(row0 + g, i, q)), y8 = lds32(sy + pair_at(row0 + g + 8, i, q));
                    acc[i][0] = st[i][0] * w0;
                    acc[i][1] = st[i][1] * w0;
                    acc[i][2] = st[i][2] * w8;
                    acc[i][3] = st[i][3] * w8;
                    f0 = fmaf(acc[i][0], lo_of(x0), fmaf(acc[i][1], hi_of(x0), f0));
                    f8 = fmaf(acc[i][2], lo_of(x8), fmaf(acc[i][3], hi_of(x8), f8));
                    d0 = fmaf(lo_of(y0), lo_of(x0), fmaf(hi_of(y0), hi_of(x0), d0));
                    d8 = fmaf(lo_of(y8), lo_of(x8), fmaf(hi_of(y8), hi_of(x8), d8));
                }
                fin0 += f0;
                fin8 += f8;
                // the chunk's own tokens
                uint32_t xa[4][4];
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) frag_a<2 * kTile>(xa[ks], sx, row0, ks, lane);
#pragma unroll
                for (int ib = 0; ib < 8; ++ib) {
                    if (ib < warp || ib * 16 >= valid) continue;
                    float zz[2][4];
                    zero(zz);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        uint32_t v[4];
                        frag_b<2 * kTile>(v, sy, ib * 16, ks, lane);
                        mma(zz[0], xa[ks], v[0], v[1]);
                        mma(zz[1], xa[ks], v[2], v[3]);
                    }
                    uint32_t a[4];
                    float dir0 = 0.f, dir8 = 0.f;
                    const float dt0 = dt[row0 + g], dt8 = dt[row0 + g + 8];
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        const int ci = ib * 16 + nb * 8 + 2 * q;
                        float pr[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = ci + (e & 1), j = row0 + g + (e >> 1) * 8;
                            pr[e] = i >= j ? sc[2 * ib + nb][e] * ex2_diff(b[i], (e >> 1) ? b8 : b0) : 0.f;
                            zz[nb][e] *= pr[e];
                        }
                        if (ib == warp) {  // the diagonal apart
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (ci + (e & 1) == row0 + g + (e >> 1) * 8) {
                                    ((e >> 1) ? own8 : own0) += zz[nb][e];
                                    zz[nb][e] = 0.f;
                                }
                        }
                        dir0 += zz[nb][0] + zz[nb][1];
                        dir8 += zz[nb][2] + zz[nb][3];
                        a[2 * nb] = pack(pr[0], pr[1]);
                        a[2 * nb + 1] = pack(pr[2], pr[3]);
                    }
                    if (ib == warp) around_each(zz, g, q);
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        const int ci = ib * 16 + nb * 8 + 2 * q;
                        float col[2] = {fmaf(dt0, zz[nb][0], dt8 * zz[nb][2]), fmaf(dt0, zz[nb][1], dt8 * zz[nb][3])};
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            col[0] += __shfl_xor_sync(0xffffffffu, col[0], d);
                            col[1] += __shfl_xor_sync(0xffffffffu, col[1], d);
                        }
                        if (g == 0) {
                            zrow[warp * kChunk + ci] += col[0];
                            zrow[warp * kChunk + ci + 1] += col[1];
                        }
                    }
                    dir0 = quad_sum(dir0);
                    dir8 = quad_sum(dir8);
                    if (q == 0) {
                        zcol[ib * kChunk + row0 + g] += dir0;
                        zcol[ib * kChunk + row0 + g + 8] += dir8;
                    }
#pragma unroll
                    for (int c2 = 0; c2 < 4; ++c2) {
                        uint32_t v[4];
                        frag_bt<2 * kTile>(v, sy, c2 * 16, ib, lane);
                        mma(acc[2 * c2], a, v[0], v[1]);
                        mma(acc[2 * c2 + 1], a, v[2], v[3]);
                    }
                }
                const float dt0 = dt[row0 + g], dt8 = dt[row0 + g + 8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t y0 = lds32(sy + pair_at(row0 + g, i, q)), y8 = lds32(sy + pair_at(row0 + g + 8, i, q));
                    acc[i][0] = fmaf(dt0, acc[i][0], dh * lo_of(y0));
                    acc[i][1] = fmaf(dt0, acc[i][1], dh * hi_of(y0));
                    acc[i][2] = fmaf(dt8, acc[i][2], dh * lo_of(y8));
                    acc[i][3] = fmaf(dt8, acc[i][3], dh * hi_of(y8));
                }
                if (p.dx)
                    store_rows(p.dx + static_cast<long long>(rg.first) * os + static_cast<long long>(h) * p.P + tile * kTile,
                               os, row0, valid, cols, acc, lane);
            }
            // C_i S_0, and <S_0, dS>
            zero(st);
#pragma unroll
            for (int part = 0; part < N / Sh::kRows; ++part) {
                __syncthreads();
                const float* s0 = p.sf + cell + part * Sh::kRows * kTile;
                const float* ds = p.df + cell + part * Sh::kRows * kTile;
                load_state<Sh::kRows, 3>(sp, s0);
                for (int i = threadIdx.x; i < Sh::kRows * kTile / 4; i += kThreads) {
                    const float4 u = reinterpret_cast<const float4*>(s0)[i], v = reinterpret_cast<const float4*>(ds)[i];
                    through = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, through))));
                }
                __syncthreads();
                if (live) {
#pragma unroll
                    for (int ks = 0; ks < Sh::kRows / 16; ++ks) {
                        uint32_t a[4];
                        frag_a<2 * N>(a, sq, row0, part * (Sh::kRows / 16) + ks, lane);
#pragma unroll
                        for (int m = 2; m >= 0; --m)
#pragma unroll
                            for (int c2 = 0; c2 < 4; ++c2) {
                                uint32_t v[4];
                                frag_bt<2 * kTile>(v, sp + m * Sh::kRows * 128, c2 * 16, ks, lane);
                                mma(st[2 * c2], a, v[0], v[1]);
                                mma(st[2 * c2 + 1], a, v[2], v[3]);
                            }
                    }
                }
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t y0 = lds32(sy + pair_at(row0 + g, i, q)), y8 = lds32(sy + pair_at(row0 + g + 8, i, q));
                    in0 = fmaf(st[i][0], lo_of(y0), fmaf(st[i][1], hi_of(y0), in0));
                    in8 = fmaf(st[i][2], lo_of(y8), fmaf(st[i][3], hi_of(y8), in8));
                }
            }
        }

        // row sums to shared memory, then the gates by the first warp
        in0 = quad_sum(in0);
        in8 = quad_sum(in8);
        own0 = quad_sum(own0);
        own8 = quad_sum(own8);
        fin0 = quad_sum(fin0);
        fin8 = quad_sum(fin8);
        d0 = quad_sum(d0);
        d8 = quad_sum(d8);
#pragma unroll
        for (int d = 16; d; d >>= 1) through += __shfl_xor_sync(0xffffffffu, through, d);
        if (q == 0) {
            const float2 b0 = b[row0 + g], b8 = b[row0 + g + 8];
            in_i[row0 + g] = in0 * ex2(b0.x + b0.y);
            in_i[row0 + g + 8] = in8 * ex2(b8.x + b8.y);
            own[row0 + g] = own0;
            own[row0 + g + 8] = own8;
            fin[row0 + g] = fin0;
            fin[row0 + g + 8] = fin8;
            row_d[row0 + g] = d0;
            row_d[row0 + g + 8] = d8;
        }
        if (lane == 0) ends[warp] = through;
        __syncthreads();
        if (warp == 0) {
            HeadSums hs{zrow, zcol, own, in_i, fin, row_d, 0.f};
#pragma unroll
            for (int w = 0; w < 8; ++w) hs.through += ends[w];
            const float2 be = b[kChunk - 1];
            hs.through *= ex2(be.x + be.y);
            const float ah = p.decay ? 0.f : __ldg(p.A + h);
            const float dt4[4] = {dt[lane * 4], dt[lane * 4 + 1], dt[lane * 4 + 2], dt[lane * 4 + 3]};
            float dl[4], dir[4], dd, da = 0.f;
            head_gates<8>(hs, dt4, valid, lane, dl, dir, dd);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = lane * 4 + k;
                if (t >= valid) continue;
                const long long at = static_cast<long long>(rg.first + t) * p.H + h;
                if (p.decay && __ldg(p.decay + at) == 0.f) dl[k] = 0.f;  // nothing passes, not 0 times a non-finite value either
                if (p.dlog) p.dlog[at] = dl[k];
                if (p.ddt) p.ddt[at] = p.decay ? dir[k] : fmaf(ah, dl[k], dir[k]);
                da = fmaf(dt4[k], dl[k], da);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) da += __shfl_xor_sync(0xffffffffu, da, d);
            if (lane == 0) {
                const long long at = static_cast<long long>(blockIdx.x) * p.H + h;
                p.part[at] = da;
                p.part[static_cast<long long>(p.slots) * p.H + at] = dd;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// dC (KEY = false) and dB (KEY = true): a block per (chunk, group, 128 state
// rows), over all heads of the group.  The chunk's own part is one product with
// the sum over the heads of L_ij dt_j (dout_i.x_j), so only the state part is a
// product per head; both sums are binary32.
// ---------------------------------------------------------------------------
template <int N>
struct DkShape {
    static constexpr int kW = N < 128 ? N : 128;                // state rows of a block
    static constexpr int kX = kChunk * kTile * 2;
    static constexpr int kState = kW * kTile * 2;
    static constexpr int kK = kChunk * kW * 2;
    static constexpr int kGates = kChunk * (8 + 4);
    static constexpr int kSmem = 2 * kX + (kState > kK ? kState : kK) + kGates;
};

template <int N, bool KEY>
__device__ __forceinline__ void dk_body(const Params& p) {
    using Sh = DkShape<N>;
    constexpr int W = Sh::kW, NB = W / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const Rows rg = slot_rows(p, blockIdx.x);
    if (!rg.valid) return;
    const int parts = N / W, group = blockIdx.y / parts, n0 = (blockIdx.y - group * parts) * W;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint32_t sx = smem_u32(smem), sy = sx + Sh::kX, ss = sy + Sh::kX;
    float2* b = reinterpret_cast<float2*>(smem + 2 * Sh::kX + (Sh::kState > Sh::kK ? Sh::kState : Sh::kK));
    float* dt = reinterpret_cast<float*>(b + kChunk);
    const int valid = rg.valid, row0 = warp * 16;
    const bool live = row0 < valid;
    const long long os = static_cast<long long>(p.H) * p.P;
    const uint32_t own = KEY ? sx : sy, other = KEY ? sy : sx;  // rows of this block's tokens, of the others
    const float* states = KEY ? p.df : p.sf;

    float sum[16][4], tot[NB][4];
    zero(sum);
    zero(tot);
    for (int hi = 0; hi < p.per; ++hi) {
        const int h = group * p.per + hi;
        const long long gate_at = (static_cast<long long>(blockIdx.x) * p.H + h) * kChunk;
        for (int tile = 0; tile < p.tiles; ++tile) {
            const int cols = min(kTile, p.P - tile * kTile);
            const long long cell = ((static_cast<long long>(blockIdx.x) * p.H + h) * p.tiles + tile) * N * kTile;
            __syncthreads();
            load_tile<2 * kTile, kChunk>(sx, p.x + rg.first * p.xs + static_cast<long long>(h) * p.P + tile * kTile, p.xs, valid, cols / 8);
            load_tile<2 * kTile, kChunk>(sy, p.dout + rg.first * os + static_cast<long long>(h) * p.P + tile * kTile, os, valid, cols / 8);
            cp_commit();
            if (threadIdx.x < kChunk) {
                b[threadIdx.x] = p.gb[gate_at + threadIdx.x];
                dt[threadIdx.x] = p.gdt[gate_at + threadIdx.x];
            }
            load_state<W, 1>(ss, states + cell + n0 * kTile);
            cp_wait<0>();
            __syncthreads();
            if (!live) continue;
            const float2 b0 = b[row0 + g], b8 = b[row0 + g + 8], be = b[kChunk - 1];
            uint32_t a[4][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) frag_a<2 * kTile>(a[ks], own, row0, ks, lane);
            // the state part
            const float w0 = KEY ? ex2_diff(be, b0) * dt[row0 + g] : ex2(b0.x + b0.y);
            const float w8 = KEY ? ex2_diff(be, b8) * dt[row0 + g + 8] : ex2(b8.x + b8.y);
#pragma unroll
            for (int nb = 0; nb < NB / 2; ++nb) {
                float t[2][4];
                zero(t);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint32_t v[4];
                    frag_b<2 * kTile>(v, ss, nb * 16, ks, lane);
                    mma(t[0], a[ks], v[0], v[1]);
                    mma(t[1], a[ks], v[2], v[3]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    tot[2 * nb + k][0] = fmaf(w0, t[k][0], tot[2 * nb + k][0]);
                    tot[2 * nb + k][1] = fmaf(w0, t[k][1], tot[2 * nb + k][1]);
                    tot[2 * nb + k][2] = fmaf(w8, t[k][2], tot[2 * nb + k][2]);
                    tot[2 * nb + k][3] = fmaf(w8, t[k][3], tot[2 * nb + k][3]);
                }
            }
            // the chunk's own pairs
#pragma unroll
            for (int ob = 0; ob < 8; ++ob) {
                if (KEY ? (ob < warp || ob * 16 >= valid) : ob > warp) continue;
                float t[2][4];
                zero(t);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint32_t v[4];
                    frag_b<2 * kTile>(v, other, ob * 16, ks, lane);
                    mma(t[0], a[ks], v[0], v[1]);
                    mma(t[1], a[ks], v[2], v[3]);
                }
#pragma unroll
                for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = ob * 16 + nb * 8 + 2 * q + (e & 1), r = row0 + g + (e >> 1) * 8;
                        const float2 br = (e >> 1) ? b8 : b0;
                        if (KEY) {
                            if (c >= r) sum[2 * ob + nb][e] = fmaf(t[nb][e], ex2_diff(b[c], br) * dt[r], sum[2 * ob + nb][e]);
                        } else {
                            if (c <= r) sum[2 * ob + nb][e] = fmaf(t[nb][e], ex2_diff(br, b[c]) * dt[c], sum[2 * ob + nb][e]);
                        }
                    }
            }
        }
    }
    __syncthreads();
    const bf16* keys = KEY ? p.Cm : p.Bm;
    const long long ks_ = KEY ? p.cs : p.bs;
    load_tile<2 * W, kChunk>(ss, keys + rg.first * ks_ + group * N + n0, ks_, valid, W / 8);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int ob = 0; ob < 8; ++ob) {
        if (KEY ? (ob < warp || ob * 16 >= valid) : ob > warp) continue;
        uint32_t a[4];
        a[0] = pack(sum[2 * ob][0], sum[2 * ob][1]);
        a[1] = pack(sum[2 * ob][2], sum[2 * ob][3]);
        a[2] = pack(sum[2 * ob + 1][0], sum[2 * ob + 1][1]);
        a[3] = pack(sum[2 * ob + 1][2], sum[2 * ob + 1][3]);
#pragma unroll
        for (int nb = 0; nb < NB / 2; ++nb) {
            uint32_t v[4];
            frag_bt<2 * W>(v, ss, nb * 16, ob, lane);
            mma(tot[2 * nb], a, v[0], v[1]);
            mma(tot[2 * nb + 1], a, v[2], v[3]);
        }
    }
    bf16* out = (KEY ? p.dBm : p.dCm) + (static_cast<long long>(rg.first) * p.G + group) * N + n0;
#pragma unroll
    for (int c = 0; c < (NB + 7) / 8; ++c) {
        float part[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[i][e] = 8 * c + i < NB ? tot[(8 * c + i) % NB][e] : 0.f;
        store_rows(out + c * 64, static_cast<long long>(p.G) * N, row0, valid, W - c * 64, part, lane);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) dk_kernel(const __grid_constant__ Params p) {
    wait_before();
    if (blockIdx.z == 0) {
        if (p.dCm) dk_body<N, false>(p);
    } else {
        if (p.dBm) dk_body<N, true>(p);
    }
}

// dA, dD: sums of the chunks' parts, eight interleaved runs in order, in binary64: thousands
// of parts whose signs differ.
__global__ void __launch_bounds__(256) sums_kernel(const __grid_constant__ Params p) {
    __shared__ double sh[8][33];
    wait_before();
    const int h = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float* out = blockIdx.y ? p.dD : p.dA;
    if (!out) return;
    const float* part = p.part + static_cast<long long>(blockIdx.y) * p.slots * p.H;
    double s = 0.;
    if (h < p.H)
        for (int i = w; i < p.slots; i += 8) s += part[static_cast<long long>(i) * p.H + h];
    sh[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && h < p.H) {
        for (int i = 1; i < 8; ++i) s += sh[i][threadIdx.x];
        out[h] = static_cast<float>(s);
    }
}

template <int N>
int backward_n(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    int err = cudaFuncSetAttribute(dx_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, DxShape<N>::kSmem);
    if (!err) err = cudaFuncSetAttribute(dk_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, DkShape<N>::kSmem);
    if (err) return err;
    if (p.slots) {
        const dim3 grid(p.slots, p.G * ((p.per + head_set - 1) / head_set));
        if (dx_tc_ok(p)) {
            err = launch_dx_tc(p, m, head_set, s);
        } else {
            err = launch(dx_kernel<N>, grid, kThreads, DxShape<N>::kSmem, s, false, p, head_set);
        }
        if (!err && (p.dBm || p.dCm)) {
            if (dk_tc_ok(p)) {
                err = launch_dk_tc(p, m, s);
            } else {
                err = launch(dk_kernel<N>, dim3(p.slots, p.G * (N / DkShape<N>::kW), 2), kThreads, DkShape<N>::kSmem, s, false, p);
            }
        }
        if (err) return err;
    }
    return p.dA || p.dD ? launch(sums_kernel, dim3((p.H + 31) / 32, 2), 256, 0, s, false, p) : 0;
}

}  // namespace

int launch_backward(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    switch (p.N) {
        case 16: return backward_n<16>(p, m, head_set, s);
        case 32: return backward_n<32>(p, m, head_set, s);
        case 64: return backward_n<64>(p, m, head_set, s);
        case 128: return backward_n<128>(p, m, head_set, s);
        default: return backward_n<256>(p, m, head_set, s);
    }
}

}  // namespace scan
}  // namespace rsq
