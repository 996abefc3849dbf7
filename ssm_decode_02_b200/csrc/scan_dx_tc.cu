// scan_dx_tc.cu -- dx and the gates' gradients on the fifth-generation tensor cores
// (tcgen05): the form of dx_kernel (scan_backward.cu, which has the formulas) for dk
// and dv of 64 and 128.
//
// A block takes one chunk and some heads of one group.  In tensor memory lie
//     g  = B C^T     128 x 128 tokens (j, i), once
//     w  = x dout^T  128 x 128 per head
//     pt = g . decays (bf16, left operand), i >= j
//     c  = pt dout   128 x 64 per tile of 64 columns
//     d  = B dS,  e = C S_0   128 x 64 per tile, the state in three bf16 terms
// with dx = dt (c + 2^(b_end-b_j) d) + D dout; the gates' sums are those of w . pt by
// row and by column (before pt is rounded), and the rows' products of d with x and of
// e with dout.  Warps, which meet at mbarriers only:
//   8 scorers     pt, and the sums of w . pt (by column: a transposing reduction over the lanes)
//   4 + 4 writers dx with its row sums; the row sums of e
//   8 converters  the states, binary32 in memory, to three terms; <S_0, dS>
//   2 loaders     x and dout, two stages
//   1 finisher    the gates' gradients of a head from the sums
//   1 issuer      of the products.
// Bound by instruction issue (23.5 thousand warp instructions per head and chunk, 51% of
// the issue slots; 13% of the tensor cycles) at 72 registers a thread: 4 x 2048 tokens, 80
// heads of 128 x 64, 303 to 324 us with caches cold; 806 with warp products.  Two groups of
// converters as in the states' kernel spill; states brought to L2 ahead, and issuing
// without a branch, were slower.
#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

constexpr int kScorers = 256, kWriters = 256, kConverters = 256, kLoaders = 64;
constexpr int kBlock = kScorers + kWriters + kConverters + kLoaders + 64;
constexpr int kUnits = 2;                       // ring of 64 state rows in three terms
constexpr int kRaw = 64 * kTile * 4;            // the same rows in binary32, two on their way
constexpr int kPlane = 64 * kTile * 2, kUnit = 3 * kPlane;
constexpr int kG = 0, kW = 128, kC = 256, kDd = 320, kE = 384, kPt = 448;
// sums of one head (floats)
constexpr int kRow = 0, kOwn = 512, kCol = 640, kIn = 1152, kFin = 1280, kDot = 1408, kThrough = 1536, kSums = 1544;

template <int N>
struct Shape {
    static constexpr int kKeys = kChunk * N * 2;
    static constexpr int kX = kChunk * kTile * 2;
    static constexpr int kSmem = 1024 + 2 * kKeys + 4 * kX + kUnits * kUnit + 2 * kRaw + 8 * 32 * (4 + 8) + 2 * kSums * 4 + 256;
};

// v[k] of the 32 lanes added up; lane l gets the sum of v[l].
__device__ __forceinline__ float transpose_sum(float (&v)[32], int lane) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int k = 0; k < d; ++k) {
            const float keep = up ? v[k + d] : v[k], send = up ? v[k] : v[k + d];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
    }
    return v[0];
}

template <int N>
__global__ void __launch_bounds__(kBlock, 1) dx_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ tc::Maps maps,
                                                           int head_set) {
    using Sh = Shape<N>;
    extern __shared__ uint8_t raw_smem[];
    wait_before();
    const Rows rg = slot_rows(p, blockIdx.x);
    const int sets = (p.per + head_set - 1) / head_set;
    const int group = blockIdx.y / sets, set = blockIdx.y - group * sets;
    const int h0 = group * p.per + set * head_set;
    const int heads = min(head_set, p.per - set * head_set), items = heads * p.tiles;
    const long long cells0 = static_cast<long long>(blockIdx.x) * p.H;
    if (!rg.valid) {
        // no rows: this slot adds nothing to the sums over tokens
        for (int i = threadIdx.x; i < heads; i += kBlock) {
            p.part[cells0 + h0 + i] = 0.f;
            p.part[static_cast<long long>(p.slots) * p.H + cells0 + h0 + i] = 0.f;
        }
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, valid = rg.valid;
    const long long os = static_cast<long long>(p.H) * p.P;

    uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem), sc = sb + Sh::kKeys, stages = sc + Sh::kKeys, units = stages + 4 * Sh::kX, raws = units + kUnits * kUnit;
    float* facs = reinterpret_cast<float*>(smem + 2 * Sh::kKeys + 4 * Sh::kX + kUnits * kUnit + 2 * kRaw);   // [8 warps][32]
    float2* pairs = reinterpret_cast<float2*>(facs + 8 * 32);                                          // [8 warps][32]
    float* sums = reinterpret_cast<float*>(pairs + 8 * 32);                                        // [2][kSums]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sums + 2 * kSums);
    uint32_t bar = smem_u32(tmem_slot + 2);
    auto next_bar = [&](int n) {
        const uint32_t b = bar;
        bar += 8 * n;
        return b;
    };
    const uint32_t keys = next_bar(1), g_done = next_bar(1), loaded = next_bar(2), emptied = next_bar(2), unit_written = next_bar(kUnits),
                   unit_free = next_bar(kUnits), w_done = next_bar(1), w_free = next_bar(1), pt_written = next_bar(1),
                   pt_free = next_bar(1), cd_done = next_bar(1), cd_free = next_bar(1), e_done = next_bar(1), e_free = next_bar(1),
                   sums_done = next_bar(2), sums_free = next_bar(2), raw_done = next_bar(2), raw_free = next_bar(2);
    if (warp == 0) tc::tmem_alloc(smem_u32(tmem_slot), 512);
    if (threadIdx.x == 0) {
        mbar_init(keys, 2);
        for (uint32_t b : {g_done, w_done, pt_free, cd_done, e_done}) mbar_init(b, 1);
        for (uint32_t b : {w_free, pt_written}) mbar_init(b, kScorers);
        for (uint32_t b : {cd_free, e_free}) mbar_init(b, 128);
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(unit_written + 8 * i, kConverters);
            mbar_init(unit_free + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(loaded + 8 * i, 1);
            mbar_init(raw_done + 8 * i, 1);
            mbar_init(raw_free + 8 * i, kConverters);
            mbar_init(emptied + 8 * i, kWriters);
            mbar_init(sums_done + 8 * i, kScorers + kWriters + kConverters);
            mbar_init(sums_free + 8 * i, 32);
        }
        fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot, lanes = (static_cast<uint32_t>(warp) & 3) << 21;
    const int quarter = warp & 3, row = quarter * 32 + lane;   // of the warps that reach tensor memory

    if (threadIdx.x < kScorers) {
        const int half = warp >> 2;                             // columns 64 half ..
        float* fac = facs + warp * 32;
        float2* pair = pairs + warp * 32;
        const bool any = half * 2 + 1 >= quarter;               // some block of its columns is not before its rows
        float2 nc[2], nr = make_float2(0.f, 0.f);
        float nd = 0.f;
        auto read = [&](int i) {
            if (i >= heads || !any) return;
            const long long at = (cells0 + h0 + i) * kChunk;
#pragma unroll
            for (int k = 0; k < 2; ++k) nc[k] = p.gb[at + half * 64 + k * 32 + lane];
            nr = p.gb[at + row];
            nd = p.gdt[at + row];
        };
        read(0);
        bool ok = tc::wait_warp(g_done, 0, p.flag);
        for (int i = 0; i < heads && ok; ++i) {
            const float2 bc[2] = {nc[0], nc[1]}, br = nr;
            const float dt = nd;
            read(i + 1);
            if (!(ok = tc::wait_warp(w_done, i, p.flag))) break;
            if (i && !(ok = tc::wait_warp(pt_free, i - 1, p.flag))) break;
            if (i >= 2 && !(ok = tc::wait_warp(sums_free + 8 * (i & 1), i / 2 - 1, p.flag))) break;
            tc::fence_after();
            float* out = sums + (i & 1) * kSums;
#pragma unroll 1   // the instruction cache holds the roles' loops only if they stay small
            for (int k = 0; k < 2; ++k) {
                const int cols = half * 2 + k;                  // this block of 32 columns
                const float2 bk = k ? bc[1] : bc[0];
                const uint32_t dst = tmem + kPt + cols * 16 + lanes;
                if (cols < quarter) {                           // before every row: zero, once
                    if (i == 0) {
                        const uint32_t z[16] = {};
                        tc::tmem_st16(dst, z);
                    }
                    continue;
                }
                const bool diagonal = cols == quarter;
                const int meet = diagonal ? 31 : 0;
                const float2 bm = make_float2(__shfl_sync(0xffffffffu, bk.x, meet), __shfl_sync(0xffffffffu, bk.y, meet));
                const float first = __shfl_sync(0xffffffffu, bk.x, 0);
                const float r = ex2_diff(bm, br);
                const bool direct = diagonal && !(first - bm.x < 100.f);
                __syncwarp();
                fac[lane] = ex2_diff(bk, bm);
                if (direct) pair[lane] = bk;
                __syncwarp();
                float v[32], own = 0.f, rows = 0.f, run = 0.f;
                uint32_t o[16];
#pragma unroll
                for (int s = 1; s >= 0; --s) {
                    float g[16], w[16];
                    tc::tmem_ld16(g, tmem + kG + cols * 32 + s * 16 + lanes);
                    tc::tmem_ld16(w, tmem + kW + cols * 32 + s * 16 + lanes);
                    tc::tmem_ld_wait();
                    if (!direct) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 f = reinterpret_cast<const float4*>(fac)[s * 4 + q];
                            g[4 * q] *= r * f.x;
                            g[4 * q + 1] *= r * f.y;
                            g[4 * q + 2] *= r * f.z;
                            g[4 * q + 3] *= r * f.w;
                        }
                    } else {
#pragma unroll 1
                        for (int q = 0; q < 16; ++q) {
                            const float f = ex2_diff(s * 16 + q >= lane ? pair[s * 16 + q] : br, br);
#pragma unroll
                            for (int e = 0; e < 16; ++e) g[e] *= e == q ? f : 1.f;
                        }
                    }
                    if (diagonal) {
#pragma unroll
                        for (int q = 15; q >= 0; --q) {         // v: the pairs around each column
                            const int c = s * 16 + q;
                            g[q] = c < lane ? 0.f : g[q];
                            const float z = w[q] * g[q];
                            if (c == lane) own = z;
                            rows += c > lane ? z : 0.f;
                            run = fmaf(z, dt, run);
                            v[c] = c > lane ? run : 0.f;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float z = w[q] * g[q];
                            rows += z;
                            v[s * 16 + q] = z * dt;
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[s * 8 + q] = pack(g[2 * q], g[2 * q + 1]);
                }
                tc::tmem_st16(dst, o);
                out[kCol + quarter * 128 + cols * 32 + lane] = transpose_sum(v, lane);
                out[kRow + cols * 128 + row] = rows;
                if (diagonal) out[kOwn + row] = own;
            }
            tc::tmem_st_wait();
            tc::fence_before();
            mbar_arrive(w_free);
            mbar_arrive(pt_written);
            mbar_arrive(sums_done + 8 * (i & 1));
        }
    } else if (threadIdx.x < kScorers + kWriters / 2) {
        // dx
        float fin = 0.f, dot = 0.f;
        float2 nb = make_float2(0.f, 0.f), ne = nb;
        float nd = 0.f, nD = 0.f;
        auto read = [&](int it) {
            if (it >= items) return;
            const int h = h0 + it / p.tiles;
            nb = p.gb[(cells0 + h) * kChunk + row];
            ne = p.gb[(cells0 + h) * kChunk + kChunk - 1];
            nd = p.gdt[(cells0 + h) * kChunk + row];
            if (p.D) nD = __ldg(p.D + h);
        };
        read(0);
        for (int it = 0; it < items; ++it) {
            const int head = it / p.tiles, tile = it - head * p.tiles, h = h0 + head;
            const float w = ex2_diff(ne, nb), dt = nd, D = nD;
            read(it + 1);
            const uint32_t sx = stages + (it & 1) * 2 * Sh::kX, sy = sx + Sh::kX;
            if (!tc::wait_warp(cd_done, it, p.flag)) break;
            tc::fence_after();
#pragma unroll 1
            for (int s = 0; s < 8; ++s) {
                float c[8], d[8];
                tc::tmem_ld8(c, tmem + kC + s * 8 + lanes);
                tc::tmem_ld8(d, tmem + kDd + s * 8 + lanes);
                uint32_t x[4], y[4], o[4];
                const uint32_t ax = sx + tile_at<128>(row, s);
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(ax) : "memory");
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(sy + tile_at<128>(row, s)) : "memory");
                tc::tmem_ld_wait();
                if (s == 7) {
                    tc::fence_before();
                    mbar_arrive(cd_free);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float d0 = d[2 * k] * w, d1 = d[2 * k + 1] * w;
                    fin = fmaf(d0, lo_of(x[k]), fmaf(d1, hi_of(x[k]), fin));
                    dot = fmaf(lo_of(y[k]), lo_of(x[k]), fmaf(hi_of(y[k]), hi_of(x[k]), dot));
                    o[k] = pack(fmaf(dt, c[2 * k] + d0, D * lo_of(y[k])), fmaf(dt, c[2 * k + 1] + d1, D * hi_of(y[k])));
                }
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(ax), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
            }
            __syncwarp();
            if (p.dx) {  // this warp's 32 rows, four whole rows at a time
                bf16* out = p.dx + static_cast<long long>(rg.first) * os + static_cast<long long>(h) * p.P + tile * kTile;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = quarter * 32 + k * 4 + (lane >> 3);
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(sx + tile_at<128>(r, lane & 7)) : "memory");
                    if (r < valid) *reinterpret_cast<uint4*>(out + r * os + (lane & 7) * 8) = v;
                }
            }
            tc::fence_smem();   // boxes overwrite what was written here
            mbar_arrive(emptied + 8 * (it & 1));
            if (tile == p.tiles - 1) {
                if (head >= 2 && !tc::wait_warp(sums_free + 8 * (head & 1), head / 2 - 1, p.flag)) break;
                float* out = sums + (head & 1) * kSums;
                out[kFin + row] = fin;
                out[kDot + row] = dot;
                mbar_arrive(sums_done + 8 * (head & 1));
                fin = dot = 0.f;
            }
        }
    } else if (threadIdx.x < kScorers + kWriters) {
        // the rows' products of e with dout
        float in = 0.f;
        for (int it = 0; it < items; ++it) {
            const int head = it / p.tiles, tile = it - head * p.tiles;
            const float2 b = p.gb[(cells0 + h0 + head) * kChunk + row];
            const uint32_t sy = stages + (it & 1) * 2 * Sh::kX + Sh::kX;
            if (!tc::wait_warp(e_done, it, p.flag)) break;
            tc::fence_after();
#pragma unroll 2
            for (int s = 0; s < 8; ++s) {
                float e[8];
                uint32_t y[4];
                tc::tmem_ld8(e, tmem + kE + s * 8 + lanes);
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(sy + tile_at<128>(row, s)) : "memory");
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) in = fmaf(e[2 * k], lo_of(y[k]), fmaf(e[2 * k + 1], hi_of(y[k]), in));
            }
            tc::fence_before();
            mbar_arrive(e_free);
            mbar_arrive(emptied + 8 * (it & 1));
            if (tile == p.tiles - 1) {
                if (head >= 2 && !tc::wait_warp(sums_free + 8 * (head & 1), head / 2 - 1, p.flag)) break;
                sums[(head & 1) * kSums + kIn + row] = in * ex2(b.x + b.y);
                mbar_arrive(sums_done + 8 * (head & 1));
                in = 0.f;
            }
        }
    } else if (threadIdx.x < kScorers + kWriters + kConverters) {
        // unit: rows 64 part .. of dS (even) or S_0 (odd) of a tile, 16 KB in a row in memory,
        // copied whole; this thread: rows r + 16 k, columns 4 c ..
        const int i0 = threadIdx.x - kScorers - kWriters, r = i0 >> 4, c = i0 & 15, cw = i0 >> 5;
        const int per_tile = 2 * (N / 64), total = items * per_tile;
        auto fetch = [&](int u) {
            const int it = u / per_tile, part = (u - it * per_tile) >> 1;
            const long long cell = (cells0 + h0 + it / p.tiles) * p.tiles + it % p.tiles;
            mbar_arrive_expect_tx(raw_done + 8 * (u & 1), kRaw);
            bulk_g2s(raws + (u & 1) * kRaw, ((u & 1) ? p.sf : p.df) + (cell * N + part * 64) * kTile, kRaw, raw_done + 8 * (u & 1));
        };
        if (i0 == 0)
            for (int u = 0; u < min(2, total); ++u) fetch(u);
        float4 ds[4];
        float through = 0.f;
        int u = 0;
        for (; u < total; ++u) {
            float4 v[4];
            if (!tc::wait_warp(raw_done + 8 * (u & 1), u / 2, p.flag)) break;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[k].x), "=f"(v[k].y), "=f"(v[k].z), "=f"(v[k].w)
                             : "r"(raws + (u & 1) * kRaw + (r + 16 * k) * kTile * 4 + c * 16) : "memory");
            mbar_arrive(raw_free + 8 * (u & 1));
            if (u & 1) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    through = fmaf(v[k].x, ds[k].x, fmaf(v[k].y, ds[k].y, fmaf(v[k].z, ds[k].z, fmaf(v[k].w, ds[k].w, through))));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) ds[k] = v[k];
            }
            if (u >= kUnits && !tc::wait_warp(unit_free + 8 * (u % kUnits), u / kUnits - 1, p.flag)) break;
            const uint32_t to = units + (u % kUnits) * kUnit + 8 * (c & 1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t t[3][2];
                split3(v[k].x, v[k].y, t[0][0], t[1][0], t[2][0]);
                split3(v[k].z, v[k].w, t[0][1], t[1][1], t[2][1]);
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(to + m * kPlane + tile_at<128>(r + 16 * k, c >> 1)), "r"(t[m][0]),
                                 "r"(t[m][1])
                                 : "memory");
            }
            tc::fence_smem();
            mbar_arrive(unit_written + 8 * (u % kUnits));
            if (i0 == 0 && u + 2 < total) {
                if (mbar_wait(raw_free + 8 * (u & 1), (u / 2) & 1, kWaitIters))
                    fetch(u + 2);
                else
                    atomicOr(p.flag, kFlagTimeout);
            }
            __syncwarp();
            const int head = u / (per_tile * p.tiles);
            if (u == (head + 1) * per_tile * p.tiles - 1) {     // the head's last unit
                if (head >= 2 && !tc::wait_warp(sums_free + 8 * (head & 1), head / 2 - 1, p.flag)) break;
#pragma unroll
                for (int d = 16; d; d >>= 1) through += __shfl_xor_sync(0xffffffffu, through, d);
                if (lane == 0) sums[(head & 1) * kSums + kThrough + cw] = through;
                __syncwarp();
                mbar_arrive(sums_done + 8 * (head & 1));
                through = 0.f;
            }
        }
        // left early: no copy may still be on its way when the block ends
        if (i0 == 0)
            for (int v = u; v < min(u + 2, total); ++v) mbar_wait(raw_done + 8 * (v & 1), (v / 2) & 1, kDrainIters);
    } else if (threadIdx.x < kScorers + kWriters + kConverters + kLoaders) {
        // a warp for each stage.  A whole chunk's tiles come in boxes; the last rows of a
        // sequence, which the next one's may follow, row by row with zeros behind them.
        const int mine = warp & 1, t = lane >> 3, c = lane & 7;
        const bool whole = valid == kChunk;
        auto rows = [&](uint32_t dst, const bf16* src, long long stride) {
#pragma unroll 4
            for (int j = 0; j < kChunk / 4; ++j) {
                const bool on = t + 4 * j < valid;
                cp16(dst + tile_at<128>(t + 4 * (j & 1), c) + (j >> 1) * 1024, src + (on ? (t + 4 * j) * stride : 0) + c * 8, on);
            }
        };
        auto announce = [&](uint32_t b) {
            cp_commit();
            cp_wait<0>();
            tc::fence_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        const uint32_t sk = mine ? sc : sb;
        if (whole) {
            if (lane == 0) {
                mbar_arrive_expect_tx(keys, Sh::kKeys);
#pragma unroll
                for (int b = 0; b < N / 64; ++b)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        tc::box(sk + b * kChunk * 128 + k * tc::kBox, mine ? &maps.Cm : &maps.Bm, group * N + b * 64, rg.first + k * 64, keys);
            }
            __syncwarp();
        } else {
#pragma unroll 1
            for (int b = 0; b < N / 64; ++b)
                rows(sk + b * kChunk * 128, (mine ? p.Cm + rg.first * p.cs : p.Bm + rg.first * p.bs) + group * N + b * 64, mine ? p.cs : p.bs);
            announce(keys);
        }
        for (int it = mine; it < items; it += 2) {
            if (it >= 2 && !tc::wait_warp(emptied + 8 * mine, it / 2 - 1, p.flag)) break;
            const int h = h0 + it / p.tiles, tile = it % p.tiles;
            const uint32_t sx = stages + mine * 2 * Sh::kX, b = loaded + 8 * mine;
            if (whole) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(b, 2 * Sh::kX);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        tc::box(sx + k * tc::kBox, &maps.x, h * p.P + tile * kTile, rg.first + k * 64, b);
                        tc::box(sx + Sh::kX + k * tc::kBox, &maps.dout, h * p.P + tile * kTile, rg.first + k * 64, b);
                    }
                }
                __syncwarp();
            } else {
                rows(sx, p.x + rg.first * p.xs + static_cast<long long>(h) * p.P + tile * kTile, p.xs);
                rows(sx + Sh::kX, p.dout + rg.first * os + static_cast<long long>(h) * p.P + tile * kTile, os);
                announce(b);
            }
        }
    } else if (warp == (kBlock >> 5) - 2) {
        // a head's gates: lane l has tokens 4 l .. 4 l + 3
        for (int i = 0; i < heads; ++i) {
            const int h = h0 + i;
            const float4 dt4 = *reinterpret_cast<const float4*>(p.gdt + (cells0 + h) * kChunk + lane * 4);
            const float2 be = p.gb[(cells0 + h) * kChunk + kChunk - 1];
            const float ah = p.decay ? 0.f : __ldg(p.A + h);
            const float dt[4] = {dt4.x, dt4.y, dt4.z, dt4.w};
            if (!tc::wait_warp(sums_done + 8 * (i & 1), i / 2, p.flag)) break;
            const float* in = sums + (i & 1) * kSums;
            HeadSums hs{in + kCol, in + kRow, in + kOwn, in + kIn, in + kFin, in + kDot, 0.f};
#pragma unroll
            for (int w = 0; w < 8; ++w) hs.through += in[kThrough + w];
            hs.through *= ex2(be.x + be.y);
            float dl[4], dir[4], dd, da = 0.f;
            head_gates<4>(hs, dt, valid, lane, dl, dir, dd);
            __syncwarp();
            mbar_arrive(sums_free + 8 * (i & 1));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = lane * 4 + k;
                if (t >= valid) continue;
                const long long at = static_cast<long long>(rg.first + t) * p.H + h;
                if (p.decay && __ldg(p.decay + at) == 0.f) dl[k] = 0.f;  // nothing passes, not 0 times a non-finite value either
                if (p.dlog) p.dlog[at] = dl[k];
                if (p.ddt) p.ddt[at] = p.decay ? dir[k] : fmaf(ah, dl[k], dir[k]);
                da = fmaf(dt[k], dl[k], da);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) da += __shfl_xor_sync(0xffffffffu, da, d);
            if (lane == 0) {
                p.part[cells0 + h] = da;
                p.part[static_cast<long long>(p.slots) * p.H + cells0 + h] = dd;
            }
        }
    } else {
        auto wait = [&](uint32_t b, int phase) { return tc::wait_warp(b, phase, p.flag); };
        bool ok = wait(keys, 0);
        const uint64_t bd = tc::desc(sb, 16), cd = tc::desc(sc, 16), stage0 = tc::desc(stages, 16), unit0 = tc::desc(units, 16);
        if (ok) {
            tc::fence_after();
            constexpr uint32_t id = tc::idesc(kChunk, false, false);
            if (tc::elect()) {
#pragma unroll
                for (int ks = 0; ks < N / 16; ++ks) {
                    const uint32_t o = ((ks / 4) * kChunk * 128 + (ks % 4) * 32) >> 4;
                    tc::mma(tmem + kG, bd + o, cd + o, id, ks);
                }
                tc::commit(g_done);
            }
            __syncwarp();
        }
        constexpr uint32_t id_w = tc::idesc(kChunk, false, false), id = tc::idesc(kTile, false, true);
        int unit = 0, head = 0, tile = 0;
        for (int it = 0; it < items && ok; ++it) {
            if (tile == 0) {
                if (head && !(ok = wait(w_free, head - 1))) break;
                for (int t = 0; t < p.tiles && ok; ++t) {
                    if (!(ok = wait(loaded + 8 * ((it + t) & 1), (it + t) / 2))) break;
                    tc::fence_after();
                    const uint64_t xd = stage0 + ((it + t) & 1) * (2 * Sh::kX >> 4), yd = xd + (Sh::kX >> 4);
                    if (tc::elect()) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) tc::mma(tmem + kW, xd + ks * 2, yd + ks * 2, id_w, t || ks);
                        if (t == p.tiles - 1) tc::commit(w_done);
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            if (it && !(ok = wait(cd_free, it - 1) && wait(e_free, it - 1))) break;
            for (int part = 0; part < N / 64 && ok; ++part)
                for (int which = 0; which < 2 && ok; ++which, ++unit) {
                    if (!(ok = wait(unit_written + 8 * (unit % kUnits), unit / kUnits))) break;
                    tc::fence_after();
                    const uint64_t a = (which ? cd : bd) + part * (kChunk * 128 >> 4), b = unit0 + (unit % kUnits) * (kUnit >> 4);
                    const uint32_t d = tmem + (which ? kE : kDd);
                    if (tc::elect()) {
#pragma unroll
                        for (int m = 2; m >= 0; --m)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc::mma(d, a + ks * 2, b + ((m * kPlane + ks * 2048) >> 4), id, m != 2 || ks || part);
                        tc::commit(unit_free + 8 * (unit % kUnits));
                    }
                    __syncwarp();
                }
            if (!ok) break;
            if (tc::elect()) tc::commit(e_done);
            __syncwarp();
            if (tile == 0 && !(ok = wait(pt_written, head))) break;
            tc::fence_after();
            const uint64_t yd = stage0 + (((it & 1) * 2 + 1) * Sh::kX >> 4);
            const bool last = tile == p.tiles - 1;
            if (tc::elect()) {
#pragma unroll
                for (int ks = 0; ks < kChunk / 16; ++ks) tc::mma_ta(tmem + kC, tmem + kPt + ks * 8, yd + ks * 128, id, ks);
                tc::commit(cd_done);
                if (last) tc::commit(pt_free);
            }
            __syncwarp();
            tile = last ? 0 : tile + 1;
            head += last;
        }
        if (!ok) {  // left early: no box may still be on its way when the block ends
            for (int i = 0; i < 2; ++i)
                for (int k = 0; k < 2; ++k) mbar_wait(loaded + 8 * i, k, kDrainIters);
            mbar_wait(keys, 0, kDrainIters);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 512);
}

template <int N>
int run(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    const int err = cudaFuncSetAttribute(dx_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<N>::kSmem);
    if (err) return err;
    const dim3 grid(p.slots, p.G * ((p.per + head_set - 1) / head_set));
    return launch(dx_tc_kernel<N>, grid, kBlock, Shape<N>::kSmem, s, false, p, m, head_set);
}

}  // namespace

int launch_dx_tc(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    return p.N == 64 ? run<64>(p, m, head_set, s) : run<128>(p, m, head_set, s);
}

}  // namespace scan
}  // namespace rsq
