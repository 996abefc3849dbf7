// scan_dk_tc.cu -- dB and dC on the fifth-generation tensor cores (tcgen05): the form
// of dk_kernel (scan_backward.cu) for dk of 64, 128 and 256 and dv of whole 64-column
// tiles.
//
// A block takes one chunk, one group and 64 state rows, over all heads of the group:
//     dC = sum_h 2^b (dout S_0^T) + M B,   dB = sum_h 2^(b_end-b) dt (x dS^T) + M^T C,
//     M  = sum_h L . dt . (dout x^T)       (128 x 128 tokens, i >= j)
// so that the products with the keys are two at the end, whatever the number of heads;
// M is rounded to bf16 once, after the sum.  M lies in tensor memory, where the
// scorers add to it; the other two sums lie in registers, a thread one row of 64.
// Warps, which meet at mbarriers only:
//   8 scorers, 4 + 4 summers, 4 converters (states to bf16), 3 loaders, 1 issuer.
// 128 blocks, one round, on 148 SMs, each bound by the chain through its roles (46% of the
// issue slots, 13% of the tensor cycles): 4 x 2048 tokens, 80 heads of 128 x 64, 150 us;
// 520 with warp products.
#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

constexpr int kScorers = 256, kSummers = 256, kConverters = 128, kLoaders = 96;
constexpr int kBlock = kScorers + kSummers + kConverters + kLoaders + 32;
constexpr int kStages = 3;                      // of x and dout, a loader warp each
constexpr int kUnits = 4, kRaws = 4;            // rings of 64 state rows in bf16, and in binary32 on their way
constexpr int kUnit = 64 * kTile * 2, kRaw = 64 * kTile * 4;
constexpr int kX = kChunk * kTile * 2;
constexpr int kW = 0, kM = 256, kT = 384;       // tensor memory: two of dout x^T, M, dout S^T and x dS^T
// M and the keys come where the stages were
constexpr int kSmem = 1024 + kStages * 2 * kX + kUnits * kUnit + kRaws * kRaw + 8 * 32 * (2 * 4 + 16) + 384;

__global__ void __launch_bounds__(kBlock, 1) dk_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ tc::Maps maps) {
    extern __shared__ uint8_t raw_smem[];
    wait_before();
    const Rows rg = slot_rows(p, blockIdx.x);
    if (!rg.valid) return;
    const int parts = p.N / 64, group = blockIdx.y / parts, n0 = (blockIdx.y - group * parts) * 64;
    const int h0 = group * p.per, heads = p.per, items = heads * p.tiles;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, valid = rg.valid;
    const long long os = static_cast<long long>(p.H) * p.P, cells0 = static_cast<long long>(blockIdx.x) * p.H;

    uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t stages = smem_u32(smem), units = stages + kStages * 2 * kX, raws = units + kUnits * kUnit;
    const uint32_t sm = stages, sk = sm + 2 * kX;  // after the last head: M; B, C
    float* facs = reinterpret_cast<float*>(smem + kStages * 2 * kX + kUnits * kUnit + kRaws * kRaw);   // [8 warps][2][32]
    float4* pairs = reinterpret_cast<float4*>(facs + 8 * 64);                  // [8 warps][32]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pairs + 8 * 32);
    uint32_t bar = smem_u32(tmem_slot + 2);
    auto next_bar = [&](int n) {
        const uint32_t b = bar;
        bar += 8 * n;
        return b;
    };
    const uint32_t keys = next_bar(1), loaded = next_bar(kStages), emptied = next_bar(kStages), unit_written = next_bar(kUnits),
                   unit_free = next_bar(kUnits), w_done = next_bar(2), w_free = next_bar(2), t_done = next_bar(1), t_free = next_bar(1),
                   m_written = next_bar(1), f_done = next_bar(1), heads_done = next_bar(1), raw_done = next_bar(kRaws), raw_free = next_bar(kRaws);
    if (warp == 0) tc::tmem_alloc(smem_u32(tmem_slot), 512);
    if (threadIdx.x == 0) {
        mbar_init(keys, 2);
        mbar_init(t_done, 1);
        mbar_init(t_free, kSummers);
        mbar_init(m_written, kScorers);
        mbar_init(f_done, 1);
        mbar_init(heads_done, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(loaded + 8 * i, 1);
            mbar_init(emptied + 8 * i, 1);
        }
        for (int i = 0; i < kRaws; ++i) {
            mbar_init(raw_done + 8 * i, 1);
            mbar_init(raw_free + 8 * i, kConverters);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(w_done + 8 * i, 1);
            mbar_init(w_free + 8 * i, kScorers);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(unit_written + 8 * i, kConverters);
            mbar_init(unit_free + 8 * i, 1);
        }
        fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot, lanes = (static_cast<uint32_t>(warp) & 3) << 21;
    const int quarter = warp & 3, row = quarter * 32 + lane;

    if (threadIdx.x < kScorers) {
        const int half = warp >> 2;                             // columns 64 half ..
        float* fac = facs + warp * 64;
        float4* pair = pairs + warp * 32;
        const bool any = half * 2 <= quarter;
        float2 nc[2] = {}, nr = make_float2(0.f, 0.f);
        float nd[2] = {};
        auto read = [&](int i) {
            if (i >= heads || !any) return;
            const long long at = (cells0 + h0 + i) * kChunk;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                nc[k] = p.gb[at + half * 64 + k * 32 + lane];
                nd[k] = p.gdt[at + half * 64 + k * 32 + lane];
            }
            nr = p.gb[at + row];
        };
        read(0);
        bool ok = true;
        for (int i = 0; i < heads; ++i) {
            const float2 bc[2] = {nc[0], nc[1]}, br = nr;
            const float dt[2] = {nd[0], nd[1]};
            read(i + 1);
            if (!(ok = tc::wait_warp(w_done + 8 * (i & 1), i / 2, p.flag))) break;
            tc::fence_after();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int cols = half * 2 + k;
                if (cols > quarter) continue;                   // behind every row
                const bool diagonal = cols == quarter;
                const int meet = diagonal ? 0 : 31;
                const float2 bm = make_float2(__shfl_sync(0xffffffffu, bc[k].x, meet), __shfl_sync(0xffffffffu, bc[k].y, meet));
                const float last = __shfl_sync(0xffffffffu, bc[k].x, 31);
                const float r = ex2_diff(br, bm);
                const bool direct = diagonal && !(bm.x - last < 100.f);
                __syncwarp();
                fac[k * 32 + lane] = dt[k] * ex2_diff(bm, bc[k]);
                if (direct) pair[lane] = make_float4(bc[k].x, bc[k].y, dt[k], 0.f);
                __syncwarp();
                const uint32_t src = tmem + kW + (i & 1) * 128 + cols * 32 + lanes, dst = tmem + kM + cols * 32 + lanes;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    float w[16], m[16];
                    tc::tmem_ld16(w, src + s * 16);
                    if (i)
                        tc::tmem_ld16(m, dst + s * 16);
                    else
#pragma unroll
                        for (int q = 0; q < 16; ++q) m[q] = 0.f;
                    tc::tmem_ld_wait();
                    if (direct) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const int c = s * 16 + q;
                            const float4 e = pair[c];
                            const float f = c <= lane ? ex2_diff(br, make_float2(e.x, e.y)) * e.z : 0.f;
                            m[q] = fmaf(c <= lane ? w[q] : 0.f, f, m[q]);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 f = reinterpret_cast<const float4*>(fac + k * 32)[s * 4 + q];
                            w[4 * q] *= r * f.x;
                            w[4 * q + 1] *= r * f.y;
                            w[4 * q + 2] *= r * f.z;
                            w[4 * q + 3] *= r * f.w;
                        }
                        if (diagonal) {
#pragma unroll
                            for (int q = 0; q < 16; ++q) w[q] = s * 16 + q <= lane ? w[q] : 0.f;
                        }
#pragma unroll
                        for (int q = 0; q < 16; ++q) m[q] += w[q];
                    }
                    tc::tmem_st16(dst + s * 16, reinterpret_cast<const uint32_t(&)[16]>(m));
                }
            }
            tc::tmem_st_wait();
            tc::fence_before();
            mbar_arrive(w_free + 8 * (i & 1));
        }
        // M as bf16 rows where the stages were, once every product is done with them: the
        // left operand, and transposed
        if (ok && (ok = tc::wait_warp(heads_done, 0, p.flag))) {
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int cols = half * 2 + s / 4;
                float m[8];
                if (cols <= quarter) {
                    tc::tmem_ld8(m, tmem + kM + half * 64 + s * 8 + lanes);
                    tc::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) m[q] = 0.f;
                }
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(sm + half * kX + tile_at<128>(row, s)), "r"(pack(m[0], m[1])),
                             "r"(pack(m[2], m[3])), "r"(pack(m[4], m[5])), "r"(pack(m[6], m[7]))
                             : "memory");
            }
            tc::fence_smem();
            mbar_arrive(m_written);
        }
    } else if (threadIdx.x < kScorers + kSummers) {
        const int key = (warp - kScorers / 32) >> 2;            // 0: dC, 1: dB
        bf16* out = key ? p.dBm : p.dCm;
        float tot[64];
#pragma unroll
        for (int k = 0; k < 64; ++k) tot[k] = 0.f;
        float2 nb = make_float2(0.f, 0.f), ne = nb;
        float nd = 0.f;
        auto read = [&](int i) {
            if (i >= heads) return;
            const long long at = (cells0 + h0 + i) * kChunk;
            nb = p.gb[at + row];
            if (key) {
                ne = p.gb[at + kChunk - 1];
                nd = p.gdt[at + row];
            }
        };
        read(0);
        bool ok = true;
        for (int i = 0; i <= heads && ok; ++i) {
            const float w = i == heads ? 1.f : (key ? ex2_diff(ne, nb) * nd : ex2(nb.x + nb.y));
            read(i + 1);
            // after the heads' products the one with M
            if (!(ok = tc::wait_warp(i < heads ? t_done : f_done, i < heads ? i : 0, p.flag))) break;
            tc::fence_after();
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                float t[8];
                tc::tmem_ld8(t, tmem + kT + key * 64 + s * 8 + lanes);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) tot[s * 8 + k] = fmaf(w, t[k], tot[s * 8 + k]);
            }
            tc::fence_before();
            if (i < heads) mbar_arrive(t_free);
        }
        if (ok && out && row < valid) {
            out += (static_cast<long long>(rg.first + row) * p.G + group) * p.N + n0;
#pragma unroll
            for (int s = 0; s < 8; ++s)
                *reinterpret_cast<uint4*>(out + s * 8) = make_uint4(pack(tot[s * 8], tot[s * 8 + 1]), pack(tot[s * 8 + 2], tot[s * 8 + 3]),
                                                                    pack(tot[s * 8 + 4], tot[s * 8 + 5]), pack(tot[s * 8 + 6], tot[s * 8 + 7]));
        }
    } else if (threadIdx.x < kScorers + kSummers + kConverters) {
        // unit: the block's 64 rows of S_0 (even) or dS (odd) of a tile, 16 KB in a row in
        // memory, copied whole; this thread: rows r + 8 k, columns 4 c ..
        const int i0 = threadIdx.x - kScorers - kSummers, r = i0 >> 4, c = i0 & 15, total = 2 * items;
        auto fetch = [&](int u) {
            const int it = u >> 1;
            const long long cell = (cells0 + h0 + it / p.tiles) * p.tiles + it % p.tiles;
            const uint32_t b = raw_done + 8 * (u % kRaws);
            mbar_arrive_expect_tx(b, kRaw);
            bulk_g2s(raws + (u % kRaws) * kRaw, ((u & 1) ? p.df : p.sf) + (cell * p.N + n0) * kTile, kRaw, b);
        };
        if (i0 == 0)
            for (int u = 0; u < min(kRaws, total); ++u) fetch(u);
        int u = 0;
        for (; u < total; ++u) {
            if (!tc::wait_warp(raw_done + 8 * (u % kRaws), u / kRaws, p.flag)) break;
            if (u >= kUnits && !tc::wait_warp(unit_free + 8 * (u % kUnits), u / kUnits - 1, p.flag)) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float4 v;
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                             : "r"(raws + (u % kRaws) * kRaw + (r + 8 * k) * kTile * 4 + c * 16) : "memory");
                asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(units + (u % kUnits) * kUnit + tile_at<128>(r + 8 * k, c >> 1) + 8 * (c & 1)),
                             "r"(pack(v.x, v.y)), "r"(pack(v.z, v.w))
                             : "memory");
            }
            mbar_arrive(raw_free + 8 * (u % kRaws));
            tc::fence_smem();
            mbar_arrive(unit_written + 8 * (u % kUnits));
            if (i0 == 0 && u + kRaws < total) {
                if (mbar_wait(raw_free + 8 * (u % kRaws), (u / kRaws) & 1, kWaitIters))
                    fetch(u + kRaws);
                else
                    atomicOr(p.flag, kFlagTimeout);
            }
            __syncwarp();
        }
        // left early: no copy may still be on its way when the block ends
        if (i0 == 0)
            for (int v = u; v < min(u + kRaws, total); ++v) mbar_wait(raw_done + 8 * (v % kRaws), (v / kRaws) & 1, kDrainIters);
    } else if (threadIdx.x < kScorers + kSummers + kConverters + kLoaders) {
        // a warp for each stage.  A whole chunk's tiles come in boxes; the last rows of a
        // sequence, which the next one's may follow, row by row with zeros behind them.
        const int mine = warp - (kScorers + kSummers + kConverters) / 32, t = lane >> 3, c = lane & 7;
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
        bool ok = true;
        for (int it = mine; it < items; it += kStages) {
            if (it >= kStages && !(ok = tc::wait_warp(emptied + 8 * mine, it / kStages - 1, p.flag))) break;
            const int h = h0 + it / p.tiles, tile = it % p.tiles;
            const uint32_t sx = stages + mine * 2 * kX, b = loaded + 8 * mine;
            if (whole) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(b, 2 * kX);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        tc::box(sx + k * tc::kBox, &maps.x, h * p.P + tile * kTile, rg.first + k * 64, b);
                        tc::box(sx + kX + k * tc::kBox, &maps.dout, h * p.P + tile * kTile, rg.first + k * 64, b);
                    }
                }
                __syncwarp();
            } else {
                rows(sx, p.x + rg.first * p.xs + static_cast<long long>(h) * p.P + tile * kTile, p.xs);
                rows(sx + kX, p.dout + rg.first * os + static_cast<long long>(h) * p.P + tile * kTile, os);
                announce(b);
            }
        }
        if (mine < 2 && ok && tc::wait_warp(heads_done, 0, p.flag)) {
            if (whole) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(keys, kX);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        tc::box(sk + mine * kX + k * tc::kBox, mine ? &maps.Cm : &maps.Bm, group * p.N + n0, rg.first + k * 64, keys);
                }
                __syncwarp();
            } else {
                rows(sk + mine * kX, (mine ? p.Cm + rg.first * p.cs : p.Bm + rg.first * p.bs) + group * p.N + n0, mine ? p.cs : p.bs);
                announce(keys);
            }
        }
    } else {
        auto wait = [&](uint32_t b, int phase) { return tc::wait_warp(b, phase, p.flag); };
        bool ok = true;
        constexpr uint32_t id_w = tc::idesc(kChunk, false, false), id_t = tc::idesc(64, false, false);
        const uint64_t stage0 = tc::desc(stages, 16), unit0 = tc::desc(units, 16);
        int head = 0, tile = 0;
        for (int it = 0; it < items && ok; ++it) {
            if (!(ok = wait(loaded + 8 * (it % kStages), it / kStages))) break;
            if (tile == 0 && head >= 2 && !(ok = wait(w_free + 8 * (head & 1), head / 2 - 1))) break;
            tc::fence_after();
            const uint64_t xd = stage0 + (it % kStages) * (2 * kX >> 4), yd = xd + (kX >> 4);
            const uint32_t w = tmem + kW + (head & 1) * 128;
            const bool last = tile == p.tiles - 1;
            if (tc::elect()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) tc::mma(w, yd + ks * 2, xd + ks * 2, id_w, ks || tile);
                if (last) tc::commit(w_done + 8 * (head & 1));
            }
            __syncwarp();
            if (tile == 0 && head && !(ok = wait(t_free, head - 1))) break;
            for (int which = 0; which < 2 && ok; ++which) {
                const int u = 2 * it + which;
                if (!(ok = wait(unit_written + 8 * (u % kUnits), u / kUnits))) break;
                tc::fence_after();
                const uint64_t a = which ? xd : yd, b = unit0 + (u % kUnits) * (kUnit >> 4);
                if (tc::elect()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) tc::mma(tmem + kT + which * 64, a + ks * 2, b + ks * 2, id_t, ks || tile);
                    tc::commit(unit_free + 8 * (u % kUnits));
                }
                __syncwarp();
            }
            if (!ok) break;
            if (tc::elect()) {
                tc::commit(emptied + 8 * (it % kStages));
                if (last) tc::commit(t_done);
            }
            __syncwarp();
            tile = last ? 0 : tile + 1;
            head += last;
        }
        if (ok && tc::elect()) tc::commit(heads_done);
        __syncwarp();
        if (ok && (ok = wait(keys, 0) && wait(m_written, 0) && wait(t_free, heads - 1))) {
            tc::fence_after();
            constexpr uint32_t id_c = tc::idesc(64, false, true), id_b = tc::idesc(64, true, true);
            const uint64_t md = tc::desc(sm, 16), mt = tc::desc(sm, kX), kd = tc::desc(sk, 16);
            if (tc::elect()) {
#pragma unroll
                for (int ks = 0; ks < kChunk / 16; ++ks) tc::mma(tmem + kT, md + (((ks / 4) * kX + (ks % 4) * 32) >> 4), kd + ks * 128, id_c, ks);
#pragma unroll
                for (int ks = 0; ks < kChunk / 16; ++ks) tc::mma(tmem + kT + 64, mt + ks * 128, kd + ((kX + ks * 2048) >> 4), id_b, ks);
                tc::commit(f_done);
            }
            __syncwarp();
        }
        if (!ok) {  // left early: no box may still be on its way when the block ends
            for (int i = 0; i < kStages; ++i)
                for (int k = 0; k < 2; ++k) mbar_wait(loaded + 8 * i, k, kDrainIters);
            mbar_wait(keys, 0, kDrainIters);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 512);
}

}  // namespace

int launch_dk_tc(const Params& p, const tc::Maps& m, cudaStream_t s) {
    const int err = cudaFuncSetAttribute(dk_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err) return err;
    return launch(dk_tc_kernel, dim3(p.slots, p.G * (p.N / 64)), kBlock, kSmem, s, false, p, m);
}

}  // namespace scan
}  // namespace rsq
