// scan_out_tc.cu -- the scan's outputs on the fifth-generation tensor cores
// (tcgen05): the form of out_kernel (scan_forward.cu) for dk of 64 and 128 and heads
// of whole 64-column tiles.
//
// A block takes units of one chunk and some heads of one group, one after the other
// (one block per SM).  The scores C_i.B_j, which do
// not depend on the head, are one product whose 128 x 128 result stays in the
// registers of the scorers; per tile of 64 columns of a head
//     inter = C S_0 (keys' rows from shared memory)       128 x 64, k = N
//     intra = (scores . decays . dt) x                    128 x 64, k = tokens
//     out   = 2^b_i inter + intra + D x
// with the left operand of `intra` in tensor memory, where the scorers write it.
// Warps, which meet at mbarriers only:
//   16 scorers    a warp 32 rows by 32 columns of the scores; per head they make the
//                 decays and write the bf16 left operand (two buffers);
//   2 x 4 writers every other tile: a thread one row of 64 columns; the output goes
//                 over x in shared memory and from there to memory in whole lines;
//   2 loaders     x and the state of each tile, and the next unit's keys;
//   1 issuer      of the products, the next unit's scores among them.
// The decay between a row and a column is the product of two powers that meet at the
// border between their blocks of 32 tokens (at most 1 each where decays are): two
// powers per lane and head in the place of 32.  On the diagonal they meet at the
// block's start and one of them grows with the decay over it, so that a block which
// decays by more than 2^100 takes a power per pair.
//
// Bound by instruction issue and the latency between the roles (46% of the issue slots,
// 15% of the tensor cycles, 0.5 GB of DRAM traffic): 8 x 2048 tokens, 80 heads of 128 x
// 64, 150 us; 157 with a block per unit, 290 with 8 scorers and a power per pair.
// 16-token blocks on the diagonal, and tiles brought to L2 ahead, were slower.
#include <algorithm>

#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

constexpr int kScorers = 512, kWriters = 256, kLoaders = 64;
constexpr int kBlock = kScorers + kWriters + kLoaders + 32;
constexpr int kTmem = 512;                                  // scores, 2 x (inter, intra), 2 x left operand
constexpr int kD = 128, kLeft = 384;

template <int N>
struct Shape {
    static constexpr int kStages = N == 64 ? 4 : 2;
    static constexpr int kKeys = kChunk * N * 2;            // of B or C; two of both
    static constexpr int kX = kChunk * kTile * 2;
    static constexpr int kStage = kX + N * kTile * 2;
    static constexpr int kGates = 16 * 32 * (4 + 16);       // per scorer warp: factors; b in two floats, dt
    static constexpr int kSmem = 1024 + 4 * kKeys + kStages * kStage + kGates + 256;
};

// One chunk and some heads of one group.
struct Unit {
    int slot, first, valid, group, h0, heads;
};

template <int N>
__global__ void __launch_bounds__(kBlock, 1) out_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ tc::Maps maps,
                                                            int head_set, int unit_count) {
    using Sh = Shape<N>;
    constexpr int kStages = Sh::kStages;
    extern __shared__ uint8_t raw_smem[];
    const int sets = (p.per + head_set - 1) / head_set;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the block's units, by every role in the same order; slots without rows are left out
    auto unit_at = [&](int u, Unit& o) {
        const int per_slot = p.G * sets, y = u % per_slot;
        o.slot = u / per_slot;
        const Rows rg = slot_rows(p, o.slot);
        o.first = rg.first;
        o.valid = rg.valid;
        o.group = y / sets;
        const int set = y - o.group * sets;
        o.h0 = o.group * p.per + set * head_set;
        o.heads = min(head_set, p.per - set * head_set);
        return rg.valid != 0;
    };

    uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t keys0 = smem_u32(smem), stages = keys0 + 4 * Sh::kKeys;   // C, B of a unit; of the next
    uint8_t* gates = smem + 4 * Sh::kKeys + kStages * Sh::kStage;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gates + Sh::kGates);
    // barriers: keys loaded x2, free x2; scores done, read; stage loaded x4, free x4; left
    // operand written x2, free x2; tile done x2, free x2
    const uint32_t keys = smem_u32(tmem_slot + 2), keys_free = keys + 16, scores = keys_free + 16, scores_read = scores + 8,
                   loaded = scores_read + 8, emptied = loaded + 32, left = emptied + 32, left_free = left + 16,
                   tile_done = left_free + 16, tile_free = tile_done + 16;
    if (warp == 0) tc::tmem_alloc(smem_u32(tmem_slot), kTmem);
    if (threadIdx.x == 0) {
        mbar_init(scores, 1);
        mbar_init(scores_read, kScorers);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(loaded + 8 * i, 1);
            mbar_init(emptied + 8 * i, 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(keys + 8 * i, 1);
            mbar_init(keys_free + 8 * i, 1);
            mbar_init(left + 8 * i, kScorers);
            mbar_init(left_free + 8 * i, 1);
            mbar_init(tile_done + 8 * i, 1);
            mbar_init(tile_free + 8 * i, 128);
        }
        fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    wait_before();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lanes = (static_cast<uint32_t>(warp) & 3) << 21;

    if (threadIdx.x < kScorers) {
        const int quarter = warp & 3, cols = warp >> 2, row = quarter * 32 + lane;   // rows 32 quarter .., columns 32 cols ..
        float* fac = reinterpret_cast<float*>(gates) + warp * 32;
        float4* pair = reinterpret_cast<float4*>(gates + 16 * 32 * 4) + warp * 32;
        const bool diagonal = cols == quarter;
        bool ok = true;
        int gh = 0, gu = 0;   // heads and units so far
        Unit un;
        for (int u = blockIdx.x; u < unit_count && ok; u += gridDim.x) {
            if (!unit_at(u, un)) continue;
            const long long at0 = (static_cast<long long>(un.slot) * p.H + un.h0) * kChunk;
            float2 nc = make_float2(0.f, 0.f), nr = nc;
            float nd = 0.f;
            auto read = [&](int i) {
                if (i >= un.heads || cols > quarter) return;
                const long long at = at0 + static_cast<long long>(i) * kChunk;
                nc = p.gb[at + cols * 32 + lane];
                nd = p.gdt[at + cols * 32 + lane];
                nr = p.gb[at + row];
            };
            read(0);
            if (!(ok = tc::wait_warp(scores, gu, p.flag))) break;
            ++gu;
            tc::fence_after();
            float g[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v[16];
                tc::tmem_ld16(v, tmem + cols * 32 + i * 16 + lanes);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) g[i * 16 + k] = v[k];
            }
            tc::fence_before();
            mbar_arrive(scores_read);
            for (int i = 0; i < un.heads; ++i, ++gh) {
                const int buf = gh & 1;
                const float2 bc = nc, br = nr;
                const float dt = nd;
                read(i + 1);
                if (gh >= 2 && !(ok = tc::wait_warp(left_free + 8 * buf, gh / 2 - 1, p.flag))) break;
                tc::fence_after();
                const uint32_t dst = tmem + kLeft + buf * 64 + cols * 16 + lanes;
                if (cols > quarter) {           // behind every row: zero, once for each buffer
                    if (gh < 2) {
                        const uint32_t z[16] = {};
                        tc::tmem_st16(dst, z);
                    }
                } else {
                    const int meet = diagonal ? 0 : 31;
                    const float2 bm = make_float2(__shfl_sync(0xffffffffu, bc.x, meet), __shfl_sync(0xffffffffu, bc.y, meet));
                    const float last = __shfl_sync(0xffffffffu, bc.x, 31);
                    __syncwarp();
                    fac[lane] = dt * ex2_diff(bm, bc);
                    const float r = ex2_diff(br, bm);
                    const bool direct = diagonal && !(bm.x - last < 100.f);
                    if (direct) pair[lane] = make_float4(bc.x, bc.y, dt, 0.f);
                    __syncwarp();
                    uint32_t w[16];
                    if (!direct) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 f = reinterpret_cast<const float4*>(fac)[k];
                            float v[4] = {g[4 * k] * (r * f.x), g[4 * k + 1] * (r * f.y), g[4 * k + 2] * (r * f.z), g[4 * k + 3] * (r * f.w)};
                            if (diagonal) {
#pragma unroll
                                for (int o = 0; o < 4; ++o) v[o] = 4 * k + o <= lane ? v[o] : 0.f;
                            }
                            w[2 * k] = pack(v[0], v[1]);
                            w[2 * k + 1] = pack(v[2], v[3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float v[2];
#pragma unroll
                            for (int o = 0; o < 2; ++o) {
                                const float4 q = pair[2 * k + o];
                                v[o] = 2 * k + o <= lane ? g[2 * k + o] * (ex2_diff(br, make_float2(q.x, q.y)) * q.z) : 0.f;
                            }
                            w[k] = pack(v[0], v[1]);
                        }
                    }
                    tc::tmem_st16(dst, w);
                }
                tc::tmem_st_wait();
                tc::fence_before();
                mbar_arrive(left + 8 * buf);
            }
        }
    } else if (threadIdx.x < kScorers + kWriters) {
        const int ww = warp - kScorers / 32, wg = ww >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const long long os = static_cast<long long>(p.H) * p.P;
        float2 nb = make_float2(0.f, 0.f);
        float nd = 0.f;
        bool ok = true;
        int gi = 0;   // tiles so far
        Unit un;
        for (int u = blockIdx.x; u < unit_count && ok; u += gridDim.x) {
            if (!unit_at(u, un)) continue;
            const int items = un.heads * p.tiles;
            auto read = [&](int it) {
                if (it >= items) return;
                const int h = un.h0 + it / p.tiles;
                nb = p.gb[(static_cast<long long>(un.slot) * p.H + h) * kChunk + row];
                if (p.D) nd = __ldg(p.D + h);
            };
            const int it0 = (wg ^ gi) & 1;   // the writers take turns over all units
            read(it0);
            for (int it = it0; it < items; it += 2) {
                const int g = gi + it, stage = g % kStages;
                const int h = un.h0 + it / p.tiles, tile = it % p.tiles;
                const float d = nd, e = ex2(nb.x + nb.y);
                read(it + 2);
                const uint32_t st = stages + stage * Sh::kStage;
                if (!(ok = tc::wait_warp(tile_done + 8 * wg, g / 2, p.flag))) break;
                tc::fence_after();
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    float a[16], v[16];
                    tc::tmem_ld16(a, tmem + kD + wg * 128 + s * 16 + lanes);
                    tc::tmem_ld16(v, tmem + kD + wg * 128 + 64 + s * 16 + lanes);
                    tc::tmem_ld_wait();
                    if (s == 3) {
                        tc::fence_before();
                        mbar_arrive(tile_free + 8 * wg);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t ad = st + tile_at<128>(row, s * 2 + k);
                        uint32_t x[4], o[4];
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(ad) : "memory");
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = k * 8 + 2 * i;
                            o[i] = pack(fmaf(d, lo_of(x[i]), fmaf(e, a[c], v[c])), fmaf(d, hi_of(x[i]), fmaf(e, a[c + 1], v[c + 1])));
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(ad), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
                    }
                }
                __syncwarp();
                // this warp's 32 rows, four whole rows at a time
                bf16* out = p.out + static_cast<long long>(un.first) * os + static_cast<long long>(h) * p.P + tile * kTile;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = quarter * 32 + k * 4 + (lane >> 3);
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(st + tile_at<128>(r, lane & 7)) : "memory");
                    if (r < un.valid) *reinterpret_cast<uint4*>(out + r * os + (lane & 7) * 8) = v;
                }
                tc::fence_smem();   // boxes overwrite what was written here
                mbar_arrive(emptied + 8 * stage);
            }
            gi += items;
        }
    } else if (threadIdx.x < kScorers + kWriters + kLoaders) {
        // a whole chunk's tiles come in boxes; the last rows of a sequence, which the next
        // one's may follow, row by row with zeros behind them.  One warp loads the keys and
        // every other tile, the other warp the other tiles.
        const int mine = warp & 1, t = lane >> 3, c = lane & 7;
        auto rows = [&](uint32_t dst, const bf16* src, long long stride, int n, int on_rows) {
#pragma unroll 4
            for (int j = 0; j < n / 4; ++j) {
                const bool on = t + 4 * j < on_rows;
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
        int gi = 0, gu = 0;
        auto load_keys = [&](const Unit& un) {
            const int buf = gu & 1;
            const uint32_t sc = keys0 + buf * 2 * Sh::kKeys, sb = sc + Sh::kKeys, bar = keys + 8 * buf;
            if (gu >= 2 && !(ok = tc::wait_warp(keys_free + 8 * buf, gu / 2 - 1, p.flag))) return;
            ++gu;
            if (un.valid == kChunk) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, 2 * Sh::kKeys);
#pragma unroll
                    for (int b = 0; b < N / 64; ++b)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            tc::box(sc + b * kChunk * 128 + k * tc::kBox, &maps.Cm, un.group * N + b * 64, un.first + k * 64, bar);
                            tc::box(sb + b * kChunk * 128 + k * tc::kBox, &maps.Bm, un.group * N + b * 64, un.first + k * 64, bar);
                        }
                }
                __syncwarp();
            } else {
#pragma unroll 1
                for (int b = 0; b < N / 64; ++b) {
                    rows(sc + b * kChunk * 128, p.Cm + un.first * p.cs + un.group * N + b * 64, p.cs, kChunk, un.valid);
                    rows(sb + b * kChunk * 128, p.Bm + un.first * p.bs + un.group * N + b * 64, p.bs, kChunk, un.valid);
                }
                announce(bar);
            }
        };
        Unit un, ahead;
        int next = blockIdx.x;   // the next unit whose keys come
        auto keys_ahead = [&] {
            while (ok && next < unit_count) {
                const bool any = unit_at(next, ahead);
                next += gridDim.x;
                if (any) {
                    load_keys(ahead);
                    return;
                }
            }
        };
        if (mine == 0) keys_ahead();
        for (int u = blockIdx.x; u < unit_count && ok; u += gridDim.x) {
            if (!unit_at(u, un)) continue;
            const int items = un.heads * p.tiles;
            const bool whole = un.valid == kChunk;
            for (int it = 0; it < items; ++it) {
                const int g = gi + it, stage = g % kStages;
                // the next unit's keys with this one's last tile: room for them came with its first
                if (mine == 0 && it == items - 1) keys_ahead();
                if ((g & 1) != mine) continue;
                if (!ok) break;
                const int h = un.h0 + it / p.tiles, tile = it % p.tiles;
                const uint32_t st = stages + stage * Sh::kStage, b = loaded + 8 * stage;
                if (g >= kStages && !(ok = tc::wait_warp(emptied + 8 * stage, g / kStages - 1, p.flag))) break;
                const long long cell = (static_cast<long long>(un.slot) * p.H + h) * p.tiles + tile;
                if (whole) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(b, Sh::kStage);
#pragma unroll
                        for (int k = 0; k < 2; ++k) tc::box(st + k * tc::kBox, &maps.x, h * p.P + tile * kTile, un.first + k * 64, b);
#pragma unroll
                        for (int k = 0; k < N / 64; ++k) tc::box(st + Sh::kX + k * tc::kBox, &maps.sh, 0, static_cast<int>(cell * N) + k * 64, b);
                    }
                    __syncwarp();
                } else {
                    rows(st, p.x + un.first * p.xs + static_cast<long long>(h) * p.P + tile * kTile, p.xs, kChunk, un.valid);
                    rows(st + Sh::kX, p.sh + cell * N * kTile, kTile, N, N);
                    announce(b);
                }
            }
            gi += items;
        }
    } else {
        bool ok = true;
        const uint64_t stage0 = tc::desc(stages, 16);
        constexpr uint32_t id_g = tc::idesc(kChunk, false, false), id = tc::idesc(kTile, false, true);
        int gi = 0, gh = 0, gu = 0, issued = 0;   // tiles, heads, units; units whose scores are issued
        auto issue_scores = [&] {
            const int buf = issued & 1;
            if (!(ok = tc::wait_warp(keys + 8 * buf, issued / 2, p.flag))) return;
            if (issued && !(ok = tc::wait_warp(scores_read, issued - 1, p.flag))) return;
            tc::fence_after();
            const uint64_t cd = tc::desc(keys0 + buf * 2 * Sh::kKeys, 16), bd = cd + (Sh::kKeys >> 4);
            if (tc::elect()) {
#pragma unroll
                for (int ks = 0; ks < N / 16; ++ks) {
                    const uint32_t o = ((ks / 4) * kChunk * 128 + (ks % 4) * 32) >> 4;
                    tc::mma(tmem, cd + o, bd + o, id_g, ks);
                }
                tc::commit(scores);
            }
            __syncwarp();
            ++issued;
        };
        Unit un, ahead;
        int next = blockIdx.x;
        auto scores_ahead = [&] {
            while (ok && next < unit_count) {
                const bool any = unit_at(next, ahead);
                next += gridDim.x;
                if (any) {
                    issue_scores();
                    return;
                }
            }
        };
        scores_ahead();
        for (int u = blockIdx.x; u < unit_count && ok; u += gridDim.x) {
            if (!unit_at(u, un)) continue;
            const int items = un.heads * p.tiles;
            const uint64_t cd = tc::desc(keys0 + (gu & 1) * 2 * Sh::kKeys, 16);
            int tile = 0;
            for (int it = 0; it < items && ok; ++it, ++gi) {
                const int buf = gh & 1, stage = gi % kStages;
                const uint64_t sd = stage0 + stage * (Sh::kStage >> 4);
                const uint32_t d = tmem + kD + (gi & 1) * 128;
                if (!(ok = tc::wait_warp(loaded + 8 * stage, gi / kStages, p.flag))) break;
                if (gi >= 2 && !(ok = tc::wait_warp(tile_free + 8 * (gi & 1), gi / 2 - 1, p.flag))) break;
                tc::fence_after();
                if (tc::elect()) {
#pragma unroll
                    for (int ks = 0; ks < N / 16; ++ks)
                        tc::mma(d, cd + (((ks / 4) * kChunk * 128 + (ks % 4) * 32) >> 4), sd + ((Sh::kX + ks * 2048) >> 4), id, ks);
                    if (it == items - 1) tc::commit(keys_free + 8 * (gu & 1));   // the unit's last use of its keys
                }
                __syncwarp();
                // the next unit's scores, so that they are there when its first head is turned to
                if (it == items - 1) scores_ahead();
                if (!ok) break;
                if (tile == 0) {
                    if (!(ok = tc::wait_warp(left + 8 * buf, gh / 2, p.flag))) break;
                    tc::fence_after();
                }
                const bool last = tile == p.tiles - 1;
                if (tc::elect()) {
#pragma unroll
                    for (int ks = 0; ks < kChunk / 16; ++ks) tc::mma_ta(d + 64, tmem + kLeft + buf * 64 + ks * 8, sd + ks * 128, id, ks);
                    tc::commit(tile_done + 8 * (gi & 1));
                    if (last) tc::commit(left_free + 8 * buf);
                }
                __syncwarp();
                tile = last ? 0 : tile + 1;
                gh += last;
            }
            ++gu;
        }
        if (!ok) {  // left early: no box may still be on its way when the block ends
            for (int k = 0; k < 2; ++k) {
                for (int i = 0; i < kStages; ++i) mbar_wait(loaded + 8 * i, k, kDrainIters);
                for (int i = 0; i < 2; ++i) mbar_wait(keys + 8 * i, k, kDrainIters);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, kTmem);
}

template <int N>
int run(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    const int err = cudaFuncSetAttribute(out_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<N>::kSmem);
    if (err) return err;
    const long long units = static_cast<long long>(p.slots) * p.G * ((p.per + head_set - 1) / head_set);
    if (units > 2000000000) return cudaErrorInvalidConfiguration;
    return launch(out_tc_kernel<N>, static_cast<unsigned>(std::min<long long>(units, kSms)), kBlock, Shape<N>::kSmem, s, false, p, m, head_set,
                  static_cast<int>(units));
}

}  // namespace

int launch_out_tc(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    return p.N == 64 ? run<64>(p, m, head_set, s) : run<128>(p, m, head_set, s);
}

}  // namespace scan
}  // namespace rsq
