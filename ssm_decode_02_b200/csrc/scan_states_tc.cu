// scan_states_tc.cu -- the states before the chunks on the fifth-generation tensor
// cores (tcgen05): the form of states_kernel (scan_forward.cu) for dk >= 64 and
// heads that fill 128 value columns.
//
// A block carries 128 value columns (two heads of 64, one of 128, half of one of
// 256) by up to 128 state rows through a sequence or segment.  Per chunk the product
// of the weighted values, 128 x tokens in three bf16 terms (split3), with the keys,
// tokens x N, is a tcgen05 product into one of two tensor-memory tiles.  Three kinds
// of warps, which meet at mbarriers only:
//   2 x 4 converters  have keys and values of half a chunk copied ahead (two stages
//                 each), weight the values and write their terms; the two groups take
//                 turns, so that the waits of one (copies, products, gates: three
//                 quarters of its time) pass while the other works;
//   8 updaters    hold the state, a thread half a column of N binary32; they store it
//                 as the state before the chunk and take in the chunk's tile while the
//                 next chunk's products run into the other;
//   1 issuer      of the products.
// Bound by instruction issue (split3 and the stores of three terms; 48% of the issue
// slots, 23% of the tensor cycles) and by 320 blocks on 148 SMs: 126 to 133 us for 8 x
// 2048 tokens, 80 heads of 128 x 64; 300 with all warps in step, 146 with one group of
// converters.  Blocks of half the size would leave as many rounds.
#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

constexpr int kHalf = 64;      // tokens of a step
constexpr int kCols = 128;     // value columns of a block
constexpr int kStages = 4;
constexpr int kConverters = 256, kUpdaters = 256, kBlock = kConverters + kUpdaters + 32;

template <int N>
struct Shape {
    static constexpr int kKeys = kHalf * N * 2;
    static constexpr int kValues = kHalf * kCols * 2;
    static constexpr int kStage = kKeys + kValues;
    static constexpr int kTerms = 3 * kValues;
    static constexpr int kSmem = 1024 + kStages * kStage + 2 * kTerms + 192;
};

template <int N, bool F32>
__global__ void __launch_bounds__(kBlock, 1) states_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ Pass fwd,
                                                               const __grid_constant__ Pass bwd,
                                                               const __grid_constant__ tc::Maps maps) {
    using Sh = Shape<N>;
    extern __shared__ uint8_t raw_smem[];
    wait_before();
    const Pass& ps = blockIdx.z ? bwd : fwd;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = p.N / N, cb = blockIdx.y / parts, row0 = (blockIdx.y - cb * parts) * N;  // first state row
    const int c0 = cb * kCols, h0 = c0 / p.P, heads = p.P >= kCols ? 1 : 2;
    const int group = h0 / p.per;
    int seq, lo, len, slot0, seg_first = 1, seg_last = 1;
    if (p.seg_chunks) {
        const Range r = slot_range(p, blockIdx.x, kChunk * p.seg_chunks);
        if (!r.valid && (p.steps || ps.local || r.index != 0)) return;   // of no rows, only a first one has a state to pass on
        seq = r.seq;
        lo = r.first;
        len = r.valid;
        slot0 = first_slot(p, seq, r.seq_first, kChunk) + r.index * p.seg_chunks;
        seg_first = r.index == 0;
        seg_last = lo + len == r.seq_first + r.seq_len;
    } else {
        seq = p.longs ? long_sequence(p, blockIdx.x) : static_cast<int>(blockIdx.x);
        if (seq < 0) return;
        sequence(p, seq, lo, len);
        if (p.steps && len <= p.steps) return;
        slot0 = first_slot(p, seq, lo, kChunk);
    }
    const int chunks = (len + kChunk - 1) / kChunk, steps = 2 * chunks;

    uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t base = smem_u32(smem);
    const uint32_t terms = base + kStages * Sh::kStage;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kStages * Sh::kStage + 2 * Sh::kTerms);
    // barriers, two of each: terms and keys written; their products done; a tile
    // complete; a tile taken in
    const uint32_t written = smem_u32(tmem_slot + 2), done = written + 16, full = done + 16, taken = full + 16,
                   arrived = taken + 16;  // and a stage's boxes, four
    if (warp == 0) tc::tmem_alloc(smem_u32(tmem_slot), 2 * N);
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(written + 8 * i, kConverters / 2);
            mbar_init(done + 8 * i, 1);
            mbar_init(full + 8 * i, 1);
            mbar_init(taken + 8 * i, kUpdaters);
        }
        for (int i = 0; i < kStages; ++i) mbar_init(arrived + 8 * i, 1);
        fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    auto chunk_of = [&](int s) { return ps.rev ? chunks - 1 - s / 2 : s / 2; };
    if (threadIdx.x < kConverters) {
        // this group's steps are those of its parity; this thread's chunks: rows t + 16 j,
        // columns 8 c.. of every 64 x 64 tile
        const int mine = warp >> 2, i0 = threadIdx.x & 127, t = i0 >> 3, c = i0 & 7;
        const uint32_t place = tile_at<128>(t, c);  // row t + 16 j: 2048 j bytes on
        const bf16* kp = ps.k + static_cast<long long>(group) * p.N + row0 + c * 8;
        const bf16* vp = ps.v + c0 + c * 8;
        const int h1 = heads - 1;                   // head of columns 64..127, from h0
        // a step of 64 rows comes in boxes that one thread asks for; the last rows of a
        // sequence, which the next one's may follow, chunk by chunk with zeros behind them
        const CUtensorMap *kmap = ps.rev ? &maps.Cm : &maps.Bm, *vmap = ps.rev ? &maps.dout : &maps.x;
        auto load = [&](int s) {
            if (s < steps) {
                const int row = chunk_of(s) * kChunk + (s & 1) * kHalf;
                const uint32_t to = base + (s % kStages) * Sh::kStage;
                const bool whole = row + kHalf <= len;
                if (i0 == 0) {
                    const uint32_t b = arrived + 8 * (s % kStages);
                    if (whole) {
                        mbar_arrive_expect_tx(b, Sh::kStage);
#pragma unroll
                        for (int k = 0; k < N / 64; ++k) tc::box(to + k * 8192, kmap, group * p.N + row0 + k * 64, lo + row, b);
#pragma unroll
                        for (int k = 0; k < 2; ++k) tc::box(to + Sh::kKeys + k * 8192, vmap, c0 + k * 64, lo + row, b);
                    } else {
                        mbar_arrive(b);
                    }
                }
#pragma unroll 1
                for (int j = 0; j < 4 && !whole; ++j) {
                    const bool on = row + t + 16 * j < len;
                    const long long at = lo + (on ? row + t + 16 * j : 0);
                    const bf16 *ksrc = kp + at * ps.ks, *vsrc = vp + at * ps.vs;
#pragma unroll
                    for (int b = 0; b < N / 64; ++b) cp16(to + place + j * 2048 + b * 8192, ksrc + b * 64, on);
#pragma unroll
                    for (int b = 0; b < 2; ++b) cp16(to + place + Sh::kKeys + j * 2048 + b * 8192, vsrc + b * 64, on);
                }
            }
            cp_commit();
        };
        // gates of the four rows for the two column tiles, read a step ahead
        float2 gb[2][4], ge[2];
        float gd[2][4];
        auto read_gates = [&](int s) {
            if (s >= steps) return;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const long long at = (static_cast<long long>(slot0 + chunk_of(s)) * p.H + h0 + b * h1) * kChunk;
                ge[b] = p.gb[at + kChunk - 1];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    gb[b][j] = p.gb[at + (s & 1) * kHalf + t + 16 * j];
                    gd[b][j] = p.gdt[at + (s & 1) * kHalf + t + 16 * j];
                }
            }
        };
        load(mine);
        read_gates(mine);
        int s = mine;
        for (; s < steps; s += 2) {
            float w[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[b][j] = ps.rev ? ex2(gb[b][j].x + gb[b][j].y) : ex2_diff(ge[b], gb[b][j]) * gd[b][j];
            read_gates(s + 2);
            // the products of step s - 2 are done with the terms' buffer and with the stage loaded next
            if (s >= 2 && !tc::wait_warp(done + 8 * mine, s / 2 - 1, p.flag)) break;
            load(s + 2);
            cp_wait<1>();
            if (!tc::wait_warp(arrived + 8 * (s % kStages), s / kStages, p.flag)) break;
            const uint32_t st = base + (s % kStages) * Sh::kStage + Sh::kKeys + place, tb = terms + mine * Sh::kTerms + place;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t o = b * 8192 + j * 2048;
                    uint32_t x[4], r[3][4];
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(st + o));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        split3(lo_of(x[k]) * w[b][j], hi_of(x[k]) * w[b][j], r[0][k], r[1][k], r[2][k]);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tb + k * Sh::kValues + o), "r"(r[k][0]),
                                     "r"(r[k][1]), "r"(r[k][2]), "r"(r[k][3])
                                     : "memory");
                }
            tc::fence_smem();
            mbar_arrive(written + 8 * mine);
        }
        cp_wait<0>();
        // left early: no box may still be on its way when the block ends
        if (i0 == 0)
            for (int k = s; k < min(s + 4, steps); k += 2) mbar_wait(arrived + 8 * (k % kStages), (k / kStages) & 1, kDrainIters);
    } else if (threadIdx.x < kConverters + kUpdaters) {
        // value column m (the tensor-memory lane), state rows n0 .. n0 + R - 1 of the block's
        constexpr int R = N / 2;
        const int uw = warp - kConverters / 32, m = (uw & 3) * 32 + lane, n0 = (uw >> 2) * R;
        const int h = h0 + m / p.P, pc = (c0 + m) % p.P;   // its head and column of the head
        const long long head_cells = static_cast<long long>(p.N) * p.P, cell0 = static_cast<long long>(row0 + n0) * p.P + pc;
        const float* init = ps.init;
        long long at0 = (static_cast<long long>(seq) * p.H + h) * head_cells + cell0;
        const long long seg_at = (static_cast<long long>(blockIdx.x) * p.H + h) * head_cells + cell0;
        float S[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float* src = ps.local ? nullptr : (p.seg_chunks ? p.seg_start[ps.rev] + seg_at : (init ? init + at0 : nullptr));
            S[i] = src ? src[static_cast<long long>(i) * p.P] : 0.f;
        }
        const long long gate_at = (static_cast<long long>(slot0) * p.H + h) * kChunk + kChunk - 1;
        bool ok = true;
        for (int i = 0; i < chunks && ok; ++i) {
            const int c = chunk_of(2 * i);
            const float2 end = p.gb[gate_at + static_cast<long long>(c) * p.H * kChunk];
            if (!ps.local) {
                const long long cell = ((static_cast<long long>(slot0 + c) * p.H + h) * p.tiles + pc / kTile) * p.N * kTile +
                                       static_cast<long long>(row0 + n0) * kTile + pc % kTile;
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    if constexpr (F32)
                        (ps.rev ? p.df : p.sf)[cell + k * kTile] = S[k];
                    else
                        p.sh[cell + k * kTile] = __float2bfloat16_rn(S[k]);   // an operand for out alone (scan.cuh, Roundings)
                }
            }
            const float a = ex2(end.x + end.y);
            if (!(ok = tc::wait_warp(full + 8 * (i & 1), i / 2, p.flag))) break;
            tc::fence_after();
            const uint32_t d = tmem + (i & 1) * N + n0 + ((static_cast<uint32_t>(warp) & 3) << 21);
#pragma unroll
            for (int b = 0; b < R / 16; ++b) {
                float v[16];
                tc::tmem_ld16(v, d + b * 16);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) S[b * 16 + k] = fmaf(a, S[b * 16 + k], v[k]);
            }
            tc::fence_before();
            mbar_arrive(taken + 8 * (i & 1));
        }
        float* end = ps.local ? p.seg_end[ps.rev] : ((ps.rev ? seg_first : seg_last) ? ps.end : nullptr);
        if (ps.local && !ps.rev && uw == 0 && lane < heads && row0 == 0 && c0 % p.P == 0) {
            double log = 0.;
            for (int c = 0; c < chunks; ++c) {
                const float2 e = p.gb[(static_cast<long long>(slot0 + c) * p.H + h0 + lane) * kChunk + kChunk - 1];
                log += static_cast<double>(e.x) + static_cast<double>(e.y);
            }
            p.seg_log[static_cast<long long>(blockIdx.x) * p.H + h0 + lane] = log;
        }
        if (end && ok) {
#pragma unroll
            for (int i = 0; i < R; ++i) end[(ps.local ? seg_at : at0) + static_cast<long long>(i) * p.P] = S[i];
        }
    } else {
        constexpr uint32_t id = tc::idesc(N, true, true);
        const uint64_t keys0 = tc::desc(base, 8192), terms0 = tc::desc(terms, 8192);
        for (int s = 0; s < steps; ++s) {
            if (!tc::wait_warp(written + 8 * (s & 1), s / 2, p.flag)) break;
            if (!(s & 1) && s >= 4 && !tc::wait_warp(taken + 8 * ((s / 2) & 1), s / 4 - 1, p.flag)) break;
            tc::fence_after();
            const uint64_t kd = keys0 + (s % kStages) * (Sh::kStage >> 4), td = terms0 + (s & 1) * (Sh::kTerms >> 4);
            const uint32_t d = tmem + ((s / 2) & 1) * N;
            if (tc::elect()) {
#pragma unroll
                for (int ks = 0; ks < kHalf / 16; ++ks)
#pragma unroll
                    for (int k = 2; k >= 0; --k) {
                        const uint64_t ad = td + ((k * Sh::kValues + ks * 2048) >> 4), bd = kd + ks * 128;
                        if (ks == 0 && k == 2)
                            tc::mma(d, ad, bd, id, s & 1);
                        else
                            tc::mma(d, ad, bd, id, true);
                    }
                tc::commit(done + 8 * (s & 1));
                if (s & 1) tc::commit(full + 8 * ((s / 2) & 1));
            }
            __syncwarp();
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 2 * N);
}

template <int N>
int run(const Params& p, const tc::Maps& m, bool backward, const Pass& f, const Pass& b, cudaStream_t s) {
    auto* k = backward ? states_tc_kernel<N, true> : states_tc_kernel<N, false>;
    const int err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<N>::kSmem);
    if (err) return err;
    const dim3 grid(p.seg_chunks ? p.seg_slots : (p.longs ? p.longs : p.n), p.H * p.P / kCols * (p.N / N), backward ? 2 : 1);
    return launch(k, grid, kBlock, Shape<N>::kSmem, s, !p.slots, p, f, b, m);
}

}  // namespace

int launch_states_tc(const Params& p, const tc::Maps& m, bool backward, const Pass& f, const Pass& b, cudaStream_t s) {
    return p.N == 64 ? run<64>(p, m, backward, f, b, s) : run<128>(p, m, backward, f, b, s);
}

}  // namespace scan
}  // namespace rsq
