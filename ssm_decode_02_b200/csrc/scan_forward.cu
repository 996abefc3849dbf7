// scan_forward.cu -- the scan's gates, states and outputs (sm_100a); the backward
// pass uses the first two as well.
#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

// ---------------------------------------------------------------------------
// Gates: b_i = sum of log2 a_t up to token i of its chunk, a warp per (chunk,
// head).  The sum is binary64 and stays as two floats: differences of two such
// sums, which become the decays between tokens, keep binary32 accuracy behind
// strong decays and behind a decay of zero.  Rows past the end of the sequence
// have a_t = 1 and dt = 0.  Bound by latency and by what it writes: 11 us for 16384
// tokens and 80 heads (21 MB).
// ---------------------------------------------------------------------------
constexpr int kGateHeads = kThreads / 32;   // of a block

__global__ void __launch_bounds__(kThreads) gates_kernel(const __grid_constant__ Params p) {
    let_next();
    // the heads' values of a token lie side by side: read so, and turned here
    __shared__ __align__(16) float sdt[kGateHeads][kChunk + 4], sa[kGateHeads][kChunk + 4];
    const int slot = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.flag = 0u;
    const int h0 = blockIdx.y * kGateHeads, h = h0 + warp;
    const Range r = slot_range(p, slot, kChunk);
    if (blockIdx.y == 0 && threadIdx.x == 0) p.rows[slot] = make_int2(r.first, r.valid);
    if (!r.valid) return;
#pragma unroll
    for (int i = threadIdx.x; i < kChunk * kGateHeads; i += kThreads) {
        const int t = i / kGateHeads, k = i % kGateHeads;
        if (t < r.valid && h0 + k < p.H) {
            const long long at = static_cast<long long>(r.first + t) * p.H + h0 + k;
            if (p.dt) sdt[k][t] = __ldg(p.dt + at);
            if (p.decay) sa[k][t] = __ldg(p.decay + at);
        }
    }
    __syncthreads();
    if (h >= p.H) return;
    double b[4];
    float dt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = lane * 4 + i;
        b[i] = 0.;
        dt[i] = 0.f;
        if (t < r.valid) {
            dt[i] = p.dt ? sdt[warp][t] : 1.f;
            if (p.decay) {
                const float a = sa[warp][t];
                b[i] = a == 0.f ? kLogZero : static_cast<double>(log2f(a));
            } else {
                b[i] = static_cast<double>(dt[i]) * static_cast<double>(__ldg(p.A + h)) * 1.4426950408889634;
            }
            if (b[i] < kLogZero) b[i] = kLogZero;
        }
        if (i) b[i] += b[i - 1];
    }
    double before = b[3];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    before -= b[3];
    const long long at = (static_cast<long long>(slot) * p.H + h) * kChunk + lane * 4;
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double s = before + b[i];
        v[i].x = static_cast<float>(s);
        v[i].y = static_cast<float>(s - static_cast<double>(v[i].x));
    }
    *reinterpret_cast<float4*>(p.gb + at) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    *reinterpret_cast<float4*>(p.gb + at + 2) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    *reinterpret_cast<float4*>(p.gdt + at) = make_float4(dt[0], dt[1], dt[2], dt[3]);
}

// ---------------------------------------------------------------------------
// States.  A block carries one tile of 64 state columns of one head through a
// sequence (or a segment of it) in the matrix products' accumulators, N x 64
// binary32 over eight warps: before each chunk it stores the tile for the
// chunk's other kernels, scales it by the chunk's decay and adds the chunk's
// product.  The weights 2^(b_end-b_j) dt_j go on the key operand, in three bf16
// terms (scan.cuh, split3): the state stays accurate to binary32.
// The backward recurrence is the same with (C, dout, 2^b_i) for (B, x, weights)
// and the chunks in reverse.  Bound by the issue of split3 and of the warp products:
// 292 us for 8 x 2048 tokens, 80 heads of 128 x 64, where scan_states_tc.cu, which has
// the shapes from dk = 64 on, takes 126 to 133.
// ---------------------------------------------------------------------------
template <int N>
struct StateShape {
    static constexpr int kRows = N >= 128 ? N / 128 : 1;    // 16-row blocks of a warp
    static constexpr int kCols = N >= 128 ? 8 : N / 16;     // 8-column blocks of a warp
    static constexpr int kRowBlocks = N / 16;
    static constexpr int kStage = 64 * N * 2 + 64 * kTile * 2;
    static constexpr int kSmem = 2 * kStage + 2 * 64 * 4;
};

template <int N, bool F32>
__global__ void __launch_bounds__(kThreads) states_kernel(const __grid_constant__ Params p,
                                                          const __grid_constant__ Pass fwd,
                                                          const __grid_constant__ Pass bwd) {
    using Sh = StateShape<N>;
    extern __shared__ __align__(128) uint8_t smem[];
    wait_before();
    const Pass& ps = blockIdx.z ? bwd : fwd;
    const int h = blockIdx.y / p.tiles, tile = blockIdx.y - h * p.tiles;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int group = h / p.per;

    // the rows: a whole sequence, or one segment of it
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
    const int chunks = (len + kChunk - 1) / kChunk;
    const int cols = min(kTile, p.P - tile * kTile);

    float* wgt = reinterpret_cast<float*>(smem + 2 * Sh::kStage);  // [2][64]
    const uint32_t base = smem_u32(smem);
    const bf16* kp = ps.k + static_cast<long long>(group) * N;
    const bf16* vp = ps.v + static_cast<long long>(h) * p.P + tile * kTile;

    const int rb0 = warp % Sh::kRowBlocks;                       // first row block
    const int cb0 = N >= 128 ? 0 : (warp / Sh::kRowBlocks) * Sh::kCols;  // first column block
    float acc[Sh::kRows][Sh::kCols][4];

    // the state at the start: the segment's from the workspace, else the caller's, else zero
    const float* init = ps.init;
    long long init_at = (static_cast<long long>(seq) * p.H + h) * N * p.P;
    if (p.seg_chunks && !ps.local) {
        init = p.seg_start[ps.rev];
        init_at = (static_cast<long long>(blockIdx.x) * p.H + h) * N * p.P;
    }
    if (ps.local) init = nullptr;
    auto place = [&](int r, int c, int e) {  // row and column of an accumulator pair (e = 0, 2)
        return make_int2((rb0 + 8 * r) * 16 + g + (e ? 8 : 0), (cb0 + c) * 8 + 2 * q);
    };
#pragma unroll
    for (int r = 0; r < Sh::kRows; ++r)
#pragma unroll
        for (int c = 0; c < Sh::kCols; ++c)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int2 at = place(r, c, e);
                float2 v = make_float2(0.f, 0.f);
                if (init && at.y < cols)
                    v = *reinterpret_cast<const float2*>(init + init_at + static_cast<long long>(at.x) * p.P + tile * kTile + at.y);
                acc[r][c][e] = v.x;
                acc[r][c][e + 1] = v.y;
            }

    const int steps = 2 * chunks;  // half chunks of 64 rows
    auto chunk_of = [&](int s) { return ps.rev ? chunks - 1 - s / 2 : s / 2; };
    auto load = [&](int s) {
        if (s < steps) {
            const int row = chunk_of(s) * kChunk + (s & 1) * 64;
            const int valid = max(0, min(64, len - row));
            const uint32_t st = base + (s & 1) * Sh::kStage;
            const long long first = lo + (valid ? row : 0);
            load_tile<2 * N, 64>(st, kp + first * ps.ks, ps.ks, valid, N / 8);
            load_tile<2 * kTile, 64>(st + 64 * N * 2, vp + first * ps.vs, ps.vs, valid, cols / 8);
            const long long at = (static_cast<long long>(slot0 + chunk_of(s)) * p.H + h) * kChunk;
            if (threadIdx.x < 64) {
                const int t = (s & 1) * 64 + threadIdx.x;
                const float2 b = p.gb[at + t], end = p.gb[at + kChunk - 1];
                wgt[(s & 1) * 64 + threadIdx.x] = ps.rev ? ex2(b.x + b.y) : ex2_diff(end, b) * p.gdt[at + t];
            }
        }
        cp_commit();
    };
    load(0);
    load(1);
    for (int s = 0; s < steps; ++s) {
        const int c = chunk_of(s);
        if (!(s & 1)) {
            const long long cell = (static_cast<long long>(slot0 + c) * p.H + h) * p.tiles + tile;
            const float2 end = p.gb[(static_cast<long long>(slot0 + c) * p.H + h) * kChunk + kChunk - 1];
            const float a = ex2(end.x + end.y);
#pragma unroll
            for (int r = 0; r < Sh::kRows; ++r)
#pragma unroll
                for (int k = 0; k < Sh::kCols; ++k)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        if (!ps.local) {
                            const int2 at = place(r, k, e);
                            const long long o = (cell * N + at.x) * kTile + at.y;
                            if constexpr (F32)
                                *reinterpret_cast<float2*>((ps.rev ? p.df : p.sf) + o) = make_float2(acc[r][k][e], acc[r][k][e + 1]);
                            else
                                *reinterpret_cast<uint32_t*>(p.sh + o) = pack(acc[r][k][e], acc[r][k][e + 1]);
                        }
                        acc[r][k][e] *= a;
                        acc[r][k][e + 1] *= a;
                    }
        }
        cp_wait<1>();
        __syncthreads();
        const uint32_t st = base + (s & 1) * Sh::kStage;
        const int valid = max(0, min(64, len - (c * kChunk + (s & 1) * 64)));
        const float* w = wgt + (s & 1) * 64;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (ks * 16 >= valid) break;
            const float w0 = w[ks * 16 + 2 * q], w1 = w[ks * 16 + 2 * q + 1];
            const float w8 = w[ks * 16 + 2 * q + 8], w9 = w[ks * 16 + 2 * q + 9];
            uint32_t vb[(Sh::kCols + 1) / 2][4];
#pragma unroll
            for (int c2 = 0; c2 < (Sh::kCols + 1) / 2; ++c2) frag_bt<2 * kTile>(vb[c2], st + 64 * N * 2, (cb0 & ~1) * 8 + c2 * 16, ks, lane);
#pragma unroll
            for (int r = 0; r < Sh::kRows; ++r) {
                uint32_t a[4], t[3][4];
                frag_at<2 * N>(a, st, (rb0 + 8 * r) * 16, ks, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    split3(lo_of(a[i]) * (i < 2 ? w0 : w8), hi_of(a[i]) * (i < 2 ? w1 : w9), t[0][i], t[1][i], t[2][i]);
#pragma unroll
                for (int k = 0; k < Sh::kCols; ++k) {
                    const int odd = Sh::kCols == 1 ? (cb0 & 1) : (k & 1);
                    const uint32_t b0 = odd ? vb[k / 2][2] : vb[k / 2][0], b1 = odd ? vb[k / 2][3] : vb[k / 2][1];
#pragma unroll
                    for (int m = 2; m >= 0; --m) mma(acc[r][k], t[m], b0, b1);
                }
            }
        }
        __syncthreads();
        load(s + 2);
    }

    float* end = ps.end;
    long long end_at = (static_cast<long long>(seq) * p.H + h) * N * p.P;
    if (ps.local) {
        end = p.seg_end[ps.rev];
        if (tile == 0 && threadIdx.x == 0 && !ps.rev) {
            double log = 0.;
            for (int c = 0; c < chunks; ++c) {
                const float2 e = p.gb[(static_cast<long long>(slot0 + c) * p.H + h) * kChunk + kChunk - 1];
                log += static_cast<double>(e.x) + static_cast<double>(e.y);
            }
            p.seg_log[static_cast<long long>(blockIdx.x) * p.H + h] = log;
        }
        end_at = (static_cast<long long>(blockIdx.x) * p.H + h) * N * p.P;
    } else if (ps.rev ? !seg_first : !seg_last) {
        end = nullptr;
    }
    if (end) {
#pragma unroll
        for (int r = 0; r < Sh::kRows; ++r)
#pragma unroll
            for (int k = 0; k < Sh::kCols; ++k)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int2 at = place(r, k, e);
                    if (at.y < cols)
                        *reinterpret_cast<float2*>(end + end_at + static_cast<long long>(at.x) * p.P + tile * kTile + at.y) =
                            make_float2(acc[r][k][e], acc[r][k][e + 1]);
                }
    }
}

// Segments: the state each starts from, from what each adds (states_kernel with
// `local`) and the decay over it, in the order of the recurrence.  The caller's
// initial state is read here and nowhere later, so that it may be overwritten.
__global__ void __launch_bounds__(kThreads) segments_kernel(const __grid_constant__ Params p,
                                                            const __grid_constant__ Pass fwd,
                                                            const __grid_constant__ Pass bwd) {
    wait_before();
    let_next();
    const bool rev = blockIdx.z & 1;
    const Pass& ps = rev ? bwd : fwd;
    const int seq = blockIdx.z >> 1, h = blockIdx.y;
    const long long cells = static_cast<long long>(p.N) * p.P;
    const long long e = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) * 4;
    if (!ps.k || e >= cells) return;
    int lo, len;
    sequence(p, seq, lo, len);
    if (p.steps && len <= p.steps) return;
    const int unit = kChunk * p.seg_chunks;
    const int slot0 = first_slot(p, seq, lo, unit), segs = max(1, (len + unit - 1) / unit);
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ps.init) S = *reinterpret_cast<const float4*>(ps.init + (static_cast<long long>(seq) * p.H + h) * cells + e);
    for (int i = 0; i < segs; ++i) {
        const long long sh = static_cast<long long>(slot0 + (rev ? segs - 1 - i : i)) * p.H + h;
        *reinterpret_cast<float4*>(p.seg_start[rev] + sh * cells + e) = S;
        if (i + 1 == segs) break;
        const float4 add = *reinterpret_cast<const float4*>(p.seg_end[rev] + sh * cells + e);
        const float a = ex2(static_cast<float>(p.seg_log[sh]));
        S = make_float4(fmaf(a, S.x, add.x), fmaf(a, S.y, add.y), fmaf(a, S.z, add.z), fmaf(a, S.w, add.w));
    }
}

// ---------------------------------------------------------------------------
// Outputs: a block per (chunk, set of heads of one group).  The scores C_i.B_j
// do not depend on the head: each warp keeps those of its 16 rows in registers
// and turns them, head by head, into the left operand of the product with x.
// The decay between two tokens of different 16-token blocks is the product of
// two powers that meet at the end of the earlier block, both at most 1 where
// decays are: a table of dt_j 2^(b_e - b_j) per head and one power per row and
// block take the place of one power per pair.  Bound by instruction issue: 315 us for 8 x
// 2048 tokens, 80 heads of 128 x 64 (scan_out_tc.cu, which has dk of 64 and 128: 150).
// ---------------------------------------------------------------------------
template <int N>
struct OutShape {
    static constexpr int kQ = kChunk * N * 2;
    static constexpr int kX = kChunk * kTile * 2;
    static constexpr int kState = N * kTile * 2;
    static constexpr int kStage = kX + kState;
    static constexpr int kSecond = kStage > kQ ? kStage : kQ;   // second stage, and first the keys
    static constexpr int kGates = kChunk * (8 + 4);             // b, dt
    static constexpr int kSmem = kQ + kStage + kSecond + 2 * kGates + kChunk * 4;
};

template <int N>
__global__ void __launch_bounds__(kThreads, N <= 128 ? 2 : 1) out_kernel(const __grid_constant__ Params p, int head_set) {
    using Sh = OutShape<N>;
    extern __shared__ __align__(128) uint8_t smem[];
    wait_before();
    const Rows rg = slot_rows(p, blockIdx.x);
    if (!rg.valid) return;
    const int sets = (p.per + head_set - 1) / head_set;
    const int group = blockIdx.y / sets, set = blockIdx.y - group * sets;
    const int h0 = group * p.per + set * head_set;
    const int items = min(head_set, p.per - set * head_set) * p.tiles;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint32_t base = smem_u32(smem);
    const uint32_t sq = base, st0 = base + Sh::kQ, st1 = st0 + Sh::kStage;
    uint8_t* gates = smem + Sh::kQ + Sh::kStage + Sh::kSecond;
    float* fac = reinterpret_cast<float*>(gates + 2 * Sh::kGates);
    const int valid = rg.valid;

    auto load = [&](int it) {
        const int h = h0 + it / p.tiles, tile = it % p.tiles;
        const int cols = min(kTile, p.P - tile * kTile);
        const uint32_t st = (it & 1) ? st1 : st0;
        load_tile<2 * kTile, kChunk>(st, p.x + rg.first * p.xs + static_cast<long long>(h) * p.P + tile * kTile, p.xs, valid, cols / 8);
        const long long cell = (static_cast<long long>(blockIdx.x) * p.H + h) * p.tiles + tile;
        load_tile<2 * kTile, N>(st + Sh::kX, p.sh + cell * N * kTile, kTile, N, kTile / 8);
        const long long at = (static_cast<long long>(blockIdx.x) * p.H + h) * kChunk;
        const uint32_t gs = base + Sh::kQ + Sh::kStage + Sh::kSecond + (it & 1) * Sh::kGates;
        if (threadIdx.x < 64) cp16(gs + threadIdx.x * 16, reinterpret_cast<const uint8_t*>(p.gb + at) + threadIdx.x * 16, true);
        else if (threadIdx.x < 96)
            cp16(gs + kChunk * 8 + (threadIdx.x - 64) * 16, reinterpret_cast<const uint8_t*>(p.gdt + at) + (threadIdx.x - 64) * 16, true);
    };

    load_tile<2 * N, kChunk>(sq, p.Cm + rg.first * p.cs + group * N, p.cs, valid, N / 8);
    load_tile<2 * N, kChunk>(st1, p.Bm + rg.first * p.bs + group * N, p.bs, valid, N / 8);
    cp_commit();
    load(0);
    cp_commit();
    cp_wait<1>();
    __syncthreads();

    // scores of rows 16 warp.. against the tokens up to them
    const int row0 = warp * 16;
    const bool live = row0 < valid;
    float sc[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
    if (live) {
#pragma unroll
        for (int ks = 0; ks < N / 16; ++ks) {
            uint32_t a[4];
            frag_a<2 * N>(a, sq, row0, ks, lane);
#pragma unroll
            for (int kb = 0; kb < 8; ++kb) {
                if (kb > warp) break;
                uint32_t b[4];
                frag_b<2 * N>(b, st1, kb * 16, ks, lane);
                mma(sc[2 * kb], a, b[0], b[1]);
                mma(sc[2 * kb + 1], a, b[2], b[3]);
            }
        }
    }
    __syncthreads();

    for (int it = 0; it < items; ++it) {
        if (it + 1 < items) load(it + 1);
        cp_commit();
        cp_wait<1>();
        __syncthreads();
        const int h = h0 + it / p.tiles, tile = it % p.tiles;
        const uint32_t st = (it & 1) ? st1 : st0;
        const float2* b = reinterpret_cast<const float2*>(gates + (it & 1) * Sh::kGates);
        const float* dt = reinterpret_cast<const float*>(gates + (it & 1) * Sh::kGates + kChunk * 8);
        if (threadIdx.x < kChunk) fac[threadIdx.x] = dt[threadIdx.x] * ex2_diff(b[threadIdx.x | 15], b[threadIdx.x]);
        __syncthreads();
        if (live) {
            float acc[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
            // what the state before the chunk gives
#pragma unroll
            for (int ks = 0; ks < N / 16; ++ks) {
                uint32_t a[4];
                frag_a<2 * N>(a, sq, row0, ks, lane);
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {
                    uint32_t v[4];
                    frag_bt<2 * kTile>(v, st + Sh::kX, c2 * 16, ks, lane);
                    mma(acc[2 * c2], a, v[0], v[1]);
                    mma(acc[2 * c2 + 1], a, v[2], v[3]);
                }
            }
            const float2 b0 = b[row0 + g], b8 = b[row0 + g + 8];
            const float e0 = ex2(b0.x + b0.y), e8 = ex2(b8.x + b8.y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i][0] *= e0;
                acc[i][1] *= e0;
                acc[i][2] *= e8;
                acc[i][3] *= e8;
            }
            // what the chunk's own tokens give
#pragma unroll
            for (int kb = 0; kb < 8; ++kb) {
                if (kb > warp) break;
                uint32_t a[4];
                if (kb < warp) {
                    const float2 be = b[kb * 16 + 15];
                    const float r0 = ex2_diff(b0, be), r8 = ex2_diff(b8, be);
                    const float2 f0 = *reinterpret_cast<const float2*>(fac + kb * 16 + 2 * q);
                    const float2 f8 = *reinterpret_cast<const float2*>(fac + kb * 16 + 8 + 2 * q);
                    a[0] = pack(sc[2 * kb][0] * (r0 * f0.x), sc[2 * kb][1] * (r0 * f0.y));
                    a[1] = pack(sc[2 * kb][2] * (r8 * f0.x), sc[2 * kb][3] * (r8 * f0.y));
                    a[2] = pack(sc[2 * kb + 1][0] * (r0 * f8.x), sc[2 * kb + 1][1] * (r0 * f8.y));
                    a[3] = pack(sc[2 * kb + 1][2] * (r8 * f8.x), sc[2 * kb + 1][3] * (r8 * f8.y));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ri = g + (i & 1) * 8, cj = 2 * q + (i >> 1) * 8;
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = row0 + cj + e;
                            const float s = sc[2 * kb + (i >> 1)][2 * (i & 1) + e];
                            v[e] = cj + e <= ri ? s * (ex2_diff(i & 1 ? b8 : b0, b[j]) * dt[j]) : 0.f;
                        }
                        a[i] = pack(v[0], v[1]);
                    }
                }
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {
                    uint32_t v[4];
                    frag_bt<2 * kTile>(v, st, c2 * 16, kb, lane);
                    mma(acc[2 * c2], a, v[0], v[1]);
                    mma(acc[2 * c2 + 1], a, v[2], v[3]);
                }
            }
            if (p.D) {
                const float d = __ldg(p.D + h);
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        uint32_t xv;
                        const uint32_t ad = st + tile_at<2 * kTile>(row0 + g + (e ? 8 : 0), i) + 4 * q;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(xv) : "r"(ad));
                        acc[i][e] = fmaf(d, lo_of(xv), acc[i][e]);
                        acc[i][e + 1] = fmaf(d, hi_of(xv), acc[i][e + 1]);
                    }
            }
            const int cols = min(kTile, p.P - tile * kTile);
            store_rows(p.out + (static_cast<long long>(rg.first) * p.H + h) * p.P + tile * kTile,
                       static_cast<long long>(p.H) * p.P, row0, valid, cols, acc, lane);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// A few tokens per sequence (serving): the recurrence itself, token by token,
// with a tile of 64 state columns of one head in registers.  A thread owns four
// columns of every kLanes-th row; the readout is summed over a warp's lanes of
// the same columns, then over the warps.  Bound by the states' one read and one
// write: 128 sequences, 80 heads of 128 x 64, one token: 111 us back to back, 6.04 TB/s,
// 92% of the measured copy rate.  The chunk kernels would make a pass over the states
// more.
// ---------------------------------------------------------------------------
template <int N>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Params p) {
    constexpr int R = N / 16;                    // rows of a thread at 64 columns
    __shared__ float key[2][N];                  // B, C of the token
    __shared__ float4 part[kThreads / 32][16];
    wait_before();
    if (!p.ragged && p.flag && blockIdx.x == 0 && threadIdx.x == 0) *p.flag = 0u;   // a whole call by itself
    const int tile = blockIdx.x % p.tiles, h = (blockIdx.x / p.tiles) % p.H;
    const int seq = blockIdx.x / p.tiles / p.H;
    int lo, len;
    sequence(p, seq, lo, len);
    if (p.ragged && len > p.steps) return;   // the chunk kernels'
    const int cols = min(kTile, p.P - tile * kTile), groups = cols / 4, lanes = kThreads / groups;
    const int cg = threadIdx.x % groups, rl = threadIdx.x / groups, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long at = ((static_cast<long long>(seq) * p.H + h) * N) * p.P + tile * kTile + cg * 4;
    float4 S[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = rl + r * lanes;
        S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.state_in && row < N) S[r] = *reinterpret_cast<const float4*>(p.state_in + at + static_cast<long long>(row) * p.P);
    }
    const int group = h / p.per;
    for (int t = 0; t < len; ++t) {
        const long long tok = lo + t;
        for (int i = threadIdx.x; i < 2 * N; i += kThreads) {
            const bf16* src = i < N ? p.Bm + tok * p.bs + group * N + i : p.Cm + tok * p.cs + group * N + i - N;
            key[i / N][i % N] = __bfloat162float(*src);
        }
        const float dt = p.dt ? __ldg(p.dt + tok * p.H + h) : 1.f;
        const float a = p.decay ? __ldg(p.decay + tok * p.H + h)
                                : static_cast<float>(exp2(static_cast<double>(dt) * __ldg(p.A + h) * 1.4426950408889634));
        const uint2 xr = __ldg(reinterpret_cast<const uint2*>(p.x + tok * p.xs + static_cast<long long>(h) * p.P + tile * kTile + cg * 4));
        const float4 x = make_float4(lo_of(xr.x), hi_of(xr.x), lo_of(xr.y), hi_of(xr.y));
        const float4 u = make_float4(dt * x.x, dt * x.y, dt * x.z, dt * x.w);
        __syncthreads();
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = rl + r * lanes;
            if (row >= N) break;
            const float k = key[0][row], c = key[1][row];
            S[r].x = fmaf(a, S[r].x, k * u.x);
            S[r].y = fmaf(a, S[r].y, k * u.y);
            S[r].z = fmaf(a, S[r].z, k * u.z);
            S[r].w = fmaf(a, S[r].w, k * u.w);
            y.x = fmaf(c, S[r].x, y.x);
            y.y = fmaf(c, S[r].y, y.y);
            y.z = fmaf(c, S[r].z, y.z);
            y.w = fmaf(c, S[r].w, y.w);
        }
        for (int d = groups; d < 32; d <<= 1) {
            y.x += __shfl_xor_sync(0xffffffffu, y.x, d);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, d);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, d);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, d);
        }
        if (lane < groups) part[warp][lane] = y;
        __syncthreads();
        if (threadIdx.x < groups) {
            const float d = p.D ? __ldg(p.D + h) : 0.f;
            y = make_float4(d * x.x, d * x.y, d * x.z, d * x.w);
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                const float4 v = part[w][threadIdx.x];
                y.x += v.x;
                y.y += v.y;
                y.z += v.z;
                y.w += v.w;
            }
            *reinterpret_cast<uint2*>(p.out + (tok * p.H + h) * p.P + tile * kTile + cg * 4) =
                make_uint2(pack(y.x, y.y), pack(y.z, y.w));
        }
    }
    if (p.state_out) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = rl + r * lanes;
            if (row < N) *reinterpret_cast<float4*>(p.state_out + at + static_cast<long long>(row) * p.P) = S[r];
        }
    }
}

template <class F>
int allow_smem(F* f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int N>
int states_n(const Params& p, const tc::Maps& m, bool backward, const Pass& f, const Pass& b, cudaStream_t s) {
    using Sh = StateShape<N>;
    if (N >= 64 && states_tc_ok(p)) return launch_states_tc(p, m, backward, f, b, s);
    const dim3 grid(p.seg_chunks ? p.seg_slots : (p.longs ? p.longs : p.n), p.H * p.tiles, backward ? 2 : 1);
    auto* k = backward ? states_kernel<N, true> : states_kernel<N, false>;
    const int err = allow_smem(k, Sh::kSmem);
    if (err) return err;
    return launch(k, grid, kThreads, Sh::kSmem, s, !p.slots, p, f, b);
}

int states_pass(const Params& p, const tc::Maps& m, bool backward, const Pass& f, const Pass& b, cudaStream_t s) {
    switch (p.N) {
        case 16: return states_n<16>(p, m, backward, f, b, s);
        case 32: return states_n<32>(p, m, backward, f, b, s);
        case 64: return states_n<64>(p, m, backward, f, b, s);
        case 128: return states_n<128>(p, m, backward, f, b, s);
        default: return states_n<256>(p, m, backward, f, b, s);
    }
}

template <int N>
int out_n(const Params& p, int head_set, cudaStream_t s) {
    using Sh = OutShape<N>;
    const int err = allow_smem(out_kernel<N>, Sh::kSmem);
    if (err) return err;
    const dim3 grid(p.slots, p.G * ((p.per + head_set - 1) / head_set));
    return launch(out_kernel<N>, grid, kThreads, Sh::kSmem, s, false, p, head_set);
}

}  // namespace

int launch_gates(const Params& p, cudaStream_t s) {
    return launch(gates_kernel, dim3(p.slots, (p.H + kGateHeads - 1) / kGateHeads), kThreads, 0, s, true, p);
}

int launch_states(const Params& p, const tc::Maps& m, bool backward, cudaStream_t s) {
    const Pass f{p.Bm, p.x, p.bs, p.xs, p.state_in, p.state_out, 0, 0};
    const Pass b{backward ? p.Cm : nullptr, p.dout, p.cs, static_cast<long long>(p.H) * p.P, p.dstate_out, p.dstate_in, 1, 0};
    if (p.seg_chunks) {
        Pass lf = f, lb = b;
        lf.local = lb.local = 1;
        int err = states_pass(p, m, backward, lf, lb, s);
        if (err) return err;
        err = launch(segments_kernel, dim3((p.N * p.P / 4 + kThreads - 1) / kThreads, p.H, 2 * p.n), kThreads, 0, s, false, p, f, b);
        if (err) return err;
    }
    return states_pass(p, m, backward, f, b, s);
}

int launch_step(const Params& p, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.n) * p.H * p.tiles;
    const bool first = !p.ragged;
    switch (p.N) {
        case 16: return launch(step_kernel<16>, grid, kThreads, 0, s, first, p);
        case 32: return launch(step_kernel<32>, grid, kThreads, 0, s, first, p);
        case 64: return launch(step_kernel<64>, grid, kThreads, 0, s, first, p);
        case 128: return launch(step_kernel<128>, grid, kThreads, 0, s, first, p);
        default: return launch(step_kernel<256>, grid, kThreads, 0, s, first, p);
    }
}

int launch_out(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s) {
    if (out_tc_ok(p)) return launch_out_tc(p, m, head_set, s);
    switch (p.N) {
        case 16: return out_n<16>(p, head_set, s);
        case 32: return out_n<32>(p, head_set, s);
        case 64: return out_n<64>(p, head_set, s);
        case 128: return out_n<128>(p, head_set, s);
        default: return out_n<256>(p, head_set, s);
    }
}

}  // namespace scan
}  // namespace rsq
