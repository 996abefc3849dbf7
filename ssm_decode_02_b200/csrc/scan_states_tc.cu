// scan_states_tc.cu -- the states before the chunks on the fifth-generation tensor
// cores (tcgen05): the form of states_kernel (scan_forward.cu) for dk >= 64 and
// heads that fill 128 value columns.
//
// A block carries 128 value columns (two heads of 64, one of 128, half of one of
// 256) through a sequence or segment.  Per chunk the product of the weighted values,
// 128 x tokens in three bf16 terms, with the keys, tokens x N, is a tcgen05 product
// into one of two tensor-memory tiles; a thread holds half a state column of N
// binary32 in registers, stores it as the state before the chunk and updates it
// from the tile while the next chunk's product runs into the other.
//
// What bounds it: a value becomes three bf16 terms in about nine instructions,
// 128 x 128 of them per chunk; the products themselves are 1536 cycles of the
// matrix unit per chunk at N = 128.
#include "tc.cuh"

namespace rsq {
namespace scan {
namespace {

constexpr int kHalf = 64;    // tokens of a step
constexpr int kCols = 128;   // value columns of a block

template <int N>
struct Shape {
    static constexpr int kStages = N <= 128 ? 3 : 2;
    static constexpr int kKeys = kHalf * N * 2;
    static constexpr int kValues = kHalf * kCols * 2;
    static constexpr int kStage = kKeys + kValues;
    static constexpr int kTerms = 3 * kValues;
    static constexpr int kSmem = 1024 + kStages * kStage + 2 * kTerms + 2 * 8 * kHalf * 4 + 64;
};

template <int N, bool F32>
__global__ void __launch_bounds__(kThreads, 1) states_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ Pass fwd,
                                                                 const __grid_constant__ Pass bwd) {
    using Sh = Shape<N>;
    extern __shared__ uint8_t raw_smem[];
    const Pass& ps = blockIdx.z ? bwd : fwd;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = blockIdx.y * kCols, h0 = c0 / p.P, heads = p.P >= kCols ? 1 : kCols / p.P;
    const int group = h0 / p.per;

    int seq, lo, len, slot0, seg_first = 1, seg_last = 1;
    if (p.seg_chunks) {
        const Range r = slot_range(p, blockIdx.x, kChunk * p.seg_chunks);
        if (!r.valid && !(r.index == 0 && !ps.local)) return;
        seq = r.seq;
        lo = r.first;
        len = r.valid;
        slot0 = first_slot(p, seq, r.seq_first, kChunk) + r.index * p.seg_chunks;
        seg_first = r.index == 0;
        seg_last = lo + len == r.seq_first + r.seq_len;
    } else {
        seq = blockIdx.x;
        sequence(p, seq, lo, len);
        slot0 = first_slot(p, seq, lo, kChunk);
    }
    const int chunks = (len + kChunk - 1) / kChunk, steps = 2 * chunks;

    uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t base = smem_u32(smem);
    const uint32_t terms = base + Sh::kStages * Sh::kStage;
    float* wgt = reinterpret_cast<float*>(smem + Sh::kStages * Sh::kStage + 2 * Sh::kTerms);  // [2][heads][kHalf]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wgt + 2 * 8 * kHalf);
    const uint32_t bars = smem_u32(tmem_slot + 2);
    if (warp == 0) tc::tmem_alloc(smem_u32(tmem_slot), 2 * N);
    if (threadIdx.x == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;

    // this thread: value column m (its tensor-memory lane), state rows n0 .. n0 + N/2 - 1
    const int m = (warp & 3) * 32 + lane, n0 = (warp >> 2) * (N / 2);
    const int h = h0 + m / p.P, pc = (c0 + m) % p.P;      // its head and column of the head
    const long long head_cells = static_cast<long long>(N) * p.P;
    float S[N / 2];
    const float* init = ps.init;
    long long at0 = (static_cast<long long>(seq) * p.H + h) * head_cells + pc;
    if (p.seg_chunks && !ps.local) {
        init = p.seg_start[ps.rev];
        at0 = (static_cast<long long>(blockIdx.x) * p.H + h) * head_cells + pc;
    }
    if (ps.local) init = nullptr;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) S[i] = init ? __ldg(init + at0 + static_cast<long long>(n0 + i) * p.P) : 0.f;

    const bf16* kp = ps.k + static_cast<long long>(group) * N;
    const bf16* vp = ps.v + c0;
    auto chunk_of = [&](int s) { return ps.rev ? chunks - 1 - s / 2 : s / 2; };
    auto load = [&](int s) {
        if (s < steps) {
            const int row = chunk_of(s) * kChunk + (s & 1) * kHalf;
            const int valid = max(0, min(kHalf, len - row));
            const uint32_t st = base + (s % Sh::kStages) * Sh::kStage;
            const long long first = lo + (valid ? row : 0);
#pragma unroll
            for (int b = 0; b < N / 64; ++b) load_tile<128, kHalf>(st + b * 8192, kp + first * ps.ks + b * 64, ps.ks, valid, 8);
#pragma unroll
            for (int b = 0; b < 2; ++b) load_tile<128, kHalf>(st + Sh::kKeys + b * 8192, vp + first * ps.vs + b * 64, ps.vs, valid, 8);
            for (int i = threadIdx.x; i < heads * kHalf; i += kThreads) {
                const long long at = (static_cast<long long>(slot0 + chunk_of(s)) * p.H + h0 + i / kHalf) * kChunk;
                const int t = (s & 1) * kHalf + i % kHalf;
                const float2 b = p.gb[at + t], end = p.gb[at + kChunk - 1];
                wgt[(s & 1) * 8 * kHalf + i] = ps.rev ? ex2(b.x + b.y) : ex2_diff(end, b) * p.gdt[at + t];
            }
        }
        cp_commit();
    };
    // the state before chunk c goes out, then takes in the chunk's product
    auto update = [&](int s_last) {
        const int c = chunk_of(s_last);
        const long long cell = ((static_cast<long long>(slot0 + c) * p.H + h) * p.tiles + pc / kTile) * N * kTile + pc % kTile;
        const float2 end = p.gb[(static_cast<long long>(slot0 + c) * p.H + h) * kChunk + kChunk - 1];
        const float a = ex2(end.x + end.y);
        const uint32_t d = tmem + ((s_last / 2) & 1) * N + n0 + ((static_cast<uint32_t>(warp) & 3) << 21);
#pragma unroll
        for (int b = 0; b < N / 64; ++b) {
            float v[32];
            tc::tmem_ld32(v, d + b * 32);
            if (!ps.local) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const long long o = cell + static_cast<long long>(n0 + b * 32 + i) * kTile;
                    if constexpr (F32)
                        (ps.rev ? p.df : p.sf)[o] = S[b * 32 + i];
                    else
                        p.sh[o] = __float2bfloat16_rn(S[b * 32 + i]);
                }
            }
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) S[b * 32 + i] = fmaf(a, S[b * 32 + i], v[i]);
        }
        tc::fence_before();
    };

    bool ok = true;
    load(0);
    for (int s = 0; s < steps; ++s) {
        // the products of step s - 2 are done with the terms that this step writes, and with
        // the stage that the next one loads (with two stages: those of step s - 1)
        const int done = Sh::kStages == 3 ? s - 2 : s - 1;
        if (s >= 2 && !(ok = tc::wait_all(bars + (s & 1) * 8, (s / 2 - 1) & 1, p.flag))) break;
        if (Sh::kStages == 2 && s >= 1 && !(ok = tc::wait_all(bars + ((s - 1) & 1) * 8, ((s - 1) / 2) & 1, p.flag))) break;
        (void)done;
        cp_wait<0>();
        __syncthreads();
        const uint32_t st = base + (s % Sh::kStages) * Sh::kStage, tb = terms + (s & 1) * Sh::kTerms;
        const float* w = wgt + (s & 1) * 8 * kHalf;
        // weighted values in three terms: eight columns of one token at a time
#pragma unroll
        for (int i = threadIdx.x; i < kHalf * 16; i += kThreads) {
            const int t = i >> 4, c = i & 15;
            const uint32_t o = (c >> 3) * 8192 + tile_at<128>(t, c & 7);
            uint32_t x[4], r[3][4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(st + Sh::kKeys + o));
            const float wt = w[(c * 8 / p.P) * kHalf + t];
#pragma unroll
            for (int k = 0; k < 4; ++k) split3(lo_of(x[k]) * wt, hi_of(x[k]) * wt, r[0][k], r[1][k], r[2][k]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tb + k * Sh::kValues + o), "r"(r[k][0]), "r"(r[k][1]),
                             "r"(r[k][2]), "r"(r[k][3])
                             : "memory");
        }
        tc::fence_smem();
        tc::fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
            tc::fence_after();
            const uint32_t d = tmem + ((s / 2) & 1) * N;
            constexpr uint32_t id = tc::idesc(N, true, true);
#pragma unroll
            for (int ks = 0; ks < kHalf / 16; ++ks)
#pragma unroll
                for (int k = 2; k >= 0; --k)
                    tc::mma(d, tc::desc(tb + k * Sh::kValues + ks * 2048, 8192), tc::desc(st + ks * 2048, 8192), id,
                            (s & 1) || ks || k != 2);
            tc::commit(bars + (s & 1) * 8);
        }
        load(s + 1);
        if (!(s & 1) && s) {  // the chunk before, while this one's product runs
            if (!(ok = tc::wait_all(bars + 8, ((s - 1) / 2) & 1, p.flag))) break;
            tc::fence_after();
            update(s - 1);
        }
    }
    cp_wait<0>();
    if (ok && steps && (ok = tc::wait_all(bars + 8, ((steps - 1) / 2) & 1, p.flag))) {
        tc::fence_after();
        update(steps - 1);
    }

    float* end = ps.end;
    long long end_at = (static_cast<long long>(seq) * p.H + h) * head_cells + pc;
    if (ps.local) {
        end = p.seg_end[ps.rev];
        if (threadIdx.x < heads && c0 % p.P == 0 && !ps.rev) {
            double log = 0.;
            for (int c = 0; c < chunks; ++c) {
                const float2 e = p.gb[(static_cast<long long>(slot0 + c) * p.H + h0 + threadIdx.x) * kChunk + kChunk - 1];
                log += static_cast<double>(e.x) + static_cast<double>(e.y);
            }
            p.seg_log[static_cast<long long>(blockIdx.x) * p.H + h0 + threadIdx.x] = log;
        }
        end_at = (static_cast<long long>(blockIdx.x) * p.H + h) * head_cells + pc;
    } else if (ps.rev ? !seg_first : !seg_last) {
        end = nullptr;
    }
    if (end) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) end[end_at + static_cast<long long>(n0 + i) * p.P] = S[i];
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 2 * N);
}

template <int N>
int run(const Params& p, bool backward, const Pass& f, const Pass& b, cudaStream_t s) {
    auto* k = backward ? states_tc_kernel<N, true> : states_tc_kernel<N, false>;
    const int err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<N>::kSmem);
    if (err) return err;
    const dim3 grid(p.seg_chunks ? p.seg_slots : p.n, p.H * p.P / kCols, backward ? 2 : 1);
    k<<<grid, kThreads, Shape<N>::kSmem, s>>>(p, f, b);
    return cudaGetLastError();
}

}  // namespace

int launch_states_tc(const Params& p, bool backward, const Pass& f, const Pass& b, cudaStream_t s) {
    switch (p.N) {
        case 64: return run<64>(p, backward, f, b, s);
        case 128: return run<128>(p, backward, f, b, s);
        default: return run<256>(p, backward, f, b, s);
    }
}

}  // namespace scan
}  // namespace rsq
