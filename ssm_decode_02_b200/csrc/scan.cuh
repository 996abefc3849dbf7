// scan.cuh -- shared parts of the scan kernels (rsq_scan, rsq_scan_backward):
// sequences and chunks, the workspace, shared-memory tiles and the warp matrix
// products.
//
// A sequence is cut into chunks of kChunk tokens.  With b_i the sum of log2 a_t
// over the chunk's tokens up to i, L_ij = 2^(b_i - b_j) for i >= j, S_0 the state
// before the chunk and dS the gradient of the state behind it (b_end at its end):
//   out_i = D x_i + 2^b_i S_0^T C_i + sum_{j<=i} L_ij dt_j (C_i.B_j) x_j
//   S_end = 2^b_end S_0 + sum_j 2^(b_end-b_j) dt_j B_j x_j^T
//   dS_0  = 2^b_end dS  + sum_i 2^b_i C_i dout_i^T
// so that both state recurrences are one matrix product per chunk and everything
// else is independent from chunk to chunk.
//
// Roundings.  The matrix products take bf16 operands.  The states themselves are carried
// in binary32; where a state, or scores times decays, enters a product whose result is
// rounded to bf16 anyway (out, dx, dB, dC), it is rounded to bf16 once on the way.  That
// leaves an error of 2.3e-3 of the result's norm, of which its own rounding is 1.7e-3;
// two terms more would triple those products and what is staged for them, in kernels that
// are bound by the issue of just that.  What reaches a binary32 result enters in three
// bf16 terms (split3).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rsq_device.cuh"
#include "rsq_internal.h"
#include "scan_launch.cuh"

namespace rsq {
namespace scan {

using bf16 = __nv_bfloat16;

constexpr int kChunk = 128;   // tokens of a chunk
constexpr int kTile = 64;     // state columns of a block's tile
constexpr int kThreads = 256;
constexpr int kSms = 148;     // of a B200
// log2 of a decay of zero: far below any exponent, so that its power is 0, and
// small enough that sums of 128 keep every other term in twice binary32
constexpr double kLogZero = -1e5;

// What every kernel of a call needs.
struct Params {
    int n, H, N, P, G, per;       // sequences, heads, state rows, state columns, groups, heads per group
    int tiles;                    // column tiles of a head
    int ragged;
    int tokens, len;              // rows of the token arrays; length of a sequence (not ragged)
    int steps;                    // ragged forward: sequences of so many tokens at most are step_kernel's
    int longs;                    // blocks of the states' kernels for the others of them (0: one for each sequence)
    const int32_t* cu;
    int slots;                    // chunk slots
    int seg_chunks, seg_slots;    // chunks of a segment (0: whole sequences), segment slots
    const bf16* x;
    const bf16* Bm;
    const bf16* Cm;
    long long xs, bs, cs;         // token strides
    const float* dt;
    const float* A;
    const float* D;
    const float* decay;
    const float* state_in;
    float* state_out;
    bf16* out;
    // workspace
    unsigned* flag;               // kFlagTimeout when a bounded wait ran out
    int2* rows;                   // [slots] first row and number of rows, for all kernels after the gates'
    float2* gb;                   // [slots][H][kChunk] b_i in two floats
    float* gdt;                   // [slots][H][kChunk] dt
    bf16* sh;                     // forward: states before the chunks [slots][H][tiles][N][kTile]
    float* sf;                    // backward: the same in binary32
    float* df;                    // backward: gradients of the states behind the chunks
    float* seg_end[2];            // per direction [seg_slots][H][N][P]: what a segment adds to the state,
    float* seg_start[2];          // and the state that it starts from
    double* seg_log;              // [seg_slots][H] log2 of a segment's decay
    // backward
    const bf16* dout;
    const float* dstate_out;
    bf16* dx;
    bf16* dBm;
    bf16* dCm;
    float* ddt;
    float* dlog;
    float* dA;
    float* dD;
    float* dstate_in;
    float* part;                  // [2][slots][H] partial dA, dD
};

struct Range {
    int seq, first, index, valid;  // sequence, first row, number within the sequence, rows (0: none)
    int seq_first, seq_len;
};

__device__ __forceinline__ void sequence(const Params& p, int b, int& lo, int& len) {
    if (!p.ragged) {
        lo = b * p.len;
        len = p.len;
        return;
    }
    lo = min(max(__ldg(p.cu + b), 0), p.tokens);
    len = min(max(__ldg(p.cu + b + 1), lo), p.tokens) - lo;
}

// The k-th sequence of more than p.steps tokens, or -1.  By a whole warp.
__device__ __forceinline__ int long_sequence(const Params& p, int k) {
    for (int i0 = 0; i0 < p.n; i0 += 32) {
        const int i = i0 + (threadIdx.x & 31);
        int lo, len = 0;
        if (i < p.n) sequence(p, i, lo, len);
        unsigned m = __ballot_sync(0xffffffffu, len > p.steps);
        const int c = __popc(m);
        if (k < c) {
            for (; k; --k) m &= m - 1;
            return i0 + __ffs(m) - 1;
        }
        k -= c;
    }
    return -1;
}

// First slot of sequence b when slots hold `unit` rows each.  Equal lengths:
// whole slots per sequence.  Ragged: lo/unit + b, which leaves every sequence
// enough slots before the next one's (ceil(len/unit) <= (lo+len)/unit - lo/unit + 1).
__device__ __forceinline__ int first_slot(const Params& p, int b, int lo, int unit) {
    return p.ragged ? lo / unit + b : b * ((p.len + unit - 1) / unit);
}

// The rows of a slot.
__device__ __forceinline__ Range slot_range(const Params& p, int slot, int unit) {
    Range r;
    int b;
    if (!p.ragged) {
        b = slot / ((p.len + unit - 1) / unit);
    } else {
        int lo = 0, hi = p.n - 1;  // the last sequence whose first slot is not behind this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (min(max(__ldg(p.cu + mid), 0), p.tokens) / unit + mid <= slot)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
    }
    sequence(p, b, r.seq_first, r.seq_len);
    r.seq = b;
    r.index = slot - first_slot(p, b, r.seq_first, unit);
    const long long at = static_cast<long long>(r.index) * unit;
    r.valid = (r.index < 0 || at >= r.seq_len || r.seq_len <= p.steps) ? 0 : static_cast<int>(min(static_cast<long long>(unit), r.seq_len - at));
    r.first = r.seq_first + static_cast<int>(r.valid ? at : 0);
    return r;
}

// The rows of a chunk slot, as the gates' kernel found them.
struct Rows {
    int first, valid;
};
__device__ __forceinline__ Rows slot_rows(const Params& p, int slot) {
    const int2 r = p.rows[slot];
    return Rows{r.x, r.y};
}

// ---------------------------------------------------------------------------
// Shared-memory tiles: rows of ROWB bytes, whose 16-byte chunks are permuted by
// the row so that the eight rows of a ldmatrix hit different banks.
// ---------------------------------------------------------------------------
template <int ROWB>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
    if constexpr (ROWB >= 128)
        chunk ^= row & 7;
    else if constexpr (ROWB == 64)
        chunk ^= (row >> 1) & 3;
    else
        chunk ^= (row >> 2) & 1;
    return static_cast<uint32_t>(row * ROWB + chunk * 16);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    const int n = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows 0..ROWS-1 of a tile from global rows `stride` elements apart; rows from
// `valid` on and chunks from `chunks` on become zero.
template <int ROWB, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const bf16* src, long long stride, int valid, int chunks) {
    constexpr int CH = ROWB / 16;
    for (int i = threadIdx.x; i < ROWS * CH; i += kThreads) {
        const int r = i / CH, c = i % CH;
        const bool on = r < valid && c < chunks;
        cp16(dst + tile_at<ROWB>(r, c), on ? src + r * stride + c * 8 : src, on);
    }
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A operand: rows row0..+15, columns 16 k.. of a row-major tile.
template <int ROWB>
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], uint32_t tile, int row0, int k, int lane) {
    ldsm4(r, tile + tile_at<ROWB>(row0 + (lane & 15), 2 * k + (lane >> 4)));
}
// A operand from the transposed tile: operand rows are tile columns col0..+15, k runs over tile rows 16 k...
template <int ROWB>
__device__ __forceinline__ void frag_at(uint32_t (&r)[4], uint32_t tile, int col0, int k, int lane) {
    ldsm4t(r, tile + tile_at<ROWB>(16 * k + (lane & 7) + ((lane >> 4) << 3), col0 / 8 + ((lane >> 3) & 1)));
}
// B operand of two 8-wide blocks (r[0], r[1] and r[2], r[3]): n runs over tile rows row0..+15, k over columns 16 k..
template <int ROWB>
__device__ __forceinline__ void frag_b(uint32_t (&r)[4], uint32_t tile, int row0, int k, int lane) {
    ldsm4(r, tile + tile_at<ROWB>(row0 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
}
// B operand from the transposed tile: n runs over tile columns col0..+15, k over tile rows 16 k..
template <int ROWB>
__device__ __forceinline__ void frag_bt(uint32_t (&r)[4], uint32_t tile, int col0, int k, int lane) {
    ldsm4t(r, tile + tile_at<ROWB>(16 * k + (lane & 15), col0 / 8 + (lane >> 4)));
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// (lo, hi) rounded to bf16, lo in the lower half
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// (lo, hi) as three bf16 terms each: 24 bits, so that products with a bf16
// operand lose no more than binary32 products do
__device__ __forceinline__ void split3(float lo, float hi, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
    t0 = pack(lo, hi);
    lo -= lo_of(t0);
    hi -= hi_of(t0);
    t1 = pack(lo, hi);
    t2 = pack(lo - lo_of(t1), hi - hi_of(t1));
}

__device__ __forceinline__ float ex2(float v) {
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}
// 2^(a - b) of exponents held in two floats
__device__ __forceinline__ float ex2_diff(float2 a, float2 b) { return ex2((a.x - b.x) + (a.y - b.y)); }

// Stores the eight 8-wide blocks of a warp's 16 x 64 product as bf16 rows, 16
// bytes a thread: lanes of a quad exchange blocks so that each holds a whole one.
__device__ __forceinline__ void store_rows(bf16* dst, long long stride, int row0, int valid, int cols,
                                           const float (&acc)[8][4], int lane) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int row = row0 + g + 8 * half;
#pragma unroll
        for (int set = 0; set < 2; ++set) {
            uint32_t v[4], o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = pack(acc[4 * set + i][2 * half], acc[4 * set + i][2 * half + 1]);
            // lane q of the quad collects block q: word s of it comes from lane s
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                // in round d this lane sends the block of lane q ^ d
                const int to = q ^ d;
                const uint32_t send = to == 0 ? v[0] : (to == 1 ? v[1] : (to == 2 ? v[2] : v[3]));
                const uint32_t got = __shfl_xor_sync(0xffffffffu, send, d);
                // it came from lane q ^ d and is word q ^ d
                if (to == 0) o[0] = got;
                if (to == 1) o[1] = got;
                if (to == 2) o[2] = got;
                if (to == 3) o[3] = got;
            }
            const int col = 32 * set + 8 * q;
            if (row < valid && col < cols)
                *reinterpret_cast<uint4*>(dst + row * stride + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// The gradients of a head's gates over one chunk, by one warp: lane l has tokens 4 l
// .. 4 l + 3.  With the tokens in NB blocks,
//   col[b][t] = sum over j of block b of Z_tj (t behind block b)
//             = sum over i >= t > j of block b of Z_ij (t in block b)
//   row[a][t] = sum over i > t of block a of Z_it / dt_t
// (Z and the other sums: scan_backward.cu).  The pairs (i, j) around a token t of
// block c, i >= t > j, are those of whole blocks around c, of later blocks with the
// tokens of c before t, of the tokens of c from t on with earlier blocks, and pairs
// within c.  No sum here is the difference of two others: every pair from t on, less
// those on t's one side, left up to 40 times the rounding error in dA, a sum over the
// tokens (over a whole chunk; 2 to 8 times within blocks of 32).  The sums around each
// token of a block cost 2% of a gradient (586 us against 575, 4 x 2048 tokens, 80 heads
// of 128 x 64).
// ---------------------------------------------------------------------------
struct HeadSums {
    const float* col;
    const float* row;
    const float* own;   // Z_tt / dt_t
    const float* in;
    const float* fin;
    const float* dot;   // x_t.dout_t
    float through;      // 2^b_end <S_0, dS>
};

template <int NB>
__device__ __forceinline__ void head_gates(const HeadSums& s, const float (&dt)[4], int valid, int lane, float (&dlog)[4],
                                           float (&dir)[4], float& dot) {
    constexpr int BS = kChunk / NB, LB = 32 / NB;   // tokens and lanes of a block
    const int c = lane / LB;
    float suf[4], pre[4], win[4], ins[4], fi[4];
    dot = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = lane * 4 + k;
        suf[k] = pre[k] = win[k] = ins[k] = fi[k] = dir[k] = 0.f;
        if (t >= valid) continue;
        float before = 0.f, after = 0.f;
        for (int b = 0; b < c; ++b) before += s.col[b * kChunk + t];
        for (int a = c + 1; a < NB; ++a) after += s.row[a * kChunk + t];
        const float within = s.row[c * kChunk + t];
        suf[k] = before;
        win[k] = s.col[c * kChunk + t];
        pre[k] = dt[k] * after;
        ins[k] = s.in[t];
        fi[k] = dt[k] * s.fin[t];
        dir[k] = ((after + within) + s.own[t]) + s.fin[t];
        dot += s.dot[t];
    }
    // whole blocks around block c
    float around = 0.f;
#pragma unroll 1
    for (int m = 1; m < NB - 1; ++m) {
        float v = 0.f;
        for (int i = (m + 1) * BS + lane; i < valid; i += 32)
            for (int b = 0; b < m; ++b) v += s.col[b * kChunk + i];
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (m == c) around = v;
    }
    // sums of the lanes behind (suf, ins) and before (pre, fi), within the block and over all
    const float s0 = (suf[0] + suf[1]) + (suf[2] + suf[3]), p0 = (pre[0] + pre[1]) + (pre[2] + pre[3]);
    const float i0 = (ins[0] + ins[1]) + (ins[2] + ins[3]), f0 = (fi[0] + fi[1]) + (fi[2] + fi[3]);
    float sb = __shfl_down_sync(0xffffffffu, s0, 1, LB), pb = __shfl_up_sync(0xffffffffu, p0, 1, LB);
    float ib = __shfl_down_sync(0xffffffffu, i0, 1), fb = __shfl_up_sync(0xffffffffu, f0, 1);
    if (lane % LB == LB - 1) sb = 0.f;
    if (lane % LB == 0) pb = 0.f;
    if (lane == 31) ib = 0.f;
    if (lane == 0) fb = 0.f;
#pragma unroll
    for (int d = 1; d < LB; d <<= 1) {
        const float a = __shfl_down_sync(0xffffffffu, sb, d, LB), b = __shfl_up_sync(0xffffffffu, pb, d, LB);
        if (lane % LB + d < LB) sb += a;
        if (lane % LB >= d) pb += b;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const float a = __shfl_down_sync(0xffffffffu, ib, d), b = __shfl_up_sync(0xffffffffu, fb, d);
        if (lane + d < 32) ib += a;
        if (lane >= d) fb += b;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    float up_p = pb, up_f = fb;
    float down_s[4], down_i[4];
#pragma unroll
    for (int k = 3; k >= 0; --k) {
        sb += suf[k];
        ib += ins[k];
        down_s[k] = sb;
        down_i[k] = ib;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        dlog[k] = (((down_s[k] + up_p) + around) + win[k]) + ((down_i[k] + up_f) + s.through);
        up_p += pre[k];
        up_f += fi[k];
    }
}

// One direction of the state recurrence.
struct Pass {
    const bf16* k;          // key rows: Bm | Cm
    const bf16* v;          // value rows: x | dout
    long long ks, vs;
    const float* init;      // [n][H][N][P] or null
    float* end;             // [n][H][N][P] or null
    int rev;
    int local;              // from zero to the segment's end only
};

// Whether the tcgen05 form of the state recurrence takes a shape: whole tiles of 64
// state rows, and blocks of 128 value columns that share their keys.
inline bool states_tc_ok(const Params& p) { return p.N >= 64 && p.P >= 64 && p.per * p.P % 128 == 0; }

// The same for the outputs.
inline bool out_tc_ok(const Params& p) { return (p.N == 64 || p.N == 128) && p.P >= 64; }

// The same for dx and the gates' gradients (two stages hold a head's tiles).
inline bool dx_tc_ok(const Params& p) { return (p.N == 64 || p.N == 128) && (p.P == 64 || p.P == 128); }

// The same for dB and dC.
inline bool dk_tc_ok(const Params& p) { return p.N >= 64 && p.P >= 64; }

namespace tc {
struct Maps;
}

// Launchers (scan_forward.cu, scan_backward.cu).  Return a cudaError_t value.
int launch_gates(const Params& p, cudaStream_t s);
int launch_states(const Params& p, const tc::Maps& m, bool backward, cudaStream_t s);  // with the segments' two passes, if any
int launch_out(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s);
int launch_out_tc(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s);
int launch_step(const Params& p, cudaStream_t s);
int launch_states_tc(const Params& p, const tc::Maps& m, bool backward, const Pass& f, const Pass& b, cudaStream_t s);  // one launch
int launch_dx_tc(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s);
int launch_dk_tc(const Params& p, const tc::Maps& m, cudaStream_t s);
int launch_backward(const Params& p, const tc::Maps& m, int head_set, cudaStream_t s);

}  // namespace scan
}  // namespace rsq
