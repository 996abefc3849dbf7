// tc.cuh -- fifth-generation tensor cores (tcgen05) for the scan kernels: tensor
// memory, shared-memory and instruction descriptors, bounded waits.
//
// Operand tiles lie in shared memory as rows of 64 bf16 (128 bytes), whose 16-byte
// chunks are permuted by the row (scan.cuh, tile_at<128>) -- the 128-byte swizzle
// of the matrix unit, eight rows repeating.  Tiles start on 1024 bytes.
//   k-major:  a row is one m (or n), its 64 columns are k
//   mn-major: a row is one k, its 64 columns are 64 m (or n)
#pragma once

#include <cuda.h>

#include "scan.cuh"

namespace rsq {
namespace scan {
namespace tc {

// ---- tiled copies ----------------------------------------------------------
// Boxes of 64 columns by 64 rows of the token arrays and of the bf16 states, written
// in the tiles' order (128-byte swizzle).  No multicast.
struct Maps {
    CUtensorMap x, Bm, Cm, dout, sh;
};
int make_maps(const Params& p, bool backward, Maps* m);  // scan_api.cu; a cudaError_t value

__device__ __forceinline__ void box(uint32_t dst, const CUtensorMap* map, int col, int row, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(col), "r"(row), "r"(bar)
                 : "memory");
}
constexpr uint32_t kBox = 64 * 128;  // bytes

// ---- tensor memory ---------------------------------------------------------
// Called by one whole warp; the base address is written to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// This thread's shared-memory writes, before the matrix unit reads them.
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 or 8 columns of this thread's lane.  The address has the warp's lane quarter in its
// upper half: a warp reaches lanes 32 (warp mod 4) .. + 31.
__device__ __forceinline__ void tmem_ld16(float (&v)[16], uint32_t a) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld8(float (&v)[8], uint32_t a) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- descriptors -----------------------------------------------------------
// Shared-memory matrix descriptor, 128-byte swizzle.  `lead`: bytes between blocks
// of 64 m or n (mn-major); groups of eight rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead) {
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 operands, binary32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// One lane of a converged warp.  The issuing warps stay together and enter only the
// products this way: descriptors are then computed once for the warp (uniform
// registers); with one lane in a branch of its own a gradient took 622 us instead of 588.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
// D[128 x n] (+)= A B, one thread.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(add ? 1 : 0)
        : "memory");
}
// The same with A in tensor memory (lane = row, two k per column).
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(add ? 1 : 0)
        : "memory");
}
// Arrives on `bar` when every product issued so far by this thread is done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A bounded wait of one warp, the same answer for every lane: false when it ran out,
// with the call's flag set.
__device__ __forceinline__ bool wait_warp(uint32_t bar, int phase, unsigned* flag) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, kWaitIters));
    if (!ok && (threadIdx.x & 31) == 0) atomicOr(flag, kFlagTimeout);
    return ok;
}

}  // namespace tc
}  // namespace scan
}  // namespace rsq
