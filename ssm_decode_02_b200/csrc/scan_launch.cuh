// scan_launch.cuh -- the kernels of one call, launched so that they follow one another
// without a gap (programmatic dependent launch).
//
// A kernel's blocks start where SMs are free once every block of the one before has
// called let_next() or ended; wait_before() holds them until that one is complete, with
// all that it wrote.  Every block calls wait_before() before it leaves and before it uses
// what a kernel before may have written, and let_next() only behind it, so that a
// complete kernel always means that those before it are complete as well.  The first
// kernel of a call starts after all that is in the stream.
//
// What a kernel of the same call writes is read by plain loads: its writer may still run
// when the reader's blocks start, and a read-only load (__ldg) may be moved over the wait.
//
// Kernels of several rounds of blocks do not call let_next(): with the next kernel's
// blocks placed while the last round ran, the gradient of 4 x 2048 tokens with 80 heads of
// 128 x 64 took 593 us instead of 562.  Against plain launches: that gradient 575 -> 562 us, the
// ragged one of a few short sequences 82 -> 76, a norm's gradient with its column sums 98.6 -> 96.4.
#pragma once

#include <cuda_runtime.h>

namespace rsq {

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Formal, class... Actual>
int launch(void (*kernel)(Formal...), dim3 grid, int threads, size_t smem, cudaStream_t s, bool first, Actual... args) {
    cudaLaunchAttribute after;
    after.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &after;
    c.numAttrs = first ? 0 : 1;
    return cudaLaunchKernelEx(&c, kernel, static_cast<Formal>(args)...);
}

}  // namespace rsq
