// Launches that overlap the end of the kernel before them in the stream.
//
// The attention-side kernels of a decode step take a few microseconds each, and
// between two plain launches the GPU stands still for about one more. These
// kernels are launched so that their blocks may take their places while the kernel
// before them still runs; they then wait, before their first access to global
// memory, until it has ended and its writes are visible, so nothing is reordered.
// Every thread waits, the idle ones too: a kernel of this kind therefore never
// ends before the one in front of it, and whatever follows it finds both done.
// What an earlier kernel may write (weights and scales too) is not read through the
// non-coherent path, since a block can be there before the write is, and no load
// may move in front of the wait: it is volatile or a plain access, or its pointer
// comes from past_wait().
#pragma once

#include "common.cuh"

namespace rssm {

// First statement of a kernel (or after set-up that touches no global memory).
__device__ __forceinline__ void after_predecessor() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// p, known only after the wait, for loads that may otherwise move freely.
template <class T>
__device__ __forceinline__ const T* past_wait(const T* p) {
    asm volatile("" : "+l"(p));
    return p;
}

template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

}  // namespace rssm
