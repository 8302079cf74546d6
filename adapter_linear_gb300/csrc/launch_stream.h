// launch_stream.h -- the launch of kernels that pass over memory without shared memory.
#pragma once

#include <utility>

#include "internal.h"

namespace lora {

// The library's kernels ask for the largest shared memory, so that an SM need not be emptied between two of them.
// That leaves L1 28 KB, and loads wait for room in it: a kernel that streams (large calls) asks for L1 instead
// (pages of a compaction, 778 MB: 143 us, so 125).
template <class... Params, class... Args>
cudaError_t launch_stream(bool streams, void (*fn)(Params...), unsigned ctas, int threads, cudaStream_t stream, Args &&...args)
{
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[0].val.sharedMemCarveout = cudaSharedmemCarveoutMaxL1;
    cfg.attrs = attr;
    cfg.numAttrs = streams ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, std::forward<Args>(args)...);
}

}  // namespace lora
