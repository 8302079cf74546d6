// launch_stream.h -- the launch of kernels that pass over memory without shared memory.
#pragma once

#include <utility>

#include "internal.h"

namespace lora {

// The library's kernels ask for the largest shared memory, so that an SM need not be emptied between two of them.
// That leaves L1 28 KB, and loads wait for room in it: a kernel that streams (large calls) asks for L1 instead
// (pages of a compaction, 778 MB: 143 us, so 125). early: the kernel waits by itself for the one ahead of it.
template <class... Params, class... Args>
cudaError_t launch_stream(bool streams, bool early, void (*fn)(Params...), unsigned ctas, int threads, cudaStream_t stream,
                          Args &&...args)
{
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (streams) {
        attr[n].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
        attr[n++].val.sharedMemCarveout = cudaSharedmemCarveoutMaxL1;
    }
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, fn, std::forward<Args>(args)...);
}

}  // namespace lora
