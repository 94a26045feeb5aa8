// early_launch.h -- kernels of one call, launched one behind the other without a
// gap (programmatic dependent launch).
#pragma once

#include <cuda_runtime.h>

namespace credit {

// A kernel of a call may be launched while the one before it still runs: it waits
// for it in wait_for_launches().  (Before the first kernel of a call that is
// whatever the stream held, which is waited for just the same.)
inline cudaLaunchAttribute early_launch() {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*fn)(Params...), dim3 grid, int threads, cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr = early_launch();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<Params>(args)...);
}

}  // namespace credit
