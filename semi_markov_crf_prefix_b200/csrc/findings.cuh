// findings.cuh -- what a kernel of the operators around the loss finds on the device: a word
// of the call's workspace, for who owns that, and a word of the library on each device,
// which outlives the workspaces that the package makes for a call and drops.  Every source
// that includes this has its own word: kernels then need no address from the host, which a
// first call under stream capture could not look up.
#pragma once

#include "device_util.cuh"

namespace semicrf {
namespace {

__device__ int32_t g_found;   // the first finding since it was cleared

__device__ __forceinline__ void report(int32_t *status, int code)
{
    set_status(status, code);
    set_status(&g_found, code);
}

// This source's word on the current device (the caller has synchronised).
cudaError_t read_found(int32_t *to) { return cudaMemcpyFromSymbol(to, g_found, sizeof(*to)); }

cudaError_t clear_found(cudaStream_t st)
{
    void *p;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_found);
    return e != cudaSuccess ? e : cudaMemsetAsync(p, 0, sizeof(int32_t), st);
}

}  // namespace
}  // namespace semicrf
