// Launch of the join behind an attention kernel.
#include "kv_dispatch.h"
#include "kv_join.cuh"

namespace gdn {

cudaError_t launch_kv_join(const KvArgs& a, int grid, cudaStream_t stream) {
    if (grid == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(grid - 1) * kvj::SHARE), cfg.blockDim = dim3(kvj::NT), cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel, a);
}

}  // namespace gdn
