// kv_launch_join.cuh -- launch of the join behind an attention kernel of `grid` CTAs.
#pragma once

#include <cuda_runtime.h>

#include "kv_join.cuh"

namespace gdn {

template <int KT, int LEAST>
cudaError_t launch_join(const KvArgs& a, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(grid - 1) * kvj::SHARE), cfg.blockDim = dim3(kvj::NT), cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<KT, LEAST>, a, grid);
}

}  // namespace gdn
