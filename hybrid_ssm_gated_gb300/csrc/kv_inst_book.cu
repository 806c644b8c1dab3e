// Launches of the commit and eviction kernels.
#include "gdn_launch.cuh"
#include "kv_book.cuh"
#include "kv_dispatch.h"

namespace gdn {

cudaError_t launch_kv_commit(const KvArgs& a, bool vec, cudaStream_t stream) {
    // the longest path's pieces, and what a thread's index passes them by
    const int64_t pieces = 2ll * a.P * a.Hkv * (a.d * dtype_size(a.dtype) / (vec ? 16 : 2));
    const bool wide = pieces > 0x7fffffff - KV_COMMIT_NT * KV_COMMIT_AHEAD;
    auto kern = vec ? (wide ? kv_commit_kernel<uint4, int64_t> : kv_commit_kernel<uint4, int>)
                    : (wide ? kv_commit_kernel<uint16_t, int64_t> : kv_commit_kernel<uint16_t, int>);
    kern<<<(unsigned)a.B, KV_COMMIT_NT, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_evict(const KvArgs& a, int cap, bool vec, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.Hkv, room = (int64_t)a.max_pages * a.page_size;
    if (units > 0x7fffffff / 8) return cudaErrorInvalidConfiguration;
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    // CTAs a unit: as many as keep every SM at one or two, with no less than 1024 entries each
    int C = 1;
    while (C < 8 && units * C * 2 <= 2 * di.sms && room / (C * 2) >= 1024) C *= 2;
    const int64_t words = ((room + C - 1) / C + 7) / 4 * 4, most = 45 * 1024;
    const int keys_cap = (int)(words < most ? words : most);
    const int smem = (int)sizeof(KvSelect) + keys_cap * 4;
    int bps = 0;
    if ((e = prepare_kernel(kv_select_kernel, KV_SEL_NT, smem, bps)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * C)), cfg.blockDim = dim3(KV_SEL_NT), cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    const bool vec4 = a.page_size % 4 == 0 && reinterpret_cast<uintptr_t>(a.weights) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.stamps) % 16 == 0;
    if ((e = cudaLaunchKernelEx(&cfg, kv_select_kernel, a, cap, keys_cap, (int)vec4)) != cudaSuccess) return e;

    // enough CTAs that the rows of few units still spread over the device
    const int64_t want = (1024 + units - 1) / units, rows = (cap + 31) / 32;  // four moves a warp at least
    const int esz = dtype_size(a.dtype), piece = vec ? 16 : 2, pieces = 2 * a.d * esz / piece;
    cudaLaunchConfig_t mv{};
    mv.gridDim = dim3((unsigned)units, (unsigned)(want < rows ? want : rows)), mv.blockDim = dim3(KV_MOVE_NT);
    mv.stream = stream;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    mv.attrs = &pdl, mv.numAttrs = 1;
    const uint32_t magic = (uint32_t)(((1ull << 32) + pieces - 1) / pieces);
    return cudaLaunchKernelEx(&mv, kv_move_kernel, a, cap, piece, pieces, magic);
}

}  // namespace gdn
