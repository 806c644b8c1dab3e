// Launches of the commit and eviction kernels.
#include "kv_book.cuh"
#include "kv_dispatch.h"

namespace gdn {

cudaError_t launch_kv_commit(const KvArgs& a, bool vec, cudaStream_t stream) {
    kv_commit_kernel<<<(unsigned)a.B, KV_COMMIT_NT, 0, stream>>>(a, vec);
    return cudaGetLastError();
}

cudaError_t launch_kv_evict(const KvArgs& a, int cap, bool vec, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.Hkv;
    if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv_select_kernel<<<(unsigned)units, KV_SEL_NT, 0, stream>>>(a, cap);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // enough CTAs that the rows of few units still spread over the device
    const int64_t want = (1024 + units - 1) / units, rows = (cap + 7) / 8;
    const dim3 grid((unsigned)units, (unsigned)(want < rows ? want : rows));
    kv_move_kernel<<<grid, KV_MOVE_NT, 0, stream>>>(a, cap, vec);
    return cudaGetLastError();
}

}  // namespace gdn
