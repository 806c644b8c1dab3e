// Instantiations and launches of the FP32-pipe attention and accumulation kernels, one a cache dtype.
#include "gdn_launch.cuh"
#include "kv_attn.cuh"
#include "kv_dispatch.h"
#include "kv_weights.cuh"

namespace gdn {

namespace {

using Kernel = void (*)(const KvArgs, const int);

Kernel attn_kernel(int dtype) {
    return dtype == GDN_F32 ? kv_attn_kernel<float> : dtype == GDN_BF16 ? kv_attn_kernel<__nv_bfloat16> : kv_attn_kernel<__half>;
}

Kernel weights_kernel(int dtype) {
    return dtype == GDN_F32 ? kv_weights_kernel<float>
                            : dtype == GDN_BF16 ? kv_weights_kernel<__nv_bfloat16> : kv_weights_kernel<__half>;
}

// CTAs of a call: one wave, and no more than the longest cache could feed.
cudaError_t wave(Kernel kern, const KvArgs& a, int smem, int least, int64_t& grid) {
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    int bps = 0;
    if ((e = prepare_kernel(kern, kvg::NT, smem, bps)) != cudaSuccess) return e;
    grid = (int64_t)di.sms * bps;
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    const int64_t blocks = ((int64_t)a.T * a.G + a.row_block - 1) / a.row_block;
    const int64_t most = (int64_t)a.B * a.Hkv * blocks * ((cap + kvg::KT - 1) / kvg::KT + 1) / least;
    if (grid > most) grid = most;
    if (grid < 1) grid = 1;
    return cudaSuccess;
}

}  // namespace

cudaError_t kv_attn_workspace(KvArgs& a, int64_t& bytes) {
    int64_t grid = 0;
    a.row_block = kvg::RB;
    const cudaError_t e = wave(attn_kernel(a.dtype), a, kvg::layout(a.d).bytes, kvg::LEAST, grid);
    bytes = kv_part_bytes(grid, kvg::RB, a.d) + grid * (int64_t)sizeof(KvBorder);
    return e;
}

cudaError_t launch_kv_attn(KvArgs& a, bool vec, cudaStream_t stream) {
    const int smem = kvg::layout(a.d).bytes;
    int64_t grid = 0;
    a.row_block = kvg::RB;
    cudaError_t e = wave(attn_kernel(a.dtype), a, smem, kvg::LEAST, grid);
    if (e != cudaSuccess) return e;
    a.border = reinterpret_cast<char*>(a.part) + kv_part_bytes(grid, kvg::RB, a.d);
    attn_kernel(a.dtype)<<<(unsigned)grid, kvg::NT, smem, stream>>>(a, vec);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_kv_join(a, (int)grid, stream);
}

cudaError_t launch_kv_weights(KvArgs& a, bool vec, cudaStream_t stream) {
    const int smem = kvg::layout(a.d).bytes;
    int64_t grid = 0;
    cudaError_t e = wave(weights_kernel(a.dtype), a, smem, 1, grid);
    if (e != cudaSuccess) return e;
    weights_kernel(a.dtype)<<<(unsigned)grid, kvg::NT, smem, stream>>>(a, vec);
    return cudaGetLastError();
}

}  // namespace gdn
