// Instantiations and launches of the FP32-pipe attention and accumulation kernels, by cache dtype.
#include "gdn_launch.cuh"
#include "kv_attn.cuh"
#include "kv_dispatch.h"
#include "kv_weights.cuh"

namespace gdn {

namespace {

using Kernel = void (*)(const KvArgs, const int);

template <int RB>
Kernel attn_kernel(int dtype) {
    return dtype == GDN_F32 ? kv_attn_kernel<float, RB>
                            : dtype == GDN_BF16 ? kv_attn_kernel<__nv_bfloat16, RB> : kv_attn_kernel<__half, RB>;
}

Kernel weights_kernel(int dtype) {
    return dtype == GDN_F32 ? kv_weights_kernel<float>
                            : dtype == GDN_BF16 ? kv_weights_kernel<__nv_bfloat16> : kv_weights_kernel<__half>;
}

// The kernel of a call, and what it takes.
struct Choice {
    Kernel kern;
    int smem;
};
// Units of 4 rows where there are no more: a decode step of up to four heads a group.
Choice choose(KvArgs& a) {
    a.row_block = a.T * a.G <= 4 ? 4 : 16;
    if (a.row_block == 4) return {attn_kernel<4>(a.dtype), kvg::layout<4>(a.d).bytes};
    return {attn_kernel<16>(a.dtype), kvg::layout<16>(a.d).bytes};
}

// CTAs of a call: one wave, and no more than the longest cache could feed.
cudaError_t wave(Kernel kern, const KvArgs& a, int smem, int64_t& grid) {
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    int bps = 0;
    if ((e = prepare_kernel(kern, kvg::NT, smem, bps)) != cudaSuccess) return e;
    grid = (int64_t)di.sms * bps;
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    const int64_t blocks = ((int64_t)a.T * a.G + a.row_block - 1) / a.row_block;
    const int64_t most = (int64_t)a.B * a.Hkv * blocks * ((cap + kvg::KT - 1) / kvg::KT + 1);
    if (grid > most) grid = most;
    if (grid < 1) grid = 1;
    return cudaSuccess;
}

}  // namespace

cudaError_t kv_attn_workspace(KvArgs& a, int64_t& bytes) {
    int64_t grid = 0;
    const Choice c = choose(a);
    const cudaError_t e = wave(c.kern, a, c.smem, grid);
    bytes = kv_part_bytes(grid, a.row_block, a.d) + grid * (int64_t)sizeof(KvBorder);
    return e;
}

cudaError_t launch_kv_attn(KvArgs& a, bool vec, cudaStream_t stream) {
    int64_t grid = 0;
    const Choice c = choose(a);
    cudaError_t e = wave(c.kern, a, c.smem, grid);
    if (e != cudaSuccess) return e;
    a.border = reinterpret_cast<char*>(a.part) + kv_part_bytes(grid, a.row_block, a.d);
    c.kern<<<(unsigned)grid, kvg::NT, c.smem, stream>>>(a, vec);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_kv_join(a, (int)grid, stream);
}

cudaError_t launch_kv_weights(KvArgs& a, bool vec, cudaStream_t stream) {
    const int smem = kvgw::layout(a.d).bytes;
    int64_t grid = 0;
    a.row_block = kvgw::RB;
    cudaError_t e = wave(weights_kernel(a.dtype), a, smem, grid);
    if (e != cudaSuccess) return e;
    weights_kernel(a.dtype)<<<(unsigned)grid, kvg::NT, smem, stream>>>(a, vec);
    return cudaGetLastError();
}

}  // namespace gdn
