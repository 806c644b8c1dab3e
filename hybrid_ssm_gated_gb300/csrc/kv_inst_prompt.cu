// Instantiations and launches of the prompt attention on the FP32 pipe, and of its join.
#include "gdn_launch.cuh"
#include "kv_dispatch.h"
#include "kv_prompt_fp32.cuh"
#include "kv_prompt_join.cuh"

namespace gdn {

namespace {

using Kernel = void (*)(const KvArgs, const int);

// Blocks of 64 outputs, and whether up to 16 more are left over. (16-bit caches come here with odd sizes and
// strides alone: for them the next whole block does.)
template <int NC, bool TAIL>
Kernel of_f32() {
    return kv_prompt_kernel<float, NC, TAIL>;
}
template <typename ST>
Kernel of_16(int d) {
    return d <= 64 ? kv_prompt_kernel<ST, 1, false> : d <= 128 ? kv_prompt_kernel<ST, 2, false> : kv_prompt_kernel<ST, 4, false>;
}
Kernel choose(const KvArgs& a) {
    if (a.dtype == GDN_BF16) return of_16<__nv_bfloat16>(a.d);
    if (a.dtype == GDN_F16) return of_16<__half>(a.d);
    static const Kernel kernels[5][2] = {{of_f32<0, true>(), of_f32<0, true>()}, {of_f32<1, false>(), of_f32<1, true>()},
                                         {of_f32<2, false>(), of_f32<2, true>()}, {of_f32<3, false>(), of_f32<3, true>()},
                                         {of_f32<4, false>(), of_f32<4, false>()}};
    const int left = a.d % 64;
    return left > 16 ? kernels[a.d / 64 + 1][0] : kernels[a.d / 64][left > 0];
}

cudaError_t wave(const KvArgs& a, int64_t& grid) {
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    int bps = 0;
    if ((e = prepare_kernel(choose(a), kpg::NT, kpg::layout(a.d).bytes, bps)) != cudaSuccess) return e;
    grid = (int64_t)di.sms * bps;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_kp_join(const KvArgs& a, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(grid * kpj::share(a.part_rows, a.d))), cfg.blockDim = dim3(kpj::NT), cfg.stream = stream;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kp_join_kernel, a);
}

cudaError_t kv_prompt_workspace(KvArgs& a, int64_t& bytes) {
    int64_t grid = 0;
    const cudaError_t e = wave(a, grid);
    bytes = kp_part_bytes(grid, kpg::RB, a.d) + grid * (int64_t)sizeof(KpBorder);
    return e;
}

cudaError_t launch_kv_prompt(KvArgs& a, bool vec, cudaStream_t stream) {
    int64_t grid = 0;
    a.extra = 128, a.least = 256;  // (two tiles; over 64 + 64)
    a.row_block = a.tile_rows = a.tile_places = a.part_rows = kpg::RB;
    cudaError_t e = wave(a, grid);
    if (e != cudaSuccess) return e;
    a.border = reinterpret_cast<char*>(a.part) + kp_part_bytes(grid, kpg::RB, a.d);
    choose(a)<<<(unsigned)grid, kpg::NT, kpg::layout(a.d).bytes, stream>>>(a, vec);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_kp_join(a, (int)grid, stream);
}

}  // namespace gdn
