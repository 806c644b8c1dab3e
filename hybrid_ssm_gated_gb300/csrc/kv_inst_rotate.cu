// Instantiations and launches of the norm, rotation and append kernels.
#include "gdn_launch.cuh"
#include "kv_dispatch.h"
#include "kv_rotate.cuh"

namespace gdn {

namespace {

using Kernel = void (*)(const KvRotateArgs, const KvArgs);

template <typename ST, bool APPEND>
Kernel of_lanes(int lanes) {
    switch (lanes) {
        case 8: return kv_rotate_kernel<ST, 8, APPEND>;
        case 16: return kv_rotate_kernel<ST, 16, APPEND>;
        case 32: return kv_rotate_kernel<ST, 32, APPEND>;
        default: return kv_rotate_kernel<ST, 0, APPEND>;
    }
}
template <bool APPEND>
Kernel choose(int dtype, int lanes) {
    return dtype == GDN_F32 ? of_lanes<float, APPEND>(lanes)
                            : dtype == GDN_BF16 ? of_lanes<__nv_bfloat16, APPEND>(lanes) : of_lanes<__half, APPEND>(lanes);
}

}  // namespace

cudaError_t launch_kv_rotate(KvRotateArgs& r, const KvArgs* cache, bool vec, cudaStream_t stream) {
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    // a lane's eight elements are turned alike: halves, or (interleaved) the whole turned part, in multiples of eight
    vec = vec && r.d % kvr::LANE == 0 && (r.interleaved ? r.rot : r.rot / 2) % kvr::LANE == 0;
    const int lanes = !vec ? 0 : r.d <= 64 ? 8 : r.d <= 128 ? 16 : 32;
    // tokens of a block: as many as leave the device four blocks a SM, so that their angles' cost is spread
    r.log_block = 0;
    const int groups = lanes ? kvr::NT / lanes : kvr::MAX_TOKENS;
    while (2 << r.log_block <= kvr::MAX_TOKENS && 2 << r.log_block <= groups && r.tokens >> (r.log_block + 1) >= di.sms * 4) ++r.log_block;
    const unsigned grid = (unsigned)((r.tokens + (1 << r.log_block) - 1) >> r.log_block);
    // tokens that one stride separates, of every row that is read and written
    const auto flat = [&](const KvTurn& t) { return cache || !t.in || (t.in_seq == r.T * t.in_node && t.out_seq == r.T * t.out_node); };
    if ((cache || r.T > 1) && flat(r.q) && flat(r.k)) {  // (an append's rows lie in strides of `node`)
        r.T = 1;
        for (KvTurn* t : {&r.q, &r.k, &r.v}) t->in_seq = t->in_node, t->out_seq = t->out_node;
    }
    if (!cache) {
        choose<false>(r.dtype, lanes)<<<grid, kvr::NT, 0, stream>>>(r, KvArgs{});
        return cudaGetLastError();
    }
    if (grid > 0) {
        choose<true>(r.dtype, lanes)<<<grid, kvr::NT, 0, stream>>>(r, *cache);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    const int warps = KV_GROW_NT / 32;
    cfg.gridDim = dim3((unsigned)((cache->B + warps - 1) / warps)), cfg.blockDim = dim3(KV_GROW_NT), cfg.stream = stream;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = grid > 0;
    cfg.attrs = &pdl, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_grow_kernel, *cache);
}

}  // namespace gdn
