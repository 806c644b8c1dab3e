// Launches of the fork and compaction kernels.
#include "gdn_launch.cuh"
#include "kv_dispatch.h"
#include "kv_share.cuh"

namespace gdn {

cudaError_t launch_kv_fork(const KvArgs& a, const int32_t* src, const int32_t* dst, const int32_t* new_pages, bool vec,
                           cudaStream_t stream) {
    DeviceInfo di;
    const cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    // blocks a fork: eight a SM over all of them, and no more than there are jobs
    const int64_t jobs = (int64_t)a.max_pages * a.Hkv, want = ((int64_t)di.sms * 8 + a.B - 1) / a.B;
    int64_t x = jobs < want ? jobs : want;
    if (x < 1) x = 1;
    auto kern = vec ? kv_fork_kernel<uint4> : kv_fork_kernel<uint16_t>;
    for (int b = 0; b < a.B; b += 65535) {  // (a grid's second dimension)
        const int n = a.B - b < 65535 ? a.B - b : 65535;
        kern<<<dim3((unsigned)x, (unsigned)n), kvs::NT, 0, stream>>>(a, src + b, dst + b, new_pages + (int64_t)b * a.max_pages);
        const cudaError_t r = cudaGetLastError();
        if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
}

namespace {

template <typename... P, typename... A>
cudaError_t behind(void (*kern)(P...), int64_t grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid), cfg.blockDim = dim3(threads), cfg.stream = stream;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_kv_compact(const KvArgs& a, int32_t* ws, int32_t* used, bool vec, cudaStream_t stream) {
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    const KvPlan p = kv_plan(ws, a.num_pages);
    const auto most = [&](int64_t blocks, int64_t per_sm) {
        const int64_t top = (int64_t)di.sms * per_sm;
        return blocks < 1 ? 1 : blocks < top ? blocks : top;
    };
    const int64_t slots = (a.num_slots + kvs::NT / 32 - 1) / (kvs::NT / 32);
    if (a.num_pages <= KV_SMALL_PAGES && a.num_slots * a.max_pages <= KV_SMALL_ENTRIES) {
        kv_plan_kernel<true><<<1, kvs::PLAN_NT, 0, stream>>>(a, p, used);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    } else {
        kv_clear_kernel<<<(unsigned)most((p.words + 8 + kvs::NT - 1) / kvs::NT, 4), kvs::NT, 0, stream>>>(ws, p.words);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = behind(kv_mark_kernel, most(slots, 4), kvs::NT, stream, a, p)) != cudaSuccess) return e;
        if ((e = behind(kv_plan_kernel<false>, 1, kvs::PLAN_NT, stream, a, p, used)) != cudaSuccess) return e;
    }
    // (no more than half of the pages can move)
    const int copiers = (int)most(a.num_pages / 2 * a.Hkv, 7), tables = (int)most(slots, 1);
    return behind(vec ? kv_pages_kernel<uint4> : kv_pages_kernel<uint16_t>, copiers + tables, kvs::NT, stream, a, p, copiers);
}

}  // namespace gdn
