// Instantiations and launch of the tensor-core accumulation kernel.
#include "gdn_launch.cuh"
#include "kv_dispatch.h"
#include "kv_maps.h"
#include "kv_weights_tc.cuh"

namespace gdn {

namespace {

template <typename ST, int NR>
cudaError_t launch(const KvArgs& a, const CUtensorMap& map, cudaStream_t stream) {
    auto kern = kv_weights_tc_kernel<ST, NR>;
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    const int boxes = boxes_of(a.d), one = (boxes > 1 ? 2 : 1) * kvt::BOX_BYTES;
    int stages = (di.smem_optin - kvw::smem_bytes<NR>(boxes, 0)) / one;
    if (stages > kvt::MAX_STAGES) stages = kvt::MAX_STAGES;
    const int smem = kvw::smem_bytes<NR>(boxes, stages);
    int bps = 0;
    if ((e = prepare_kernel(kern, kvw::NT, smem, bps)) != cudaSuccess) return e;
    const int64_t cap = (int64_t)a.max_pages * a.page_size, most = (int64_t)a.B * a.Hkv * ((cap + kvt::KT - 1) / kvt::KT);
    const int grid = (int)(most < 1 ? 1 : most < di.sms ? most : di.sms);
    kern<<<grid, kvw::NT, smem, stream>>>(a, map, boxes, stages, box_rows_of(a.page_size));
    return cudaGetLastError();
}

template <typename ST>
cudaError_t launch_rows(const KvArgs& a, const CUtensorMap& map, cudaStream_t s) {
    const int64_t rows = (int64_t)a.P * a.G;
    const int most = boxes_of(a.d) > 2 ? 64 : 128;  // the queries of four boxes leave the ring short at 128
    if (rows <= 16) return launch<ST, 16>(a, map, s);
    if (rows <= 32) return launch<ST, 32>(a, map, s);
    if (rows <= 64 || most == 64) return launch<ST, 64>(a, map, s);
    return launch<ST, 128>(a, map, s);
}

}  // namespace

cudaError_t launch_kv_weights_tc(const KvArgs& a, cudaStream_t stream) {
    CUtensorMap map;
    if (!encoder() || !encode(map, a.dtype, a.k.p, a.d, a.page_size, a.k.token, a.Hkv, a.k.head, a.num_pages, a.k.page,
                              box_rows_of(a.page_size)))
        return cudaErrorNotSupported;
    return a.dtype == GDN_BF16 ? launch_rows<__nv_bfloat16>(a, map, stream) : launch_rows<__half>(a, map, stream);
}

}  // namespace gdn
