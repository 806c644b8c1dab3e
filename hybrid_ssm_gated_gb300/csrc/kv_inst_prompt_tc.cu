// Instantiations and launch of the prompt attention on the tensor cores, and its tensor maps.
#include "gdn_launch.cuh"
#include "kv_dispatch.h"
#include "kv_maps.h"
#include "kv_prompt_tc.cuh"

namespace gdn {

namespace {

template <typename ST, int QT>
cudaError_t launch(const KvArgs& a, const kpt::Maps& maps, int boxes, int box_rows, const DeviceInfo& di, cudaStream_t stream) {
    auto kern = kv_prompt_tc_kernel<ST, QT>;
    int stages = (di.smem_optin - kpt::smem_bytes<QT>(boxes, 0)) / kpt::stage_bytes<QT>(boxes);
    if (stages > kpt::MAX_STAGES) stages = kpt::MAX_STAGES;
    // V waits for the weights: it gets the odd stage
    const int k_stages = stages / 2, v_stages = stages - k_stages, smem = kpt::smem_bytes<QT>(boxes, stages);
    int bps = 0;
    cudaError_t e = prepare_kernel(kern, kpt::threads(QT), smem, bps);
    if (e != cudaSuccess) return e;
    kern<<<di.sms, kpt::threads(QT), smem, stream>>>(a, maps, boxes, k_stages, v_stages, box_rows);
    return cudaGetLastError();
}

// Tiles of query rows a unit: two where their outputs fit tensor memory, there are units for every SM, and the sequences
// have rows for them in the mean. (32 / 8 heads, d = 128: 2048 tokens, 256 units of two tiles, take 61 us so and 70 with
// one; 1024 tokens, 128 such units, 35.3 and 34.9; 512 tokens, 64, 25 and 22.)
int tiles_of(const KvArgs& a, int sms) {
    if (a.d > 128) return 1;
    const int64_t tokens = 2 * (kpt::TILE / a.G);
    const int64_t units = a.total / tokens;
    return units * a.Hkv >= sms && units >= a.B ? 2 : 1;
}

}  // namespace

bool kv_prompt_tc_fits(const KvArgs& a) {
    return a.dtype != GDN_F32 && a.d % 8 == 0 && box_rows_of(a.page_size) > 0 && a.num_pages > 0 && a.G <= kpt::TILE;
}

cudaError_t kv_prompt_tc_workspace(KvArgs& a, int64_t& bytes) {
    DeviceInfo di;
    const cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    // (of the larger form: a smaller call may take either)
    const int places = (a.d > 128 ? 1 : 2) * kpt::TILE;
    bytes = kp_part_bytes(di.sms, places, a.d) + di.sms * (int64_t)sizeof(KpBorder);
    return cudaSuccess;
}

cudaError_t launch_kv_prompt_tc(KvArgs& a, cudaStream_t stream) {
    const int boxes = boxes_of(a.d), tokens = kpt::TILE / a.G;
    if (a.total == 0) return cudaErrorNotSupported;  // (no row to describe)
    DeviceInfo di;
    cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    const int QT = tiles_of(a, di.sms), keys = kpt::keys_of(QT), most = box_rows_of(a.page_size), box_rows = most < keys ? most : keys;
    kpt::Maps maps{};
    if (!encoder() ||
        !encode(maps.k, a.dtype, a.k.p, a.d, a.page_size, a.k.token, a.Hkv, a.k.head, a.num_pages, a.k.page, box_rows) ||
        !encode(maps.v, a.dtype, a.v.p, a.d, a.page_size, a.v.token, a.Hkv, a.v.head, a.num_pages, a.v.page, box_rows) ||
        !encode(maps.q, a.dtype, a.q.p, a.d, a.Hq, a.q.head, a.total, a.q.node, 1, a.d, a.G, tokens))
        return cudaErrorNotSupported;
    a.extra = QT == 2 ? 512 : 384;  // (measured: 9 us where a tile of 128 takes 2, 5 to 6 where one of 64 takes 1)
    a.least = QT == 2 ? 512 : 256;  // (over 128 + 256, 64 + 128)
    a.tile_rows = tokens * a.G, a.tile_places = kpt::TILE, a.row_block = QT * a.tile_rows, a.part_rows = QT * kpt::TILE;
    a.border = reinterpret_cast<char*>(a.part) + kp_part_bytes(di.sms, a.part_rows, a.d);
    if (a.dtype == GDN_BF16)
        e = QT == 2 ? launch<__nv_bfloat16, 2>(a, maps, boxes, box_rows, di, stream)
                    : launch<__nv_bfloat16, 1>(a, maps, boxes, box_rows, di, stream);
    else
        e = QT == 2 ? launch<__half, 2>(a, maps, boxes, box_rows, di, stream)
                    : launch<__half, 1>(a, maps, boxes, box_rows, di, stream);
    if (e != cudaSuccess) return e;
    return launch_kp_join(a, di.sms, stream);
}

}  // namespace gdn
