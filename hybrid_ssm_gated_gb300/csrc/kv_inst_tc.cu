// Instantiations and launch of the tensor-core attention kernel, and its tensor maps.
#include "gdn_launch.cuh"
#include "kv_dispatch.h"
#include "kv_maps.h"
#include "kv_tc.cuh"

namespace gdn {

namespace {

// Query rows a unit: the smallest block that holds them all, up to 128 (64 where d has two halves: at 128
// their outputs, the folds of these and the scores are more than tensor memory's 512 columns, and shared memory
// would leave the rings one tile each).
int row_block_of(int64_t rows, int boxes) {
    const int most = boxes > 2 ? 64 : 128;
    int nr = 16;
    while (nr < rows && nr < most) nr *= 2;
    return nr;
}

template <typename ST, int NR>
cudaError_t launch(KvArgs& a, const kvt::Maps& maps, int boxes, int box_rows, int grid, int optin, cudaStream_t stream) {
    auto kern = kv_attn_tc_kernel<ST, NR>;
    // stages that fit beside two weight buffers, or beside one where that gives a stage more
    const int one = (boxes > 1 ? 2 : 1) * kvt::BOX_BYTES;
    const auto fit = [&](int bufs) {
        const int n = (optin - kvt::smem_bytes<NR>(boxes, bufs, 0)) / one;
        return n < kvt::MAX_STAGES ? n : kvt::MAX_STAGES;
    };
    const int p_bufs = fit(1) > fit(2) && fit(2) < 6 ? 1 : 2, stages = fit(p_bufs);
    // V waits for the weights: it gets the odd stage
    const int k_stages = stages / 2, v_stages = stages - k_stages, smem = kvt::smem_bytes<NR>(boxes, p_bufs, stages);
    int bps = 0;
    cudaError_t e = prepare_kernel(kern, kvt::threads(NR), smem, bps);
    if (e != cudaSuccess) return e;
    kern<<<grid, kvt::threads(NR), smem, stream>>>(a, maps, boxes, k_stages, v_stages, p_bufs, box_rows);
    return cudaGetLastError();
}

template <typename ST>
cudaError_t launch_rows(KvArgs& a, const kvt::Maps& maps, int boxes, int box_rows, int grid, int optin, cudaStream_t s) {
    switch (a.row_block) {
        case 16: return launch<ST, 16>(a, maps, boxes, box_rows, grid, optin, s);
        case 32: return launch<ST, 32>(a, maps, boxes, box_rows, grid, optin, s);
        case 64: return launch<ST, 64>(a, maps, boxes, box_rows, grid, optin, s);
        default: return launch<ST, 128>(a, maps, boxes, box_rows, grid, optin, s);
    }
}

cudaError_t wave(const KvArgs& a, DeviceInfo& di, int64_t& grid) {
    const cudaError_t e = device_info(di);
    if (e != cudaSuccess) return e;
    const int64_t cap = (int64_t)a.max_pages * a.page_size, blocks = ((int64_t)a.T * a.G + a.row_block - 1) / a.row_block;
    const int64_t most = (int64_t)a.B * a.Hkv * blocks * ((cap + kvt::KT - 1) / kvt::KT + 1);
    grid = di.sms < most ? di.sms : most;
    if (grid < 1) grid = 1;
    return cudaSuccess;
}

}  // namespace

bool kv_tc_fits(const KvArgs& a) {
    return a.dtype != GDN_F32 && a.d % 8 == 0 && box_rows_of(a.page_size) > 0 && a.num_pages > 0;
}

cudaError_t kv_attn_tc_workspace(KvArgs& a, int64_t& bytes) {
    DeviceInfo di;
    int64_t grid = 0;
    a.row_block = row_block_of((int64_t)a.T * a.G, boxes_of(a.d));
    const cudaError_t e = wave(a, di, grid);
    bytes = kv_part_bytes(grid, a.row_block, a.d) + grid * (int64_t)sizeof(KvBorder);
    return e;
}

cudaError_t launch_kv_attn_tc(KvArgs& a, cudaStream_t stream) {
    const int boxes = boxes_of(a.d), box_rows = box_rows_of(a.page_size);
    kvt::Maps maps{};
    if (!encoder() ||
        !encode(maps.k, a.dtype, a.k.p, a.d, a.page_size, a.k.token, a.Hkv, a.k.head, a.num_pages, a.k.page, box_rows) ||
        !encode(maps.v, a.dtype, a.v.p, a.d, a.page_size, a.v.token, a.Hkv, a.v.head, a.num_pages, a.v.page, box_rows) ||
        !encode(maps.kn, a.dtype, a.kn.p, a.d, a.T, a.kn.node, a.Hkv, a.kn.head, a.B, a.kn.seq, a.T) ||
        !encode(maps.vn, a.dtype, a.vn.p, a.d, a.T, a.vn.node, a.Hkv, a.vn.head, a.B, a.vn.seq, a.T))
        return cudaErrorNotSupported;
    a.row_block = row_block_of((int64_t)a.T * a.G, boxes);
    // queries: a block of rows is whole nodes' heads of one group
    if (a.row_block % a.G == 0 &&
        !encode(maps.q, a.dtype, a.q.p, a.d, a.Hq, a.q.head, a.T, a.q.node, a.B, a.q.seq, a.G, a.row_block / a.G))
        return cudaErrorNotSupported;
    DeviceInfo di;
    int64_t grid = 0;
    cudaError_t e = wave(a, di, grid);
    if (e != cudaSuccess) return e;
    a.border = reinterpret_cast<char*>(a.part) + kv_part_bytes(grid, a.row_block, a.d);
    e = a.dtype == GDN_BF16 ? launch_rows<__nv_bfloat16>(a, maps, boxes, box_rows, (int)grid, di.smem_optin, stream)
                            : launch_rows<__half>(a, maps, boxes, box_rows, (int)grid, di.smem_optin, stream);
    if (e != cudaSuccess) return e;
    return launch_kv_join(a, (int)grid, stream);
}

}  // namespace gdn
