// kv_weights.cuh -- accumulation of attention weight per cache entry on the
// FP32 pipe (any cache dtype, head size, page size and stride; the tensor-core
// kernel takes the 16-bit caches whose copies it can address).
//
// Mathematics. With the rows' log-sum-exps known, entry e gathers
// sum_r e^(scale q_r.k_e - lse_r): no maximum, no order between tiles. Every
// entry of a key head belongs to one thread's sum, so no atomics and one order
// of additions. Shape: 128 threads, tiles of 64 keys in a ring of three buffers
// (as kv_attn.cuh), blocks of 32 rows (16 of the largest heads, beside whose ring
// 32 do not fit); longer paths take their blocks one after another over the CTA's
// tiles. One token's weights over 8 sequences of up to 4096 fp32 entries (32 / 8
// heads, d = 128): 49 us, 1.8 TB/s; three tokens' 75 us: bound by latency and
// shared-memory loads.
#pragma once

#include "kv_attn.cuh"

namespace gdn {

namespace kvgw {

using kvg::BUFS;
using kvg::KT;
using kvg::NT;
constexpr int RB = 32;

struct Layout {
    int dp, pitch, rb, off_q, off_sum, off_row, off_at, off_scan, bytes;
};
__host__ __device__ inline Layout layout(int d) {
    Layout L;
    L.dp = align_up(d, 4), L.pitch = L.dp + 4;
    L.rb = d <= 192 ? RB : RB / 2;
    L.off_q = BUFS * KT * L.pitch * 4;
    L.off_sum = L.off_q + L.rb * L.dp * 4;
    L.off_row = L.off_sum + 4 * KT * 4;
    L.off_at = L.off_row + RB * 16;
    L.off_scan = L.off_at + 2 * KT * 8;
    L.bytes = L.off_scan + (int)sizeof(KvScan<NT>);
    return L;
}

}  // namespace kvgw

// Rows of the accepted path: row r is node path[b][r / G], head r % G of the group. Its last seen entry
// is len - n + r / G.
template <typename ST>
__global__ void __launch_bounds__(kvg::NT) kv_weights_kernel(const __grid_constant__ KvArgs a, const int vec) {
    using namespace kvgw;
    extern __shared__ __align__(128) unsigned char smem[];
    const Layout L = layout(a.d);
    float* ring = reinterpret_cast<float*>(smem);
    float* sq = reinterpret_cast<float*>(smem + L.off_q);
    float* sum = reinterpret_cast<float*>(smem + L.off_sum);  // [4 warps][KT]
    int64_t* q_at = reinterpret_cast<int64_t*>(smem + L.off_row);
    float* slse = reinterpret_cast<float*>(q_at + RB);
    int64_t* at = reinterpret_cast<int64_t*>(smem + L.off_at);  // [2 tiles][KT]
    KvScan<NT>& scan = *reinterpret_cast<KvScan<NT>*>(smem + L.off_scan);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const KvSeq s = kv_seq<false>(a, b);
        if (s.err && tid == 0) set_error(a.dev_err, s.err);
    }
    const KvSplit split = kv_locate<false, KT, NT>(a, scan, gridDim.x, 1);
    bool some;
    KvWalk<false, KT> w(a, split, scan, some);
    if (!some) return;
    int checked = -1;
    bool ok = true;
    do {
        const KvSeq& s = w.s;
        const int b = w.b, h = w.h;
        const int32_t* table = a.page_table + (int64_t)s.slot * a.max_pages;
        if (checked != b) {
            const bool pages_ok = kv_pages_ok(a, s, tid, NT);
            const bool nodes_ok = tid >= s.nodes || (uint32_t)a.path[(int64_t)b * a.P + tid] < (uint32_t)a.T;
            if (!pages_ok || !nodes_ok) set_error(a.dev_err, (nodes_ok ? 0 : KV_DEVERR_NODES) | (pages_ok ? 0 : KV_DEVERR_PAGE));
            ok = __syncthreads_and(pages_ok && nodes_ok);
            checked = b;
        }
        const int rows_all = s.nodes * a.G, loads = ok ? w.t1 - w.t0 : 0;
        const auto place_rows = [&](int t) {
            if (tid < KT && t < w.t1 && t * KT + tid < s.len) {
                const int e = t * KT + tid, pg = e / a.page_size;
                at[(t & 1) * KT + tid] = kv_at(a.k, table[pg], h, e - pg * a.page_size);
            }
        };
        const auto load = [&](int i) {
            if (i < loads) {
                const int t = w.t0 + i;
                const int64_t* off = at + (t & 1) * KT;
                kv_load_rows<ST, NT>(ring + (i % BUFS) * KT * L.pitch, L.pitch, L.dp, KT, min(KT, s.len - t * KT), a.k.p, a.d,
                                     vec, [&](int r) { return off[r]; });
            }
            cp_async_commit();
        };
        for (int r0 = 0; r0 < rows_all && ok; r0 += L.rb) {
            const int rows = min(L.rb, rows_all - r0);
            __syncthreads();  // the last block is read
            if (tid < RB) {
                const int r = r0 + min(tid, rows - 1), j = r / a.G, hq = h * a.G + r - j * a.G;
                const int node = a.path[(int64_t)b * a.P + j];
                q_at[tid] = (int64_t)b * a.q.seq + (int64_t)node * a.q.node + (int64_t)hq * a.q.head;
                slse[tid] = tid < rows ? a.lse_in[((int64_t)b * a.T + node) * a.Hq + hq] : -INFINITY;
            }
            place_rows(w.t0), place_rows(w.t0 + 1);
            __syncthreads();
            kv_load_rows<ST, NT>(sq, L.dp, L.dp, L.rb, rows, a.q.p, a.d, vec, [&](int r) { return q_at[r]; });
            load(0), load(1);
            for (int i = 0; i < loads; ++i) {
                const int t = w.t0 + i, e0 = t * KT, n = min(KT, s.len - e0);
                float* x = a.weights;
                float old = 0.f;
                if (tid < n) {
                    const int e = e0 + tid, pg = e / a.page_size;
                    x += ((int64_t)table[pg] * a.Hkv + h) * a.page_size + (e - pg * a.page_size);
                    old = *x;
                }
                cp_async_wait<1>();
                __syncthreads();  // load i is there for everyone; the buffer and the sums of tile i - 1 are read
                place_rows(t + 2);
                const float *k0 = ring + (i % BUFS) * KT * L.pitch + lane * L.pitch, *k1 = k0 + 32 * L.pitch;
                float add[2] = {0.f, 0.f};
                const auto weigh = [&](float dot, int r, int key) {  // row r of the block, a key of the tile
                    const float lse = slse[r];
                    const int last = s.len - s.nodes + (r0 + r) / a.G;  // the row's own entry
                    // the exponent is formed before it is scaled to base 2: a weight near one keeps a small one
                    return e0 + key <= last && lse != -INFINITY ? kv_ex2(fmaf(dot, a.scale, -lse) * LOG2E) : 0.f;
                };
                if (rows <= 4) {  // two threads a key: the rows of one token would leave three warps idle
                    float acc[4] = {};
                    const int key = tid >> 1;
                    const float* k = ring + ((i % BUFS) * KT + key) * L.pitch;
#pragma unroll 2
                    for (int e = 4 * (tid & 1); e < L.dp; e += 8) {
                        const float4 y = *reinterpret_cast<const float4*>(k + e);
#pragma unroll
                        for (int r = 0; r < 4; ++r) kv_dot4(acc[r], y, *reinterpret_cast<const float4*>(sq + r * L.dp + e));
                    }
                    float x = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) x += weigh(acc[r] + __shfl_xor_sync(FULL_MASK, acc[r], 1), r, key);
                    if ((tid & 1) == 0) sum[key] = x, sum[KT + key] = 0.f, sum[2 * KT + key] = 0.f, sum[3 * KT + key] = 0.f;
                } else {
#pragma unroll 1
                    for (int rq = warp * 4; rq < rows; rq += 16) {
                        float acc[2][4] = {};
                        const float* q = sq + rq * L.dp;
#pragma unroll 2
                        for (int e = 0; e < L.dp; e += 4) {
                            const float4 y = *reinterpret_cast<const float4*>(k0 + e);
                            const float4 z = *reinterpret_cast<const float4*>(k1 + e);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float4 u = *reinterpret_cast<const float4*>(q + r * L.dp + e);
                                kv_dot4(acc[0][r], y, u), kv_dot4(acc[1][r], z, u);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            add[0] += weigh(acc[0][r], rq + r, lane), add[1] += weigh(acc[1][r], rq + r, lane + 32);
                    }
                    sum[warp * KT + lane] = add[0], sum[warp * KT + 32 + lane] = add[1];
                }
                __syncthreads();
                load(i + 2);  // (its rows were placed before the last barrier)
                if (tid < n)
                    *x = fmaf(old, r0 == 0 ? a.decay : 1.f, sum[tid] + sum[KT + tid] + sum[2 * KT + tid] + sum[3 * KT + tid]);
            }
            cp_async_wait<0>();
        }
    } while (w.next());
}

}  // namespace gdn
