// kv_weights.cuh -- accumulation of attention weight per cache entry on the
// FP32 pipe (any cache dtype, head size, page size and stride; the tensor-core
// kernel takes the 16-bit caches whose copies it can address).
//
// Mathematics. With the rows' log-sum-exps known, entry e gathers
// sum_r e^(scale q_r.k_e - lse_r): no maximum, no order between tiles. Every
// entry of a key head belongs to one thread's sum, so no atomics and one order
// of additions.
#pragma once

#include "kv_attn.cuh"

namespace gdn {

// Rows of the accepted path: row r is node path[b][r / G], head r % G of the group. Its last seen entry
// is len - n + r / G.
template <typename ST>
__global__ void __launch_bounds__(kvg::NT) kv_weights_kernel(const KvArgs a, const int vec) {
    using namespace kvg;
    extern __shared__ __align__(128) unsigned char smem[];
    const Layout L = layout(a.d);
    float* sq = reinterpret_cast<float*>(smem);
    float* sk = reinterpret_cast<float*>(smem + L.off_k);
    float* sp = reinterpret_cast<float*>(smem + L.off_p);  // sums [4][KT]
    float* slse = reinterpret_cast<float*>(smem + L.off_row);
    int* snode = reinterpret_cast<int*>(slse + RB);
    KvScan<NT>& scan = *reinterpret_cast<KvScan<NT>*>(smem + L.off_scan);
    const int tid = threadIdx.x;

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
            bool nodes_ok = true;
            for (int j = tid; j < s.nodes; j += NT) nodes_ok = nodes_ok && (uint32_t)a.path[(int64_t)b * a.P + j] < (uint32_t)a.T;
            nodes_ok = __syncthreads_and(nodes_ok);
            const bool pages_ok = __syncthreads_and(kv_pages_ok(a, s, tid, NT));
            ok = nodes_ok && pages_ok;
            if (!ok && tid == 0)
                set_error(a.dev_err, (nodes_ok ? 0 : KV_DEVERR_NODES) | (pages_ok ? 0 : KV_DEVERR_PAGE));
            checked = b;
        }
        for (int tile = w.t0; tile < w.t1 && ok; ++tile) {
            const int e0 = tile * KT, n = min(KT, s.len - e0), rows = s.nodes * a.G;
            const int key = tid & (KT - 1), g = tid / KT;
            __syncthreads();  // the last tile's sums and keys are read
            kv_load_rows<ST, NT>(sk, L.pitch, L.dp, KT, n, a.k.p, a.d, vec, [&](int r) {
                const int pg = (e0 + r) / a.page_size;
                return kv_at(a.k, table[pg], h, e0 + r - pg * a.page_size);
            });
            float sum = 0.f;
            for (int r0 = 0; r0 < rows; r0 += RB) {
                const int nr = min(RB, rows - r0);
                __syncthreads();  // the last block of rows is read
                if (tid < RB) {
                    const int j = min(r0 + tid, rows - 1) / a.G;
                    const int node = a.path[(int64_t)b * a.P + j];
                    const int hq = h * a.G + min(r0 + tid, rows - 1) - j * a.G;
                    snode[tid] = node;
                    slse[tid] = a.lse_in[((int64_t)b * a.T + node) * a.Hq + hq];
                }
                __syncthreads();
                kv_load_rows<ST, NT>(sq, L.dp, L.dp, RB, nr, a.q.p, a.d, vec, [&](int r) {
                    return (int64_t)b * a.q.seq + (int64_t)snode[r] * a.q.node +
                           (int64_t)(h * a.G + (r0 + r) % a.G) * a.q.head;
                });
                __syncthreads();
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                for (int e = 0; e < L.dp; e += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(sk + key * L.pitch + e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 y = *reinterpret_cast<const float4*>(sq + (4 * g + i) * L.dp + e);
                        acc[i] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc[i]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * g + i;
                    const float lse = slse[r];
                    // the exponent is formed before it is scaled to base 2: a weight near one keeps a small one
                    if (r < nr && e0 + key <= s.len - s.nodes + (r0 + r) / a.G && lse != -INFINITY)
                        sum += kv_ex2(fmaf(acc[i], a.scale, -lse) * LOG2E);
                }
            }
            sp[g * KT + key] = sum;
            __syncthreads();
            if (tid < n) {
                const int e = e0 + tid, pg = e / a.page_size;
                float* x = a.weights + ((int64_t)table[pg] * a.Hkv + h) * a.page_size + (e - pg * a.page_size);
                *x = fmaf(*x, a.decay, sp[tid] + sp[KT + tid] + sp[2 * KT + tid] + sp[3 * KT + tid]);
            }
        }
    } while (w.next());
}

}  // namespace gdn
