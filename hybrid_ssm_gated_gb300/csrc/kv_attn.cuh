// kv_attn.cuh -- attention of drafted nodes over the paged cache on the FP32
// pipe: any cache dtype, head size up to 256, page size and stride. It serves
// fp32 caches, whose scores and outputs keep FP32 products, and 16-bit caches
// that the tensor-core kernel's copies cannot address.
//
// Mathematics. One pass over the keys with a running maximum m and sum l a
// row (base-2 exponents): for a tile of scores s, m' = max(m, max s),
// l' = l 2^{m - m'} + sum 2^{s - m'}, O' = O 2^{m - m'} + sum 2^{s - m'} v; at
// the end out = O / l and lse = (m + log2 l) ln 2.
//
// Shape: 256 threads, units of up to 16 query rows (node-major: row = node *
// G + head of the group), tiles of 64 keys held in shared memory as FP32. A
// thread takes four rows of one key for the scores, and a run of four
// consecutive output elements of up to four rows for the products with the
// values.
#pragma once

#include "kv_common.cuh"

namespace gdn {

namespace kvg {

constexpr int KT = 64, RB = 16, NT = 256;
constexpr int LEAST = 2;  // tiles a CTA at least

struct Layout {
    int dp, pitch, off_k, off_v, off_p, off_row, off_mask, off_scan, bytes;
};
__host__ __device__ inline Layout layout(int d) {
    Layout L;
    L.dp = align_up(d, 4);
    L.pitch = L.dp + 4;  // keys of neighbouring lanes in distinct banks, 16 bytes at a time
    L.off_k = RB * L.dp * 4;
    L.off_v = L.off_k + KT * L.pitch * 4;
    L.off_p = L.off_v + KT * L.pitch * 4;
    L.off_row = L.off_p + RB * (KT + 4) * 4;
    L.off_mask = L.off_row + 3 * RB * 4;
    L.off_scan = L.off_mask + RB * 8;
    L.bytes = L.off_scan + (int)sizeof(KvScan<NT>);
    return L;
}

}  // namespace kvg

// Load `n` rows of d elements (row i at base + off(i), elements of type ST) into FP32 rows of `pitch`
// floats; the other rows and the padding of d are zero. vec: rows may be read 16 bytes at a time.
template <typename ST, int NT, typename Off>
__device__ __forceinline__ void kv_load_rows(float* dst, int pitch, int dp, int rows, int n, const void* base, int d,
                                             bool vec, Off off) {
    constexpr int VEC = Store<ST>::VEC;
    const ST* src = static_cast<const ST*>(base);
    if (vec) {  // d is a multiple of VEC: no padding
        const int per = d / VEC;
        for (int i = threadIdx.x; i < rows * per; i += NT) {
            const int r = i / per, c = (i - r * per) * VEC;
            float x[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = 0.f;
            if (r < n) Store<ST>::unpack(*reinterpret_cast<const uint4*>(src + off(r) + c), x);
#pragma unroll
            for (int e = 0; e < VEC; e += 4)
                *reinterpret_cast<float4*>(dst + r * pitch + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
    } else {
        for (int i = threadIdx.x; i < rows * dp; i += NT) {
            const int r = i / dp, c = i - r * dp;
            dst[r * pitch + c] = r < n && c < d ? load_elem(src, off(r) + c, Store<ST>::code) : 0.f;
        }
    }
}

template <typename ST>
__global__ void __launch_bounds__(kvg::NT) kv_attn_kernel(const KvArgs a, const int vec) {
    using namespace kvg;
    extern __shared__ __align__(128) unsigned char smem[];
    const Layout L = layout(a.d);
    float* sq = reinterpret_cast<float*>(smem);
    float* sk = reinterpret_cast<float*>(smem + L.off_k);
    float* sv = reinterpret_cast<float*>(smem + L.off_v);
    float* sp = reinterpret_cast<float*>(smem + L.off_p);  // scores, then weights: [RB][KT + 4]
    float* sm = reinterpret_cast<float*>(smem + L.off_row);
    float* sl = sm + RB;
    float* sa = sl + RB;  // factor of the tile on earlier sums
    uint64_t* smask = reinterpret_cast<uint64_t*>(smem + L.off_mask);
    KvScan<NT>& scan = *reinterpret_cast<KvScan<NT>*>(smem + L.off_scan);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float c2 = a.scale * LOG2E;

    kv_grid_launch();
    kv_empty_rows(a, nullptr, tid, NT);
    const KvSplit split = kv_locate<true, KT, NT>(a, scan, gridDim.x, LEAST);
    bool some;
    KvWalk<true, KT> w(a, split, scan, some);
    if (!some) {
        if (tid == 0) static_cast<KvBorder*>(a.border)[blockIdx.x].rows = 0;
        return;
    }
    int checked = -1;
    bool pages_ok = true;
    do {
        const KvSeq& s = w.s;
        const int b = w.b, h = w.h, nt = w.nt, r0 = w.rb * RB;
        const int rows = min(RB, s.nodes * a.G - r0);
        const int32_t* table = a.page_table + (int64_t)s.slot * a.max_pages;
        if (checked != b) {
            pages_ok = __syncthreads_and(kv_pages_ok(a, s, tid, NT));
            if (!pages_ok && tid == 0) set_error(a.dev_err, KV_DEVERR_PAGE);
            checked = b;
        }
        // queries, row state
        kv_load_rows<ST, NT>(sq, L.dp, L.dp, RB, rows, a.q.p, a.d, vec, [&](int r) {
            const int node = (r0 + r) / a.G, hq = h * a.G + (r0 + r) - node * a.G;
            return (int64_t)b * a.q.seq + (int64_t)node * a.q.node + (int64_t)hq * a.q.head;
        });
        if (tid < RB) {
            sm[tid] = -INFINITY, sl[tid] = 0.f;
            smask[tid] = tid < rows ? a.mask[(int64_t)b * a.T + (r0 + tid) / a.G] : 0;
        }
        // outputs: this thread's run of four elements, rows rg, rg + groups, ...
        const int runs = L.dp / 4, groups = NT / runs, run = tid % runs, rg = tid / runs;
        float o[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

        for (int t = w.t0; t < w.t1 && pages_ok; ++t) {
            const bool tree = t == nt - 1;
            const int n = tree ? s.nodes : min(KT, s.len - t * KT);
            __syncthreads();  // the last tile is read
            if (tree) {
                const auto off_k = [&](int r) {
                    return (int64_t)b * a.kn.seq + (int64_t)r * a.kn.node + (int64_t)h * a.kn.head;
                };
                const auto off_v = [&](int r) {
                    return (int64_t)b * a.vn.seq + (int64_t)r * a.vn.node + (int64_t)h * a.vn.head;
                };
                kv_load_rows<ST, NT>(sk, L.pitch, L.dp, KT, n, a.kn.p, a.d, vec, off_k);
                kv_load_rows<ST, NT>(sv, L.pitch, L.dp, KT, n, a.vn.p, a.d, vec, off_v);
            } else {
                const auto page = [&](int r) { return (t * KT + r) / a.page_size; };
                const auto off_k = [&](int r) {
                    const int pg = page(r);
                    return kv_at(a.k, table[pg], h, t * KT + r - pg * a.page_size);
                };
                const auto off_v = [&](int r) {
                    const int pg = page(r);
                    return kv_at(a.v, table[pg], h, t * KT + r - pg * a.page_size);
                };
                kv_load_rows<ST, NT>(sk, L.pitch, L.dp, KT, n, a.k.p, a.d, vec, off_k);
                kv_load_rows<ST, NT>(sv, L.pitch, L.dp, KT, n, a.v.p, a.d, vec, off_v);
            }
            __syncthreads();
            {  // scores of key `key`, rows 4 g .. 4 g + 3
                const int key = tid & (KT - 1), g = tid / KT;
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
                    const bool seen = key < n && (!tree || (smask[r] >> key & 1));
                    sp[r * (KT + 4) + key] = seen ? acc[i] * c2 : -INFINITY;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RB / (NT / 32); ++i) {  // softmax of the warp's rows, two keys a lane
                const int r = warp * (RB / (NT / 32)) + i;
                const float x0 = sp[r * (KT + 4) + lane], x1 = sp[r * (KT + 4) + 32 + lane];
                // fmaxf drops a NaN; the weights below keep it
                float m = fmaxf(x0, x1);
#pragma unroll
                for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, x));
                const float old = sm[r];
                m = fmaxf(m, old);
                const float base = m == -INFINITY ? 0.f : m;  // a row without a key yet
                const float p0 = kv_ex2(x0 - base), p1 = kv_ex2(x1 - base);
                const float sum = group_sum<32>(p0 + p1);
                sp[r * (KT + 4) + lane] = p0, sp[r * (KT + 4) + 32 + lane] = p1;
                if (lane == 0) {
                    const float f = kv_ex2(old - base);
                    sa[r] = f, sl[r] = sl[r] * f + sum, sm[r] = m;
                }
            }
            __syncthreads();
            if (rg < groups) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = rg + i * groups;
                    if (r >= RB) break;
                    const float f = sa[r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= f;
                    const float* pr = sp + r * (KT + 4);
                    for (int key = 0; key < n; ++key) {
                        const float p = pr[key];
                        // a node that a row does not attend adds nothing, whatever its value holds
                        if (tree && p == 0.f) continue;
                        const float4 y = *reinterpret_cast<const float4*>(sv + key * L.pitch + 4 * run);
                        o[i][0] = fmaf(p, y.x, o[i][0]), o[i][1] = fmaf(p, y.y, o[i][1]);
                        o[i][2] = fmaf(p, y.z, o[i][2]), o[i][3] = fmaf(p, y.w, o[i][3]);
                    }
                }
            }
        }
        __syncthreads();
        if (rg < groups) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = rg + i * groups;
                if (r >= rows) break;
                const float l = sl[r];
                if (w.whole()) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const int node = (r0 + r) / a.G, hq = h * a.G + (r0 + r) - node * a.G;
                    const int64_t row = ((int64_t)b * a.T + node) * a.Hq + hq;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * run + e < a.d) store_elem(a.out, row * a.d + 4 * run + e, a.dtype, o[i][e] * inv);
                    if (run == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (sm[r] + log2f(l)) * LN2;
                } else {
                    float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later) * kv_part_floats(RB, a.d);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * run + e < a.d) part[r * a.d + 4 * run + e] = o[i][e];
                    if (run == 0) part[RB * a.d + r] = sm[r], part[RB * a.d + RB + r] = l;
                }
            }
        }
        __syncthreads();
        if (tid == 0 && w.last()) static_cast<KvBorder*>(a.border)[blockIdx.x] = kv_border(a, split, w);
    } while (w.next());
}

}  // namespace gdn
