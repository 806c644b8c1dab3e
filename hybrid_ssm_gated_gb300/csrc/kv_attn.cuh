// kv_attn.cuh -- attention of drafted nodes over the paged cache on the FP32
// pipe: any cache dtype, head size up to 256, page size and stride. It serves
// fp32 caches, whose scores and outputs keep FP32 products, and 16-bit caches
// that the tensor-core kernel's copies cannot address.
//
// Mathematics. One pass over the keys with a running maximum m and sum l a
// row (base-2 exponents): for a tile of scores s, m' = max(m, max s),
// l' = l 2^{m - m'} + sum 2^{s - m'}, O' = O 2^{m - m'} + sum 2^{s - m'} v; at
// the end out = O / l and lse = (m + log2 l) ln 2. A tile's sum is formed by
// itself and added to O' with the rescaling: entries summed one after another
// into O' were each rounded to its steps, which over 131072 like entries made
// outputs up to 0.8% wrong.
//
// Shape: 128 threads, units of up to RB query rows (node-major: row = node *
// G + head of the group; 4 for the rows of a plain decode step, else 16), tiles
// of 64 keys in shared memory as FP32, in a ring of three buffers that K and V
// tiles take in turn (cp.async where the rows allow 16-byte copies of FP32), so
// that two tiles are in flight while one is computed on.
//   RB = 16: a thread takes two keys x four rows of the scores (its warp's), and
//   four outputs x four or eight rows: 6 shared loads for 32 products, 2 for 16;
//   RB = 4: two threads a key, each half of d x four rows; for the outputs the
//   threads split the keys too and are summed when the unit ends.
// Bound by shared-memory loads at 16 rows, by latency at 4. fp32, 32 / 8 heads,
// d = 128, 8 sequences of 1301 to 4096 tokens, 21297 in all (0.17 GB): a decode
// step 56 us (3.1 TB/s), 16-node trees 484 us (11.5 TFLOP/s). (With synchronous
// loads of tiles by 256 threads: 188 and 640 us.) 16-bit rows are unpacked by the
// threads that load them, with nothing in flight beside: the same decode step of
// bf16 with d = 124 takes 354 us, with d = 128 on the tensor cores 21.
#pragma once

#include "kv_common.cuh"

namespace gdn {

namespace kvg {

constexpr int KT = 64, NT = 128, BUFS = 3;
constexpr int LEAST = 2;  // of the line a CTA at least

template <int RB>
struct Layout {
    int dp, pitch, off_q, off_s, off_p, off_row, off_mask, off_at, off_scan, bytes;
};
template <int RB>
__host__ __device__ inline Layout<RB> layout(int d) {
    Layout<RB> L;
    L.dp = align_up(d, 4);
    L.pitch = L.dp + (RB == 4 ? 8 : 4);  // the threads of a 16-byte load's phase meet distinct banks
    L.off_q = BUFS * KT * L.pitch * 4;
    L.off_s = L.off_q + RB * L.dp * 4;
    L.off_p = L.off_s + RB * (KT + 4) * 4;
    L.off_row = L.off_p + KT * (RB + 4) * 4;
    L.off_mask = L.off_row + 3 * 16 * 4;
    L.off_at = L.off_mask + 16 * 8;
    L.off_scan = L.off_at + 2 * 2 * KT * 8;
    L.bytes = L.off_scan + (int)sizeof(KvScan<NT>);
    return L;
}

// 16 bytes asynchronously, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

}  // namespace kvg

// `rows` rows of d elements (row i at base + off[i], elements of type ST; the ones from n on are zero)
// into FP32 rows of `pitch` floats, the padding of d zero. vec: rows may be read 16 bytes at a time; FP32
// ones are then copied asynchronously (the caller commits and waits).
template <typename ST, int NT, typename Off>
__device__ __forceinline__ void kv_load_rows(float* dst, int pitch, int dp, int rows, int n, const void* base, int d,
                                             bool vec, Off off) {
    constexpr int VEC = Store<ST>::VEC;
    const ST* src = static_cast<const ST*>(base);
    if (vec) {  // d is a multiple of VEC: no padding
        // piece i = r per + c of the rows, and NT pieces further each time (without a division a piece, which
        // took longer than the copies)
        const int per = d / VEC, dr = NT / per, dc = NT - dr * per;
        int r = (int)threadIdx.x / per, piece = (int)threadIdx.x - r * per;
        const auto next = [&]() {
            r += dr, piece += dc;
            if (piece >= per) piece -= per, ++r;
        };
        if constexpr (sizeof(ST) == 4) {
#pragma unroll 4
            for (; r < rows; next()) {
                const int c = piece * VEC;
                const bool live = r < n;
                kvg::cp_async16_or_zero(dst + r * pitch + c, live ? src + off(r) + c : src, live);
            }
        } else {
            for (; r < rows; next()) {
                const int c = piece * VEC;
                float x[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = 0.f;
                if (r < n) Store<ST>::unpack(*reinterpret_cast<const uint4*>(src + off(r) + c), x);
#pragma unroll
                for (int e = 0; e < VEC; e += 4)
                    *reinterpret_cast<float4*>(dst + r * pitch + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
        }
    } else {
        for (int i = threadIdx.x; i < rows * dp; i += NT) {
            const int r = i / dp, c = i - r * dp;
            dst[r * pitch + c] = r < n && c < d ? load_elem(src, off(r) + c, Store<ST>::code) : 0.f;
        }
    }
}

// x += sum of four products
__device__ __forceinline__ void kv_dot4(float& x, const float4& a, const float4& b) {
    x = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, x))));
}

template <typename ST, int RB>
__global__ void __launch_bounds__(kvg::NT) kv_attn_kernel(const __grid_constant__ KvArgs a, const int vec) {
    using namespace kvg;
    constexpr int QUADS = RB / 4, MINE = QUADS == 1 ? 1 : 2;  // row quads, and of a thread at most
    extern __shared__ __align__(128) unsigned char smem[];
    const Layout<RB> L = layout<RB>(a.d);
    float* ring = reinterpret_cast<float*>(smem);
    float* sq = reinterpret_cast<float*>(smem + L.off_q);
    float* ss = reinterpret_cast<float*>(smem + L.off_s);  // scores [RB][KT + 4]
    float* sp = reinterpret_cast<float*>(smem + L.off_p);  // weights, transposed [KT][RB + 4]
    float* sm = reinterpret_cast<float*>(smem + L.off_row);
    float* sl = sm + 16;
    float* sa = sl + 16;  // factor of the tile on earlier sums
    uint64_t* smask = reinterpret_cast<uint64_t*>(smem + L.off_mask);
    int64_t* at = reinterpret_cast<int64_t*>(smem + L.off_at);  // [2 tiles][K, V][KT] element offsets of rows
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
    // outputs: this thread's run of four elements; the other threads of the run take other rows (RB = 16) or
    // other keys (RB = 4)
    const int runs = L.dp / 4, groups = NT / runs, run = tid % runs, grp = tid / runs;
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
        const auto live_of = [&](int t) { return t == nt - 1 ? s.nodes : min(KT, s.len - t * KT); };
        const auto place_rows = [&](int t) {  // offsets of tile t's rows
            if (tid < KT && t < w.t1) {
                int64_t* to = at + (t & 1) * 2 * KT + tid;
                if (t == nt - 1) {
                    to[0] = (int64_t)b * a.kn.seq + (int64_t)tid * a.kn.node + (int64_t)h * a.kn.head;
                    to[KT] = (int64_t)b * a.vn.seq + (int64_t)tid * a.vn.node + (int64_t)h * a.vn.head;
                } else if (t * KT + tid < s.len) {
                    const int e = t * KT + tid, pg = e / a.page_size, place = e - pg * a.page_size, page = table[pg];
                    to[0] = kv_at(a.k, page, h, place), to[KT] = kv_at(a.v, page, h, place);
                }
            }
        };
        // load i of the segment: K of tile t0 + i / 2, or its V
        const int loads = 2 * (w.t1 - w.t0);
        const auto load = [&](int i) {
            if (i < loads) {
                const int t = w.t0 + (i >> 1), val = i & 1;
                const bool tree = t == nt - 1;
                const int64_t* off = at + ((t & 1) * 2 + val) * KT;
                const void* base = val ? (tree ? a.vn.p : a.v.p) : (tree ? a.kn.p : a.k.p);
                kv_load_rows<ST, NT>(ring + (i % BUFS) * KT * L.pitch, L.pitch, L.dp, KT, live_of(t), base, a.d, vec,
                                     [&](int r) { return off[r]; });
            }
            cp_async_commit();
        };
        float o[MINE][4][4];
#pragma unroll
        for (int q = 0; q < MINE; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[q][i][e] = 0.f;
        if (tid < RB) {
            sm[tid] = -INFINITY, sl[tid] = 0.f;
            smask[tid] = tid < rows ? a.mask[(int64_t)b * a.T + (r0 + tid) / a.G] : 0;
        }
        if (pages_ok) {
            place_rows(w.t0);
            kv_load_rows<ST, NT>(sq, L.dp, L.dp, RB, rows, a.q.p, a.d, vec, [&](int r) {
                const int node = (r0 + r) / a.G, hq = h * a.G + (r0 + r) - node * a.G;
                return (int64_t)b * a.q.seq + (int64_t)node * a.q.node + (int64_t)hq * a.q.head;
            });
            __syncthreads();
            load(0), load(1);
        }
        for (int i = 0; i < loads && pages_ok; ++i) {
            const int t = w.t0 + (i >> 1);
            const bool tree = t == nt - 1;
            const int n = live_of(t);
            const float* buf = ring + (i % BUFS) * KT * L.pitch;
            if ((i & 1) == 0) place_rows(t + 1);
            cp_async_wait<1>();
            __syncthreads();  // load i is there for everyone, and the buffer of load i - 1 is read
            load(i + 2);
            if ((i & 1) == 0) {
                // ---- scores
                if constexpr (RB == 16) {
                    float acc[2][4] = {};
                    const float *k0 = buf + lane * L.pitch, *k1 = k0 + 32 * L.pitch, *q = sq + 4 * warp * L.dp;
#pragma unroll 2
                    for (int e = 0; e < L.dp; e += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(k0 + e);
                        const float4 y = *reinterpret_cast<const float4*>(k1 + e);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float4 z = *reinterpret_cast<const float4*>(q + r * L.dp + e);
                            kv_dot4(acc[0][r], x, z), kv_dot4(acc[1][r], y, z);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int row = 4 * warp + r, key = lane + 32 * k;
                            const bool seen = key < n && (!tree || (smask[row] >> key & 1));
                            ss[row * (KT + 4) + key] = seen ? acc[k][r] * c2 : -INFINITY;
                        }
                } else {
                    float acc[4] = {};
                    const int key = tid >> 1;
                    const float* k = buf + key * L.pitch;
#pragma unroll 2
                    for (int e = 4 * (tid & 1); e < L.dp; e += 8) {
                        const float4 x = *reinterpret_cast<const float4*>(k + e);
#pragma unroll
                        for (int r = 0; r < 4; ++r) kv_dot4(acc[r], x, *reinterpret_cast<const float4*>(sq + r * L.dp + e));
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = acc[r] + __shfl_xor_sync(FULL_MASK, acc[r], 1);
                        const bool seen = key < n && (!tree || (smask[r] >> key & 1));
                        if ((r >> 1) == (tid & 1)) ss[r * (KT + 4) + key] = seen ? x * c2 : -INFINITY;
                    }
                }
                __syncthreads();
                // ---- softmax of the warp's rows, two keys a lane
#pragma unroll
                for (int x = 0; x < RB / 4; ++x) {
                    const int r = warp * (RB / 4) + x;
                    const float x0 = ss[r * (KT + 4) + lane], x1 = ss[r * (KT + 4) + 32 + lane];
                    float m = fmaxf(x0, x1);  // (drops a NaN; the weights below keep it)
#pragma unroll
                    for (int y = 16; y; y >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, y));
                    const float old = sm[r];
                    m = fmaxf(m, old);
                    const float base = m == -INFINITY ? 0.f : m;  // a row without a key yet
                    const float p0 = kv_ex2(x0 - base), p1 = kv_ex2(x1 - base);
                    const float sum = group_sum<32>(p0 + p1);
                    sp[lane * (RB + 4) + r] = p0, sp[(32 + lane) * (RB + 4) + r] = p1;
                    __syncwarp();
                    if (lane == 0) {
                        const float f = kv_ex2(old - base);
                        sa[r] = f, sl[r] = sl[r] * f + sum, sm[r] = m;
                    }
                }
                continue;  // the next step's barrier publishes the weights
            }
            // ---- outputs
            if (grp >= groups) continue;
            const int first = RB == 16 ? 0 : grp, step = RB == 16 ? 1 : groups;  // keys
#pragma unroll
            for (int q = 0; q < MINE; ++q) {
                const int quad = RB == 16 ? grp + q * groups : 0;
                if (quad >= QUADS) break;
                const float4 f = *reinterpret_cast<const float4*>(sa + 4 * quad);
                const float fs[4] = {f.x, f.y, f.z, f.w};
                float tile[4][4] = {};  // the tile's own sums
                const float *p = sp + 4 * quad, *v = buf + 4 * run;
                const auto add = [&](int key, bool skip) {
                    const float4 pk = *reinterpret_cast<const float4*>(p + key * (RB + 4));
                    const float4 y = *reinterpret_cast<const float4*>(v + key * L.pitch);
                    const float ps[4] = {pk.x, pk.y, pk.z, pk.w};
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (skip && ps[r] == 0.f) continue;
                        tile[r][0] = fmaf(ps[r], y.x, tile[r][0]), tile[r][1] = fmaf(ps[r], y.y, tile[r][1]);
                        tile[r][2] = fmaf(ps[r], y.z, tile[r][2]), tile[r][3] = fmaf(ps[r], y.w, tile[r][3]);
                    }
                };
                if (tree) {  // a node that a row does not attend adds nothing, whatever its value holds
                    for (int key = first; key < n; key += step) add(key, true);
                } else {
#pragma unroll 4
                    for (int key = first; key < n; key += step) add(key, false);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[q][r][e] = fmaf(o[q][r][e], fs[r], tile[r][e]);
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        if constexpr (RB == 4) {  // the groups' sums over their keys, into the first
            if (grp > 0 && grp < groups) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<float4*>(ring + ((grp - 1) * 4 + r) * L.dp + 4 * run) =
                        make_float4(o[0][r][0], o[0][r][1], o[0][r][2], o[0][r][3]);
            }
            __syncthreads();
            if (grp == 0)
                for (int x = 1; x < groups; ++x)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 y = *reinterpret_cast<const float4*>(ring + ((x - 1) * 4 + r) * L.dp + 4 * run);
                        o[0][r][0] += y.x, o[0][r][1] += y.y, o[0][r][2] += y.z, o[0][r][3] += y.w;
                    }
        }
        float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later) * kv_part_floats(RB, a.d);
        if (RB == 16 ? grp < groups : grp == 0) {
#pragma unroll
            for (int q = 0; q < MINE; ++q) {
                const int quad = RB == 16 ? grp + q * groups : 0;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = 4 * quad + x;
                    if (quad >= QUADS || r >= rows) break;
                    const float l = sl[r];
                    if (w.whole()) {
                        const float inv = l == 0.f ? 0.f : 1.f / l;
                        const int node = (r0 + r) / a.G, hq = h * a.G + (r0 + r) - node * a.G;
                        const int64_t row = ((int64_t)b * a.T + node) * a.Hq + hq;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * run + e < a.d) store_elem(a.out, row * a.d + 4 * run + e, a.dtype, o[q][x][e] * inv);
                        if (run == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (sm[r] + log2f(l)) * LN2;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * run + e < a.d) part[r * a.d + 4 * run + e] = o[q][x][e];
                        if (run == 0) part[RB * a.d + r] = sm[r], part[RB * a.d + RB + r] = l;
                    }
                }
            }
        }
        if (tid == 0 && w.last()) static_cast<KvBorder*>(a.border)[blockIdx.x] = kv_border(a, split, w);
        __syncthreads();
    } while (w.next());
}

}  // namespace gdn
