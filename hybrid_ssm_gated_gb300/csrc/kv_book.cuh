// kv_book.cuh -- bookkeeping of the paged cache: the commit of an accepted
// path, and the eviction of the entries with the least attention weight.
#pragma once

#include <cooperative_groups.h>

#include "kv_common.cuh"

namespace gdn {

// One CTA a sequence: the whole path is checked first, and its entries' places are left in shared memory;
// then every thread copies 16-byte pieces (2-byte ones where the rows allow no more) that do not depend
// on one another, four in flight (a warp a row, one after the other, took 9 us for six tokens of eight
// heads; bound by latency, three loads deep). Index: 32 bits, or 64 where a call's pieces need them (tens of
// thousands of key heads).
constexpr int KV_COMMIT_NT = 256, KV_COMMIT_AHEAD = 4;
template <typename Piece, typename Index>
__global__ void __launch_bounds__(KV_COMMIT_NT) kv_commit_kernel(const __grid_constant__ KvArgs a) {
    constexpr int NT = KV_COMMIT_NT;
    __shared__ int s_node[KV_MAX_NODES], s_page[KV_MAX_NODES], s_place[KV_MAX_NODES];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int slot = a.slots[b], n = a.n_path[b];
    const int node0 = tid < a.P ? a.path[(int64_t)b * a.P + tid] : 0;  // (asked for before the slot is known)
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (tid == 0) set_error(a.dev_err, GDN_DEVERR_SLOT);
        return;
    }
    const int len = a.lengths[slot], count = a.counts ? a.counts[slot] : 0;
    int err = 0;
    if (n < 0 || n > a.P) err |= KV_DEVERR_NODES;
    if (len < 0 || (int64_t)len + (n > 0 ? n : 0) > (int64_t)a.max_pages * a.page_size) err |= KV_DEVERR_LENGTH;
    if (!err && tid < n) {
        const int e = len + tid, pg = e / a.page_size, page = a.page_table[(int64_t)slot * a.max_pages + pg];
        if ((uint32_t)node0 >= (uint32_t)a.T) err |= KV_DEVERR_NODES;
        if ((uint32_t)page >= (uint64_t)a.num_pages) err |= KV_DEVERR_PAGE;
        s_node[tid] = node0, s_page[tid] = page, s_place[tid] = e - pg * a.page_size;
    }
    if (err) set_error(a.dev_err, err);
    if (__syncthreads_or(err)) return;  // the lengths were read by every thread: they may change now
    const int esz = dtype_size(a.dtype), per = a.d * esz / (int)sizeof(Piece);
    const Index rows = (Index)n * a.Hkv, total = 2 * rows * per;
    for (Index i0 = tid; i0 < total; i0 += NT * KV_COMMIT_AHEAD) {
        Piece x[KV_COMMIT_AHEAD];
        Piece* to[KV_COMMIT_AHEAD];
#pragma unroll
        for (int y = 0; y < KV_COMMIT_AHEAD; ++y) {
            const Index i = i0 + y * NT;
            to[y] = nullptr;
            if (i < total) {
                const Index q = i / per;
                const bool val = q >= rows;
                const Index r = val ? q - rows : q;
                const int p = (int)(i - q * per), j = (int)(r / a.Hkv), h = (int)(r - (Index)j * a.Hkv);
                const KvPages& c = val ? a.v : a.k;
                const KvRows& from = val ? a.vn : a.kn;
                to[y] = reinterpret_cast<Piece*>(static_cast<char*>(const_cast<void*>(c.p)) +
                                                 kv_at(c, s_page[j], h, s_place[j]) * esz) + p;
                x[y] = reinterpret_cast<const Piece*>(static_cast<const char*>(from.p) +
                                                      ((int64_t)b * from.seq + (int64_t)s_node[j] * from.node +
                                                       (int64_t)h * from.head) * esz)[p];
            }
        }
#pragma unroll
        for (int y = 0; y < KV_COMMIT_AHEAD; ++y)
            if (to[y]) *to[y] = x[y];
    }
    if (a.weights)
        for (Index i = tid; i < rows; i += NT) {
            const int j = (int)(i / a.Hkv), h = (int)(i - (Index)j * a.Hkv);
            const int64_t w = ((int64_t)s_page[j] * a.Hkv + h) * a.page_size + s_place[j];
            a.weights[w] = 0.f, a.stamps[w] = count + j;
        }
    if (tid == 0 && n > 0) {
        a.lengths[slot] = len + n;
        if (a.counts) a.counts[slot] = count + n;
    }
}

// ---------------------------------------------------------------- eviction

// Order of an entry as an unsigned number: kept-by-age above everything, then NaN, then the weights.
__device__ __forceinline__ uint32_t kv_rank_key(float w, int stamp, int newest) {
    if (stamp >= newest) return 0xFFFFFFFFu;
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
    return u >> 31 ? ~u : u | 0x80000000u;
}

// Selection. A unit (sequence, key head) is the work of one CTA, or of a cluster of up to 8 that each
// take a slice of the entries, so that one long sequence is not left to a handful of SMs. The entries'
// order keys are formed once, into shared memory; three histogram passes of 11, 11 and 10 bits (summed
// over the cluster's shared memories) find the budget-th largest key; then every warp counts, and in a
// second walk lists, a run of entries, 128 at a time, so that the lists are written in lines
// (a run of entries a thread wrote them four bytes a line, and took half of the kernel's time). Bound by
// latency: the loads and barriers of a dozen steps (18 us for 192 units of 4352 entries, 35 us for 8 of
// 131072). Slices that do not fit shared memory form their keys again at each pass.
constexpr int KV_SEL_NT = 512, KV_SEL_WARPS = KV_SEL_NT / 32, KV_SEL_BINS = 2048;

// Entries of a slice, or of a warp's run: above the threshold and at it, below the budget and not.
struct KvCounts {
    unsigned above_low, at_low, above_high, at_high;
};
__device__ __forceinline__ KvCounts operator+(const KvCounts& x, const KvCounts& y) {
    return {x.above_low + y.above_low, x.at_low + y.at_low, x.above_high + y.above_high, x.at_high + y.at_high};
}

struct __align__(16) KvSelect {
    unsigned hist[3][KV_SEL_BINS];
    unsigned warp_sum[KV_SEL_WARPS];
    KvCounts counts[KV_SEL_WARPS], total;  // the CTA's warps', and all of them
    unsigned digit, need;
    int bad;  // a page of the slice lies outside the pool
};

// keys_cap: keys that the dynamic shared memory holds; vec: four entries' weights and stamps in one load.
__global__ void __launch_bounds__(KV_SEL_NT, 4) kv_select_kernel(const __grid_constant__ KvArgs a, const int cap, const int keys_cap,
                                                              const int vec) {
    namespace cg = cooperative_groups;
    constexpr int NT = KV_SEL_NT, WARPS = KV_SEL_WARPS;
    extern __shared__ __align__(128) unsigned char smem[];
    KvSelect& st = *reinterpret_cast<KvSelect*>(smem);
    uint32_t* skey = reinterpret_cast<uint32_t*>(smem + sizeof(KvSelect));
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* list = a.moves + kv_moves_at(unit, cap);
    kv_grid_launch();
    const int slot = a.slots[b];
    int err = 0, len = 0;
    if (slot >= a.num_slots) err = GDN_DEVERR_SLOT;
    if (slot >= 0 && !err) {
        len = a.lengths[slot];
        if (len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size) err = KV_DEVERR_LENGTH;
    }
    if (err && tid == 0) set_error(a.dev_err, err);
    if (slot < 0 || err || len <= a.budget) {  // (the same in every CTA of the cluster)
        if (rank == 0 && tid == 0) list[0] = -1;
        return;
    }
    const int32_t* table = a.page_table + (int64_t)slot * a.max_pages;
    const int newest = a.counts[slot] - a.recent;
    const int per = align_up((len + C - 1) / C, 4), e0 = min(len, rank * per), n = min(len, e0 + per) - e0;
    const bool kept_here = per <= keys_cap;
    for (int i = tid; i < 3 * KV_SEL_BINS / 4; i += NT) reinterpret_cast<uint4*>(st.hist)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) st.bad = 0;
    __syncthreads();

    // ---- order keys; the slice's pages are looked at on the way
    bool bad = false;
    const auto place_of = [&](int e) {  // of entry e in weights and stamps, -1 on a page outside the pool
        const int pg = e / a.page_size, page = table[pg];
        if ((uint32_t)page >= (uint64_t)a.num_pages) {
            bad = true;
            return (int64_t)-1;
        }
        return ((int64_t)page * a.Hkv + h) * a.page_size + (e - pg * a.page_size);
    };
    const auto form = [&](int i) {
        const int64_t x = place_of(e0 + i);
        return x < 0 ? 0u : kv_rank_key(a.weights[x], a.stamps[x], newest);
    };
    if (!kept_here || !vec) {
        for (int i = tid; i < n; i += NT) {
            const uint32_t key = form(i);
            if (kept_here) skey[i] = key;
        }
    } else {
        constexpr int AHEAD = 2;  // loads of a thread that wait for nothing but their pages
        for (int i0 = tid * 4; i0 < n; i0 += NT * 4 * AHEAD) {
            int64_t x[AHEAD];
            float4 w[AHEAD];
            int4 t[AHEAD];
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                const int i = i0 + y * NT * 4;
                x[y] = i < n ? place_of(e0 + i) : -1;
            }
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                w[y] = make_float4(0.f, 0.f, 0.f, 0.f), t[y] = make_int4(0, 0, 0, 0);
                if (x[y] >= 0) {
                    w[y] = *reinterpret_cast<const float4*>(a.weights + x[y]);
                    t[y] = *reinterpret_cast<const int4*>(a.stamps + x[y]);
                }
            }
#pragma unroll
            for (int y = 0; y < AHEAD; ++y)
                if (x[y] >= 0)
                    *reinterpret_cast<uint4*>(skey + i0 + y * NT * 4) =
                        make_uint4(kv_rank_key(w[y].x, t[y].x, newest), kv_rank_key(w[y].y, t[y].y, newest),
                                   kv_rank_key(w[y].z, t[y].z, newest), kv_rank_key(w[y].w, t[y].w, newest));
        }
    }
    if (bad) st.bad = 1;
    __syncthreads();

    // ---- the budget-th largest key
    uint32_t prefix = 0;
    unsigned need = a.budget;  // entries still to be taken among those that share the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        const uint32_t dm = (1u << bits) - 1u;
        const auto take = [&](uint32_t key) {
            if (pass == 0 || (key ^ prefix) >> (shift + bits) == 0) atomicAdd(&st.hist[pass][key >> shift & dm], 1u);
        };
        if (kept_here) {
#pragma unroll 2
            for (int i = tid * 4; i < n; i += NT * 4) {
                const uint4 k = *reinterpret_cast<const uint4*>(skey + i);
                take(k.x);
                if (i + 1 < n) take(k.y);
                if (i + 2 < n) take(k.z);
                if (i + 3 < n) take(k.w);
            }
        } else {
            for (int i = tid; i < n; i += NT) take(form(i));
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        if (pass == 0) {  // a page outside the pool, in any slice: the sequence stays as it is
            const int one = lane < C ? (C > 1 ? *cluster.map_shared_rank(&st.bad, lane) : st.bad) : 0;
            if (__any_sync(FULL_MASK, one)) {
                if (rank == 0 && tid == 0) list[0] = -1, set_error(a.dev_err, KV_DEVERR_PAGE);
                if (C > 1) cluster.sync();
                return;
            }
        }
        // thread t sums bins from the top: 4 (NT - 1 - t) ..
        const int bin = 4 * (NT - 1 - tid);
        uint4 v = *reinterpret_cast<const uint4*>(&st.hist[pass][bin]);
        if (C > 1) {
            uint4 x[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                x[c] = make_uint4(0, 0, 0, 0);
                if (c < C && c != rank) x[c] = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&st.hist[pass][bin], c));
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) v.x += x[c].x, v.y += x[c].y, v.z += x[c].z, v.w += x[c].w;
        }
        const unsigned mine = v.x + v.y + v.z + v.w;
        unsigned inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(FULL_MASK, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) st.warp_sum[warp] = inc;
        __syncthreads();
        unsigned warps = lane < warp ? st.warp_sum[lane & (WARPS - 1)] : 0;  // (warp < 16 lanes)
#pragma unroll
        for (int o = 8; o; o >>= 1) warps += __shfl_xor_sync(FULL_MASK, warps, o);
        unsigned above = __shfl_sync(FULL_MASK, warps, 0) + inc - mine;
        if (above < need && need <= above + mine) {
            int d = bin + 3;
            unsigned in = v.w;
            if (need > above + in) above += in, --d, in = v.z;
            if (need > above + in) above += in, --d, in = v.y;
            if (need > above + in) above += in, --d, in = v.x;
            st.digit = d, st.need = need - above;
        }
        __syncthreads();
        prefix |= st.digit << shift, need = st.need;
    }

    // ---- entries above the threshold are kept, and the first `need` of those at it. A lane takes four
    // entries of its warp's run at a time, its warp 128.
    const int run = align_up((n + WARPS - 1) / WARPS, 128), i0 = min(n, warp * run), i1 = min(n, i0 + run);
    const auto four = [&](int i, uint32_t (&k)[4]) {  // keys of entries i .. i + 3 of the slice (0 past its end)
        if (kept_here) {
            const uint4 x = i < i1 ? *reinterpret_cast<const uint4*>(skey + i) : make_uint4(0, 0, 0, 0);
            k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
        } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) k[y] = i + y < i1 ? form(i + y) : 0;
        }
    };
    KvCounts here{};
    for (int i = i0 + 4 * lane; i < i1; i += 128) {
        uint32_t k[4];
        four(i, k);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const bool in = i + y < i1, low = e0 + i + y < a.budget;
            here.above_low += in && low && k[y] > prefix, here.above_high += in && !low && k[y] > prefix;
            here.at_low += in && low && k[y] == prefix, here.at_high += in && !low && k[y] == prefix;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        here = here + KvCounts{__shfl_xor_sync(FULL_MASK, here.above_low, o), __shfl_xor_sync(FULL_MASK, here.at_low, o),
                               __shfl_xor_sync(FULL_MASK, here.above_high, o), __shfl_xor_sync(FULL_MASK, here.at_high, o)};
    if (lane == 0) st.counts[warp] = here;
    __syncthreads();
    KvCounts before{}, all{};  // in the CTA before this warp's run; in the whole line
    for (int w = 0; w < WARPS; ++w) {
        const KvCounts x = st.counts[w];
        if (w < warp) before = before + x;
        all = all + x;
    }
    if (C > 1) {
        if (tid == 0) st.total = all;
        cluster.sync();
        all = KvCounts{};
        for (int c = 0; c < C; ++c) {
            const KvCounts x = *cluster.map_shared_rank(&st.total, c);
            if (c < rank) before = before + x;
            all = all + x;
        }
        cluster.sync();  // nobody leaves while its counts may be read
    }
    // Places on the lists. Entries at the threshold are kept in their order: those below the budget, which
    // come first, while `need` lasts.
    unsigned at_before = before.at_low + before.at_high;
    const unsigned kept_low = min(need, all.at_low);  // of those at the threshold
    unsigned hole = (unsigned)min(e0 + i0, a.budget) - before.above_low - min(need, before.at_low);
    unsigned fill = before.above_high + min(need, at_before) - min(need, before.at_low);
    int32_t *holes = list + 4, *fills = holes + align_up(cap, 4);
    for (int base = i0; base < i1; base += 128) {
        const int i = base + 4 * lane;
        uint32_t k[4];
        four(i, k);
        // of the lane's entries: at the threshold; then holes and fillers
        unsigned at = 0, mine = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) at += i + y < i1 && k[y] == prefix;
        unsigned inc = at;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(FULL_MASK, inc, o);
            if (lane >= o) inc += x;
        }
        unsigned at_here = at_before + inc - at;
        bool hole_y[4], fill_y[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const bool in = i + y < i1, low = e0 + i + y < a.budget, eq = in && k[y] == prefix;
            const bool kept = (in && k[y] > prefix) || (eq && at_here < need);
            at_here += eq;
            hole_y[y] = in && low && !kept, fill_y[y] = kept && !low;
            mine += (hole_y[y] ? 1u : 0u) + (fill_y[y] ? 0x10000u : 0u);
        }
        unsigned line = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(FULL_MASK, line, o);
            if (lane >= o) line += x;
        }
        unsigned ih = hole + ((line - mine) & 0xffffu), jf = fill + ((line - mine) >> 16);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (hole_y[y]) holes[ih++] = e0 + i + y;
            if (fill_y[y]) fills[jf++] = e0 + i + y;
        }
        const unsigned all_here = __shfl_sync(FULL_MASK, line, 31);
        hole += all_here & 0xffffu, fill += all_here >> 16, at_before += __shfl_sync(FULL_MASK, inc, 31);
    }
    if (rank == 0 && tid == 0) list[0] = a.budget - (int)(all.above_low + kept_low);
}

// The moves of every unit. A warp takes some of them: a lane finds a move's rows, then all lanes copy the
// rows' 16-byte pieces, eight in flight each (a warp a row, one load after the other, took three times
// as long). Bound by HBM: 262144 moves of two 256-byte rows (272 MB read and written) take 42 us, 6.4 TB/s. pieces: of a key and a value row together; magic: its reciprocal, 2^32 / pieces rounded up.
constexpr int KV_MOVE_NT = 256, KV_MOVE_AHEAD = 8;
__global__ void __launch_bounds__(KV_MOVE_NT) kv_move_kernel(const __grid_constant__ KvArgs a, const int cap, const int piece_bytes,
                                                             const int pieces, const uint32_t magic) {
    struct Rows {
        const char* from[2];  // key, value
        char* to[2];
    };
    __shared__ Rows rows[KV_MOVE_NT / 32][32];
    const int unit = blockIdx.x, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = a.slots[b];
    const int esz = dtype_size(a.dtype), half = pieces / 2;
    char* k = static_cast<char*>(const_cast<void*>(a.k.p));
    char* v = static_cast<char*>(const_cast<void*>(a.v.p));
    kv_grid_wait();  // the lists are written
    const int32_t* list = a.moves + kv_moves_at(unit, cap);
    const int n = list[0];
    if (n < 0) return;
    const int32_t *holes = list + 4, *fills = holes + align_up(cap, 4);
    const int32_t* table = a.page_table + (int64_t)slot * a.max_pages;
    if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.lengths[slot] = a.budget;
    // up to 32 moves a warp at a time, fewer where there are more warps than that
    const int warps = gridDim.y * (KV_MOVE_NT / 32), chunk = min(32, (n + warps - 1) / warps);
    for (int first = (blockIdx.y * (KV_MOVE_NT / 32) + warp) * chunk; first < n; first += warps * chunk) {
        const int some = min(chunk, n - first);
        __syncwarp();
        if (lane < some) {
            const int to = holes[first + lane], from = fills[first + lane];
            const int pt = to / a.page_size, pf = from / a.page_size;
            const int ot = to - pt * a.page_size, of = from - pf * a.page_size;
            const int gt = table[pt], gf = table[pf];
            Rows& r = rows[warp][lane];
            r.to[0] = k + kv_at(a.k, gt, h, ot) * esz, r.from[0] = k + kv_at(a.k, gf, h, of) * esz;
            r.to[1] = v + kv_at(a.v, gt, h, ot) * esz, r.from[1] = v + kv_at(a.v, gf, h, of) * esz;
            const int64_t wt = ((int64_t)gt * a.Hkv + h) * a.page_size + ot;
            const int64_t wf = ((int64_t)gf * a.Hkv + h) * a.page_size + of;
            a.weights[wt] = a.weights[wf], a.stamps[wt] = a.stamps[wf];
        }
        __syncwarp();
        const int total = some * pieces;
        for (int i0 = lane; i0 < total; i0 += 32 * KV_MOVE_AHEAD) {
            if (piece_bytes == 16) {
                uint4 x[KV_MOVE_AHEAD];
                char* to[KV_MOVE_AHEAD];
#pragma unroll
                for (int y = 0; y < KV_MOVE_AHEAD; ++y) {
                    const int i = i0 + 32 * y;
                    to[y] = nullptr;
                    if (i < total) {
                        const int m = (int)__umulhi((uint32_t)i, magic), p = i - m * pieces, val = p >= half;
                        const Rows& r = rows[warp][m];
                        const int off = (p - val * half) * 16;
                        x[y] = *reinterpret_cast<const uint4*>(r.from[val] + off), to[y] = r.to[val] + off;
                    }
                }
#pragma unroll
                for (int y = 0; y < KV_MOVE_AHEAD; ++y)
                    if (to[y]) *reinterpret_cast<uint4*>(to[y]) = x[y];
            } else {
                for (int i = i0; i < min(total, i0 + 32 * KV_MOVE_AHEAD); i += 32) {
                    const int m = (int)__umulhi((uint32_t)i, magic), p = i - m * pieces, val = p >= half;
                    const Rows& r = rows[warp][m];
                    const int off = (p - val * half) * 2;
                    *reinterpret_cast<uint16_t*>(r.to[val] + off) = *reinterpret_cast<const uint16_t*>(r.from[val] + off);
                }
            }
        }
    }
}

}  // namespace gdn
