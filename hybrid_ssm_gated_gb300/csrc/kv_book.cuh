// kv_book.cuh -- bookkeeping of the paged cache: the commit of an accepted
// path, and the eviction of the entries with the least attention weight.
#pragma once

#include <cooperative_groups.h>

#include "kv_common.cuh"

namespace gdn {

// One CTA a sequence: the whole path is checked first, and its entries' places are left in shared memory;
// then every thread copies 16-byte pieces (2-byte ones where the rows allow no more) that do not depend
// on one another, four in flight (a warp a row, one after the other, took 9 us for six tokens of eight
// heads; bound by latency, three loads deep).
constexpr int KV_COMMIT_NT = 256, KV_COMMIT_AHEAD = 4;
template <typename Piece>
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
    const int rows = n * a.Hkv, total = 2 * rows * per;
    for (int i0 = tid; i0 < total; i0 += NT * KV_COMMIT_AHEAD) {
        Piece x[KV_COMMIT_AHEAD];
        Piece* to[KV_COMMIT_AHEAD];
#pragma unroll
        for (int y = 0; y < KV_COMMIT_AHEAD; ++y) {
            const int i = i0 + y * NT;
            to[y] = nullptr;
            if (i < total) {
                const int q = i / per, p = i - q * per;
                const bool val = q >= rows;
                const int r = val ? q - rows : q, j = r / a.Hkv, h = r - j * a.Hkv;
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
        for (int i = tid; i < rows; i += NT) {
            const int j = i / a.Hkv, h = i - j * a.Hkv;
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
// over the cluster's shared memories) find the budget-th largest key; then every thread counts and lists
// a run of consecutive entries, placed by scans over threads and CTAs. Slices that do not fit shared
// memory form their keys again at each pass.
constexpr int KV_SEL_NT = 512, KV_SEL_BINS = 2048;

struct __align__(16) KvSelect {
    unsigned hist[3][KV_SEL_BINS];
    unsigned long long warp_sum[KV_SEL_NT / 32];
    unsigned long long total[2];  // of this CTA: entries at the threshold; holes and fillers
    unsigned digit, need;
};

// Sum of x over the threads before this one; `all` is the sum over the block.
__device__ __forceinline__ unsigned long long kv_block_before(KvSelect& st, unsigned long long x, unsigned long long& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(FULL_MASK, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();  // the last sums are read
    if (lane == 31) st.warp_sum[warp] = inc;
    __syncthreads();
    unsigned long long before = inc - x;
    all = 0;
    for (int w = 0; w < KV_SEL_NT / 32; ++w) {
        if (w < warp) before += st.warp_sum[w];
        all += st.warp_sum[w];
    }
    return before;
}

// keys_cap: keys that the dynamic shared memory holds (one word in 32 is padding, so that threads that
// walk runs of 32 entries meet different banks); vec: four entries' weights and stamps in one load each.
__global__ void __launch_bounds__(KV_SEL_NT) kv_select_kernel(const __grid_constant__ KvArgs a, const int cap, const int keys_cap,
                                                              const int vec) {
    namespace cg = cooperative_groups;
    constexpr int NT = KV_SEL_NT;
    extern __shared__ __align__(128) unsigned char smem[];
    KvSelect& st = *reinterpret_cast<KvSelect*>(smem);
    uint32_t* skey = reinterpret_cast<uint32_t*>(smem + sizeof(KvSelect));
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int unit = blockIdx.x / C, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int tid = threadIdx.x;
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
    const KvSeq s{slot, len, 0, 0};
    if (!__syncthreads_and(kv_pages_ok(a, s, tid, NT))) {
        if (rank == 0 && tid == 0) list[0] = -1, set_error(a.dev_err, KV_DEVERR_PAGE);
        return;
    }
    const int32_t* table = a.page_table + (int64_t)slot * a.max_pages;
    const int newest = a.counts[slot] - a.recent;
    const int per = align_up((len + C - 1) / C, 4), e0 = min(len, rank * per), n = min(len, e0 + per) - e0;
    const bool kept_here = per + (per >> 5) <= keys_cap;
    const auto at = [](int i) { return i + (i >> 5); };
    const auto place_of = [&](int e) {
        const int pg = e / a.page_size;
        return ((int64_t)table[pg] * a.Hkv + h) * a.page_size + (e - pg * a.page_size);
    };
    const auto form = [&](int i) {
        const int64_t x = place_of(e0 + i);
        return kv_rank_key(a.weights[x], a.stamps[x], newest);
    };
    const auto key_of = [&](int i) { return kept_here ? skey[at(i)] : form(i); };

    for (int i = tid; i < 3 * KV_SEL_BINS; i += NT) (&st.hist[0][0])[i] = 0;
    if (kept_here) {
        if (vec) {
#pragma unroll 2
            for (int i = tid * 4; i < n; i += NT * 4) {
                const int64_t x = place_of(e0 + i);
                const float4 w = *reinterpret_cast<const float4*>(a.weights + x);
                const int4 t = *reinterpret_cast<const int4*>(a.stamps + x);
                uint32_t* k = skey + at(i);
                k[0] = kv_rank_key(w.x, t.x, newest), k[1] = kv_rank_key(w.y, t.y, newest);
                k[2] = kv_rank_key(w.z, t.z, newest), k[3] = kv_rank_key(w.w, t.w, newest);
            }
        } else {
            for (int i = tid; i < n; i += NT) skey[at(i)] = form(i);
        }
    }
    __syncthreads();

    uint32_t prefix = 0;
    unsigned need = a.budget;  // entries still to be taken among those that share the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        const uint32_t dm = (1u << bits) - 1u;
        for (int i = tid; i < n; i += NT) {
            const uint32_t key = key_of(i);
            if (pass == 0 || (key ^ prefix) >> (shift + bits) == 0) atomicAdd(&st.hist[pass][key >> shift & dm], 1u);
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        // thread t sums bins from the top: 4 (NT - 1 - t) ..
        const int bin = 4 * (NT - 1 - tid);
        uint4 v = make_uint4(0, 0, 0, 0);
        for (int c = 0; c < C; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(C > 1 ? cluster.map_shared_rank(&st.hist[pass][bin], c) : &st.hist[pass][bin]);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        unsigned long long all;
        unsigned above = (unsigned)kv_block_before(st, (unsigned long long)v.x + v.y + v.z + v.w, all);
        if (above < need && need <= above + v.x + v.y + v.z + v.w) {
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

    // entries above the threshold are kept, and the first `need` of those at it
    const int run = (n + NT - 1) / NT, i0 = min(n, tid * run), i1 = min(n, i0 + run);
    unsigned long long eq = 0, all;
    for (int i = i0; i < i1; ++i) eq += key_of(i) == prefix;
    unsigned long long eq_before = kv_block_before(st, eq, all);
    const auto before_cta = [&](int which, unsigned long long mine) {  // sum over the cluster's CTAs before this one
        if (C == 1) return 0ull;
        if (tid == 0) st.total[which] = mine;
        cluster.sync();
        unsigned long long x = 0;
        for (int c = 0; c < rank; ++c) x += *cluster.map_shared_rank(&st.total[which], c);
        return x;
    };
    eq_before += before_cta(0, all);
    unsigned long long count = 0;  // holes in the low half, fillers in the high one
    unsigned left = eq_before < need ? need - (unsigned)eq_before : 0;  // of those at the threshold, still to keep
    const unsigned left0 = left;
    const auto walk = [&](auto&& hole, auto&& fill) {
        left = left0;
        for (int i = i0; i < i1; ++i) {
            const uint32_t key = key_of(i);
            bool kept = key > prefix;
            if (key == prefix && left > 0) kept = true, --left;
            const int e = e0 + i;
            if (e < a.budget) {
                if (!kept) hole(e);
            } else if (kept) {
                fill(e);
            }
        }
    };
    walk([&](int) { ++count; }, [&](int) { count += 1ull << 32; });
    unsigned long long before = kv_block_before(st, count, all);
    before += before_cta(1, all);
    int ih = (int)(before & 0xffffffffu), jf = (int)(before >> 32);
    int32_t *holes = list + 4, *fills = holes + align_up(cap, 4);
    walk([&](int e) { holes[ih++] = e; }, [&](int e) { fills[jf++] = e; });
    if (rank == C - 1 && tid == NT - 1) list[0] = ih;  // all of them: the last thread's count ends the line
    if (C > 1) cluster.sync();  // nobody leaves while its sums may be read
}

// The moves of every unit. A warp takes 32 of them: a lane finds a move's rows, then all lanes copy the
// rows' 16-byte pieces, eight in flight each (a warp a row, one load after the other, took three times
// as long). pieces: of a key and a value row together; magic: its reciprocal, 2^32 / pieces rounded up.
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
    for (int first = (blockIdx.y * (KV_MOVE_NT / 32) + warp) * 32; first < n; first += gridDim.y * KV_MOVE_NT) {
        const int some = min(32, n - first);
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
