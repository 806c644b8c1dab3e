// kv_share.cuh -- pages that several sequences share: forks of sequences, and the
// compaction of the pool.
//
// Both are copies, bound by HBM where they are large and by the latency of a few
// dependent loads (slot, length, table, page) where they are small. A job of a copy
// is one head of one page: its keys, values, weights and stamps, eight 16-byte pieces in
// flight a thread. 32 forks with pages of their own (fp16, 0.69 GB read and written) take
// 119 us, 5.8 TB/s or 0.85 of the measured copy bandwidth; a compaction that moves 0.31 GB
// 66 us, of which 12 are the kernels' beginnings and the plan; a fork that shares
// all pages but the last 5 us.
#pragma once

#include "kv_common.cuh"

namespace gdn {

namespace kvs {

constexpr int NT = 256, AHEAD = 8;
constexpr int PLAN_NT = 1024;

}  // namespace kvs

// Pages of `len` entries (len + page_size may not fit 32 bits).
__device__ __forceinline__ int kv_pages_of(int len, int page_size) { return len > 0 ? (len - 1) / page_size + 1 : 0; }

// Entries 0 .. n - 1 of head h of page `from` to page `to`, by the whole block. Piece: what rows are copied by.
template <typename Piece>
__device__ __forceinline__ void kv_copy_head(const KvArgs& a, int from, int to, int h, int n) {
    using namespace kvs;
    const int per = a.d * dtype_size(a.dtype) / (int)sizeof(Piece), esz = dtype_size(a.dtype);
    const uint32_t rows = 2u * n;
    // piece i: row i / per (keys, then values), and NT pieces further each time
    const int dr = NT / per, dc = NT - dr * per;
    uint32_t r = threadIdx.x / per;
    int c = (int)(threadIdx.x - r * per);
    while (r < rows) {
        Piece x[AHEAD];
        Piece* out[AHEAD];
#pragma unroll
        for (int y = 0; y < AHEAD; ++y) {
            out[y] = nullptr;
            if (r < rows) {
                const bool val = r >= (uint32_t)n;
                const KvPages& p = val ? a.v : a.k;
                const int64_t at = (int64_t)h * p.head + (int64_t)(val ? r - n : r) * p.token;
                char* base = static_cast<char*>(const_cast<void*>(p.p));
                x[y] = reinterpret_cast<const Piece*>(base + ((int64_t)from * p.page + at) * esz)[c];
                out[y] = reinterpret_cast<Piece*>(base + ((int64_t)to * p.page + at) * esz) + c;
            }
            r += dr, c += dc;
            if (c >= per) c -= per, ++r;
        }
#pragma unroll
        for (int y = 0; y < AHEAD; ++y)
            if (out[y]) *out[y] = x[y];
    }
    if (a.weights) {
        const int64_t f = ((int64_t)from * a.Hkv + h) * a.page_size, t = ((int64_t)to * a.Hkv + h) * a.page_size;
        for (int i = threadIdx.x; i < n; i += NT) a.weights[t + i] = a.weights[f + i], a.stamps[t + i] = a.stamps[f + i];
    }
}

// Block (x, i): fork i, jobs x, x + gridDim.x ... of its pages' heads. Every block looks at all of the fork's
// pages before it writes.
template <typename Piece>
__global__ void __launch_bounds__(kvs::NT) kv_fork_kernel(const __grid_constant__ KvArgs a, const int32_t* src, const int32_t* dst,
                                                           const int32_t* new_pages) {
    using namespace kvs;
    const int i = blockIdx.y, tid = threadIdx.x, from = src[i], to = dst[i];
    if (from < 0 || to < 0) return;
    int err = 0, len = 0;
    if (from >= a.num_slots || to >= a.num_slots || from == to) err = GDN_DEVERR_SLOT;
    if (!err) {
        len = a.lengths[from];
        if (len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size) err = KV_DEVERR_LENGTH;
    }
    const int pages = err ? 0 : kv_pages_of(len, a.page_size);
    const int32_t* old = a.page_table + (int64_t)from * a.max_pages;
    const int32_t* fresh = new_pages + (int64_t)i * a.max_pages;
    bool bad = false;
    for (int j = tid; j < pages; j += NT)
        bad = bad || (uint32_t)old[j] >= (uint64_t)a.num_pages || (fresh[j] >= 0 && fresh[j] >= a.num_pages);
    if (__syncthreads_or(bad)) err |= KV_DEVERR_PAGE;
    if (err) {
        if (blockIdx.x == 0 && tid == 0) set_error(a.dev_err, err);
        return;
    }
    if (blockIdx.x == 0) {
        int32_t* row = const_cast<int32_t*>(a.page_table) + (int64_t)to * a.max_pages;
        for (int j = tid; j < pages; j += NT) row[j] = fresh[j] >= 0 ? fresh[j] : old[j];
        if (tid == 0) {
            a.lengths[to] = len;
            if (a.counts) a.counts[to] = a.counts[from];
        }
    }
    const int64_t jobs = (int64_t)pages * a.Hkv;
    // (from the end: the last page, often the only one to be copied, is begun at once)
    for (int64_t x = jobs - 1 - blockIdx.x; x >= 0; x -= gridDim.x) {
        const int j = (int)(x / a.Hkv), h = (int)(x - (int64_t)j * a.Hkv), page = fresh[j];
        if (page < 0 || page >= a.num_pages) continue;
        const int source = old[j];
        if ((uint32_t)source >= (uint64_t)a.num_pages) continue;
        kv_copy_head<Piece>(a, source, page, h, min(a.page_size, len - j * a.page_size));
    }
}

// ---------------------------------------------------------------- compaction

__global__ void __launch_bounds__(kvs::NT) kv_clear_kernel(int32_t* ws, int words) {
    kv_grid_launch();
    for (int64_t i = (int64_t)blockIdx.x * kvs::NT + threadIdx.x; i < 8 + (int64_t)words; i += (int64_t)gridDim.x * kvs::NT) ws[i] = 0;
}

// The bits of a slot's pages, by a warp; whether something of it is out of range.
__device__ __forceinline__ bool kv_mark_slot(const KvArgs& a, int64_t s, int lane, uint32_t* bits) {
    const int len = a.lengths[s];
    int err = 0;
    if (len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size) err = KV_DEVERR_LENGTH;
    const int pages = err ? 0 : kv_pages_of(len, a.page_size);
    const int32_t* row = a.page_table + s * a.max_pages;
    for (int j = lane; j < pages; j += 32) {
        const int x = row[j];
        if ((uint32_t)x >= (uint64_t)a.num_pages) err = KV_DEVERR_PAGE;
        else atomicOr(&bits[x >> 5], 1u << (x & 31));
    }
    if (err) set_error(a.dev_err, err);
    return err != 0;
}

// A warp a slot at a time.
__global__ void __launch_bounds__(kvs::NT) kv_mark_kernel(const __grid_constant__ KvArgs a, const KvPlan p) {
    using namespace kvs;
    kv_grid_launch();
    kv_grid_wait();
    const int64_t warps = (int64_t)gridDim.x * (NT / 32);
    for (int64_t s = (int64_t)blockIdx.x * (NT / 32) + (threadIdx.x >> 5); s < a.num_slots; s += warps)
        if (kv_mark_slot(a, s, threadIdx.x & 31, p.bits)) p.head[0] = -1;
}

// One block: the number of held pages U, then the lists of holes below U and of held pages from U on. SMALL: it marks the
// pages too, in shared memory, where tables and pool are small (two kernels less ahead of it: 9.7 us instead of 11.2 for
// 4 sequences of 700 entries).
constexpr int KV_SMALL_PAGES = 1 << 18, KV_SMALL_ENTRIES = 1 << 14;
template <bool SMALL>
__global__ void __launch_bounds__(kvs::PLAN_NT) kv_plan_kernel(const __grid_constant__ KvArgs a, const KvPlan p, int32_t* used) {
    using namespace kvs;
    __shared__ int s_warp[PLAN_NT / 32], s_hole[PLAN_NT / 32];
    __shared__ uint32_t s_bits[SMALL ? KV_SMALL_PAGES / 32 : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    kv_grid_launch();
    const uint32_t* bits = p.bits;
    if constexpr (SMALL) {
        bits = s_bits;
        for (int w = tid; w < p.words; w += PLAN_NT) s_bits[w] = 0;
        __syncthreads();
        bool bad = false;
        for (int64_t s = warp; s < a.num_slots; s += PLAN_NT / 32) bad |= kv_mark_slot(a, s, lane, s_bits);
        if (__syncthreads_or(bad)) {
            if (tid == 0) p.head[0] = -1, *used = -1;
            return;
        }
    } else {
        kv_grid_wait();
        if (p.head[0] < 0) {
            if (tid == 0) *used = -1;
            return;
        }
    }
    const auto scan = [&](int x, int* sums, int& total) {  // sum over the threads before this one
        int inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int before = inc - x;
        total = 0;
        for (int w = 0; w < PLAN_NT / 32; ++w) {
            if (w < warp) before += sums[w];
            total += sums[w];
        }
        __syncthreads();
        return before;
    };
    const int run = (p.words + PLAN_NT - 1) / PLAN_NT, w0 = min(p.words, tid * run), w1 = min(p.words, w0 + run);
    int held = 0, U, moves;
    for (int w = w0; w < w1; ++w) held += __popc(bits[w]);
    scan(held, s_warp, U);
    // bits of a word below U, of those that exist
    const auto low = [&](int w) { return U >= 32 * w + 32 ? 0xffffffffu : U <= 32 * w ? 0u : (1u << (U - 32 * w)) - 1; };
    int holes = 0, movers = 0, other;
    for (int w = w0; w < w1; ++w) holes += __popc(~bits[w] & low(w)), movers += __popc(bits[w] & ~low(w));
    int at_hole = scan(holes, s_hole, moves), at_mover = scan(movers, s_warp, other);
    for (int w = w0; w < w1; ++w) {
        for (uint32_t x = ~bits[w] & low(w); x; x &= x - 1) p.hole[at_hole++] = 32 * w + __ffs(x) - 1;
        for (uint32_t x = bits[w] & ~low(w); x; x &= x - 1) p.mover[at_mover++] = 32 * w + __ffs(x) - 1;
    }
    __syncthreads();  // (global writes of the block, read by it: the barrier orders them)
    for (int i = tid; i < moves; i += PLAN_NT) p.to[p.mover[i]] = p.hole[i];
    if (tid == 0) p.head[0] = moves, p.head[1] = U, *used = U;
}

// The moves: blocks 0 .. copiers - 1 copy heads of pages, the others rewrite the tables.
template <typename Piece>
__global__ void __launch_bounds__(kvs::NT) kv_pages_kernel(const __grid_constant__ KvArgs a, const KvPlan p, const int copiers) {
    using namespace kvs;
    kv_grid_wait();
    const int moves = p.head[0], U = p.head[1];
    if (moves <= 0) return;
    if ((int)blockIdx.x < copiers) {
        const int64_t jobs = (int64_t)moves * a.Hkv;
        for (int64_t x = blockIdx.x; x < jobs; x += copiers) {
            const int i = (int)(x / a.Hkv), h = (int)(x - (int64_t)i * a.Hkv);
            kv_copy_head<Piece>(a, p.mover[i], p.hole[i], h, a.page_size);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)(gridDim.x - copiers) * (NT / 32);
    for (int64_t s = (int64_t)(blockIdx.x - copiers) * (NT / 32) + (threadIdx.x >> 5); s < a.num_slots; s += warps) {
        const int pages = kv_pages_of(a.lengths[s], a.page_size);
        int32_t* row = const_cast<int32_t*>(a.page_table) + s * a.max_pages;
        for (int j = lane; j < pages; j += 32) {
            const int x = row[j];
            if (x >= U) row[j] = p.to[x];
        }
    }
}

}  // namespace gdn
