// kv_book.cuh -- bookkeeping of the paged cache: the commit of an accepted
// path, and the eviction of the entries with the least attention weight.
#pragma once

#include "kv_common.cuh"

namespace gdn {

// Copy one row of d elements (esz bytes each); 16 bytes a lane where both ends allow it.
__device__ __forceinline__ void kv_copy_row(char* dst, const char* src, int bytes, bool vec, int lane, int lanes) {
    if (vec) {
        for (int i = lane * 16; i < bytes; i += lanes * 16)
            *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(src + i);
    } else {
        for (int i = lane * 2; i < bytes; i += lanes * 2)
            *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
    }
}

// One CTA a sequence: checks the whole path first, then copies, a warp a row. vec: every row of the
// cache and of the activations can be copied 16 bytes at a time.
constexpr int KV_COMMIT_NT = 256;
__global__ void __launch_bounds__(KV_COMMIT_NT) kv_commit_kernel(const KvArgs a, const int vec) {
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = a.slots[b];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (tid == 0) set_error(a.dev_err, GDN_DEVERR_SLOT);
        return;
    }
    const int len = a.lengths[slot], n = a.n_path[b];
    const int count = a.counts ? a.counts[slot] : 0;
    const int32_t* table = a.page_table + (int64_t)slot * a.max_pages;
    int err = 0;
    if (n < 0 || n > a.P) err |= KV_DEVERR_NODES;
    if (len < 0 || (int64_t)len + (n > 0 ? n : 0) > (int64_t)a.max_pages * a.page_size) err |= KV_DEVERR_LENGTH;
    if (!err)
        for (int j = tid; j < n; j += KV_COMMIT_NT) {
            if ((uint32_t)a.path[(int64_t)b * a.P + j] >= (uint32_t)a.T) err |= KV_DEVERR_NODES;
            if ((uint32_t)table[(len + j) / a.page_size] >= (uint64_t)a.num_pages) err |= KV_DEVERR_PAGE;
        }
    if (err) set_error(a.dev_err, err);
    if (__syncthreads_or(err)) return;  // the lengths were read by every thread: they may change now
    const int esz = dtype_size(a.dtype), bytes = a.d * esz;
    const int rows = n * a.Hkv;
    for (int i = warp; i < 2 * rows; i += KV_COMMIT_NT / 32) {
        const bool val = i >= rows;
        const int r = val ? i - rows : i, j = r / a.Hkv, h = r - j * a.Hkv;
        const int e = len + j, pg = e / a.page_size, place = e - pg * a.page_size;
        const KvPages& c = val ? a.v : a.k;
        const KvRows& x = val ? a.vn : a.kn;
        const int node = a.path[(int64_t)b * a.P + j];
        const int64_t from = (int64_t)b * x.seq + (int64_t)node * x.node + (int64_t)h * x.head;
        char* dst = static_cast<char*>(const_cast<void*>(c.p)) + kv_at(c, table[pg], h, place) * esz;
        kv_copy_row(dst, static_cast<const char*>(x.p) + from * esz, bytes, vec, lane, 32);
        if (!val && lane == 0 && a.weights) {
            const int64_t w = ((int64_t)table[pg] * a.Hkv + h) * a.page_size + place;
            a.weights[w] = 0.f, a.stamps[w] = count + j;
        }
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

constexpr int KV_SEL_NT = 512;
// One CTA a (sequence, key head): the budget-th largest order key by radix selection (four digits of
// eight bits), then the holes and fillers in order of entry.
__global__ void __launch_bounds__(KV_SEL_NT) kv_select_kernel(const KvArgs a, const int cap) {
    constexpr int NT = KV_SEL_NT;
    __shared__ int hist[256];
    __shared__ int warp_count[NT / 32][3];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int unit = blockIdx.x, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* list = a.moves + kv_moves_at(unit, cap);
    const int slot = a.slots[b];
    int err = 0, len = 0;
    if (slot >= a.num_slots) err = GDN_DEVERR_SLOT;
    if (slot >= 0 && !err) {
        len = a.lengths[slot];
        if (len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size) err = KV_DEVERR_LENGTH;
    }
    if (err && tid == 0) set_error(a.dev_err, err);
    if (slot < 0 || err || len <= a.budget) {
        if (tid == 0) list[0] = -1;
        return;
    }
    const KvSeq s{slot, len, 0, 0};
    if (!__syncthreads_and(kv_pages_ok(a, s, tid, NT))) {
        if (tid == 0) list[0] = -1, set_error(a.dev_err, KV_DEVERR_PAGE);
        return;
    }
    const int32_t* table = a.page_table + (int64_t)slot * a.max_pages;
    const int newest = a.counts[slot] - a.recent;
    const auto key_of = [&](int e) {
        const int pg = e / a.page_size;
        const int64_t i = ((int64_t)table[pg] * a.Hkv + h) * a.page_size + (e - pg * a.page_size);
        return kv_rank_key(a.weights[i], a.stamps[i], newest);
    };
    uint32_t prefix = 0;
    int need = a.budget;  // entries still to be taken among those that share the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += NT) hist[i] = 0;
        __syncthreads();
        for (int e = tid; e < len; e += NT) {
            const uint32_t key = key_of(e);
            if (shift == 24 || (key ^ prefix) >> (shift + 8) == 0) atomicAdd(&hist[key >> shift & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int d = 255, left = need;
            while (hist[d] < left) left -= hist[d--];
            s_prefix = prefix | (uint32_t)d << shift, s_need = left;
        }
        __syncthreads();
        prefix = s_prefix, need = s_need;
    }
    // entries above the threshold are kept, and the first `need` of those at it
    int eq0 = 0, hole0 = 0, fill0 = 0;
    for (int base = 0; base < len; base += NT) {
        const int e = base + tid;
        const uint32_t key = e < len ? key_of(e) : 0;
        const bool eq = e < len && key == prefix;
        const unsigned me = __ballot_sync(FULL_MASK, eq), below = (1u << lane) - 1u;
        if (lane == 0) warp_count[warp][0] = __popc(me);
        __syncthreads();
        int eq_before = eq0 + __popc(me & below);
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) eq_before += warp_count[w][0];
            eq0 += warp_count[w][0];
        }
        const bool kept = e < len && (key > prefix || (eq && eq_before < need));
        const bool hole = e < a.budget && !kept, fill = kept && e >= a.budget;
        const unsigned mh = __ballot_sync(FULL_MASK, hole), mf = __ballot_sync(FULL_MASK, fill);
        if (lane == 0) warp_count[warp][1] = __popc(mh), warp_count[warp][2] = __popc(mf);
        __syncthreads();
        int ih = hole0 + __popc(mh & below), jf = fill0 + __popc(mf & below);
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) ih += warp_count[w][1], jf += warp_count[w][2];
            hole0 += warp_count[w][1], fill0 += warp_count[w][2];
        }
        if (hole) list[4 + ih] = e;
        if (fill) list[4 + align_up(cap, 4) + jf] = e;
        __syncthreads();
    }
    if (tid == 0) list[0] = hole0;
}

// The moves of every unit, a warp a row, the CTAs of a unit taking rows in turn.
constexpr int KV_MOVE_NT = 256;
__global__ void __launch_bounds__(KV_MOVE_NT) kv_move_kernel(const KvArgs a, const int cap, const int vec) {
    const int unit = blockIdx.x, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t* list = a.moves + kv_moves_at(unit, cap);
    const int n = list[0];
    if (n < 0) return;
    const int slot = a.slots[b];
    const int32_t* table = a.page_table + (int64_t)slot * a.max_pages;
    const int esz = dtype_size(a.dtype), bytes = a.d * esz;
    for (int i = blockIdx.y * (KV_MOVE_NT / 32) + warp; i < n; i += gridDim.y * (KV_MOVE_NT / 32)) {
        const int to = list[4 + i], from = list[4 + align_up(cap, 4) + i];
        const int pt = to / a.page_size, pf = from / a.page_size;
        const int ot = to - pt * a.page_size, of = from - pf * a.page_size;
        const int gt = table[pt], gf = table[pf];
        char* k = static_cast<char*>(const_cast<void*>(a.k.p));
        char* v = static_cast<char*>(const_cast<void*>(a.v.p));
        kv_copy_row(k + kv_at(a.k, gt, h, ot) * esz, k + kv_at(a.k, gf, h, of) * esz, bytes, vec, lane, 32);
        kv_copy_row(v + kv_at(a.v, gt, h, ot) * esz, v + kv_at(a.v, gf, h, of) * esz, bytes, vec, lane, 32);
        if (lane == 0) {
            const int64_t wt = ((int64_t)gt * a.Hkv + h) * a.page_size + ot;
            const int64_t wf = ((int64_t)gf * a.Hkv + h) * a.page_size + of;
            a.weights[wt] = a.weights[wf], a.stamps[wt] = a.stamps[wf];
        }
    }
    if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.lengths[slot] = a.budget;
}

}  // namespace gdn
