// kv_common.cuh -- what the key/value-cache kernels share: launch arguments,
// addresses of cache entries, and the division of a batch's key tiles over a
// persistent grid.
//
// Division. A sequence of a call is a row of units (key head, block of query
// rows), each a run of key tiles behind a few cost tiles that stand for what a
// unit costs beyond its tiles (start, sums, outputs); all units of all
// sequences in order make one line of W, and CTA c of G takes [W c / G,
// W (c + 1) / G) of it. So every CTA has the same work whatever the lengths,
// with no host knowledge of them; a unit that spans several CTAs leaves one
// partial result (unnormalised output, maximum and sum) a CTA, joined
// afterwards by kv_join_kernel. A CTA holds at most two partials: that of the
// unit it starts in and that of the unit it ends in. (Without the cost tiles
// the CTAs that met five units of 16-node trees took 81 us, those that met two
// 58 us.)
#pragma once

#include "../../include/kv.h"
#include "gdn_device.cuh"

namespace gdn {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct KvPages {  // one of k, v: base address and strides in elements
    const void* p;
    int64_t page, head, token;
};

struct KvRows {
    const void* p;
    int64_t seq, node, head;
};

struct KvArgs {
    KvPages k, v;
    const int32_t* page_table;
    const int32_t* slots;
    int32_t* lengths;
    int32_t* counts;
    float* weights;
    int32_t* stamps;
    int32_t* dev_err;
    int64_t num_pages, num_slots;
    int B, T, P, Hq, Hkv, G;  // G: query heads a key head
    int d, page_size, max_pages, dtype;
    // attention and accumulation
    KvRows q, kn, vn;
    const uint64_t* mask;
    const int32_t* num_nodes;  // attention: nodes of each sequence
    const int32_t* path;
    const int32_t* n_path;
    const float* lse_in;
    float scale, decay;
    void* out;
    float* lse;
    float* part;  // partials: [CTA][2] blocks of row_block x (d + 2) floats
    void* border;  // a KvBorder a CTA
    int row_block;  // query rows a unit at most
    // eviction
    int budget, recent;
    int32_t* moves;
    // prompts
    const int32_t* cu;  // row offsets of the packed sequences
    int total;
    int extra;  // keys that a unit's start and end cost as much as
    int least;  // keys of a CTA's range at least: two tiles, and over a tile and a block's tokens
    int tile_rows, tile_places, part_rows;  // rows of a tile of a unit, places for them, places of a unit
};

// Entry e of a sequence with page-table row `row`: its page and place.
__device__ __forceinline__ int64_t kv_at(const KvPages& c, int page, int head, int place) {
    return (int64_t)page * c.page + (int64_t)head * c.head + (int64_t)place * c.token;
}

struct KvSeq {
    int slot;   // -1: padding, or refused with an error bit
    int len;    // entries
    int nodes;  // live nodes (attention), path length (accumulation)
    int err;
};

// Sequence b of the call, checked. ATTN: nodes from num_nodes; else from n_path.
template <bool ATTN>
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int b) {
    KvSeq s{-1, 0, 0, 0};
    const int slot = a.slots[b];
    if (slot < 0) return s;
    if (slot >= a.num_slots) {
        s.err = GDN_DEVERR_SLOT;
        return s;
    }
    const int len = a.lengths[slot];
    const int n = ATTN ? (a.num_nodes ? a.num_nodes[b] : a.T) : a.n_path[b];
    if (len < 0 || (int64_t)len > (int64_t)a.max_pages * a.page_size || (!ATTN && len < n)) s.err = KV_DEVERR_LENGTH;
    if (n < 0 || n > (ATTN ? a.T : a.P)) s.err |= KV_DEVERR_NODES;
    if (s.err) return s;
    s.slot = slot, s.len = len, s.nodes = n;
    return s;
}

// Key tiles of one unit of the sequence: the cache's, and for attention one of the drafted nodes.
template <bool ATTN, int KT>
__device__ __forceinline__ int kv_tiles(const KvSeq& s) {
    if (s.slot < 0 || s.nodes == 0) return 0;
    return (s.len + KT - 1) / KT + (ATTN ? 1 : 0);
}

// Blocks of query rows, and units, of the sequence (accumulation takes all rows of a tile at once).
template <bool ATTN>
__device__ __forceinline__ int kv_row_blocks(const KvArgs& a, const KvSeq& s) {
    return ATTN ? (s.nodes * a.G + a.row_block - 1) / a.row_block : 1;
}
// Cost tiles of a unit.
template <bool ATTN, int KT>
__host__ __device__ constexpr int kv_extra() {
    return ATTN ? 2 : 1;
}
// The sequence's share of the line.
template <bool ATTN, int KT>
__device__ __forceinline__ long long kv_seq_cost(const KvArgs& a, const KvSeq& s) {
    const int nt = kv_tiles<ATTN, KT>(s);
    return nt ? (long long)(nt + kv_extra<ATTN, KT>()) * kv_row_blocks<ATTN>(a, s) * a.Hkv : 0;
}

__device__ __forceinline__ long long kv_div(long long a, long long b) {  // a, b >= 0; mostly both fit 32 bits
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line cut into ranges of W / parts, the first W % parts of them one longer. No CTA gets less than
// `least`, so that small calls are not cut into partials that cost more to join than they save.
struct KvSplit {
    long long W, q;
    int parts, r;
    __device__ __forceinline__ KvSplit(long long W_, int grid, int least) : W(W_) {
        const long long most = kv_div(W, least);
        parts = (int)(most < 1 ? 1 : (most < grid ? most : grid));
        q = kv_div(W, parts), r = (int)(W - q * parts);
    }
    __device__ __forceinline__ bool busy(int c) const { return W > 0 && c < parts; }
    __device__ __forceinline__ long long start(int c) const { return q * c + min(c, r); }
    __device__ __forceinline__ int owner(long long t) const {
        const long long head = (q + 1) * r;
        return (int)(t < head ? kv_div(t, q + 1) : r + kv_div(t - head, q));
    }
};

// What the scan over sequences leaves in shared memory.
template <int NT>
struct KvScan {
    KvSeq seq[NT];  // the batch's sequences, where there are at most NT
    long long warp_sum[NT / 32];
    long long before;  // where the found sequence's share of the line begins
    int b;
};

// The split of the batch's tiles and (by the whole block of NT threads) the sequence in which this CTA's
// range begins. Each thread sums a run of sequences; a scan over the block places the runs.
template <bool ATTN, int KT, int NT>
__device__ __forceinline__ KvSplit kv_locate(const KvArgs& a, KvScan<NT>& sc, int grid, int least) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = a.B <= NT ? 1 : (a.B + NT - 1) / NT;
    const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
        const KvSeq s = kv_seq<ATTN>(a, b);
        if (run == 1) sc.seq[b] = s;
        sum += kv_seq_cost<ATTN, KT>(a, s);
    }
    long long inc = sum;
    if (a.B > 1) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(FULL_MASK, inc, o);
            if (lane >= o) inc += y;
        }
    }
    const long long in_warp = __shfl_sync(FULL_MASK, inc, a.B > 1 ? 31 : 0);
    if (lane == 0) sc.warp_sum[warp] = in_warp;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sc.warp_sum[w];
        total += sc.warp_sum[w];
    }
    before += inc - sum;
    const KvSplit split(total, grid, least);
    if (split.busy(blockIdx.x)) {
        const long long want = split.start(blockIdx.x);
        if (want >= before && want < before + sum) {
            int b = b0;
            for (; run > 1 && b < b1; ++b) {
                const long long n = kv_seq_cost<ATTN, KT>(a, kv_seq<ATTN>(a, b));
                if (want < before + n) break;
                before += n;
            }
            sc.b = b, sc.before = before;
        }
    }
    __syncthreads();
    return split;
}

// A walk along a CTA's tiles, segment by segment: a segment is the run of tiles of one unit (key head h,
// row block rb of sequence b) within the CTA's range. Every warp role of a kernel walks by itself.
template <bool ATTN, int KT>
struct KvWalk {
    static constexpr int X = kv_extra<ATTN, KT>();
    const KvArgs& a;
    const KvSeq* seq;  // the batch's sequences in shared memory, or NULL
    long long u0, end;  // where the unit begins on the line, end of the range
    int b, unit, units, blocks, nt;
    KvSeq s;
    int h, rb, t0, t1;  // the segment: tiles t0 .. t1 - 1 of nt
    bool later;         // it is not the CTA's first: its partial is the second one

    // This CTA's range, which begins in sequence sc.b. `some`: it has a tile.
    template <int NT>
    __device__ __forceinline__ KvWalk(const KvArgs& a_, const KvSplit& split, const KvScan<NT>& sc, bool& some)
        : a(a_), seq(a_.B <= NT ? sc.seq : nullptr), later(false) {
        some = split.busy(blockIdx.x);
        t0 = t1 = nt = 0;
        if (!some) return;
        b = sc.b;
        load();
        const long long at = split.start(blockIdx.x), off = at - sc.before;
        end = split.start(blockIdx.x + 1);
        unit = (int)kv_div(off, nt + X);
        const int p = (int)(off - (long long)unit * (nt + X));
        u0 = at - p;
        segment(max(0, p - X));
        some = t1 > t0;  // not where the whole range is cost tiles
    }
    __device__ __forceinline__ void load() {
        s = seq ? seq[b] : kv_seq<ATTN>(a, b);
        nt = kv_tiles<ATTN, KT>(s), blocks = kv_row_blocks<ATTN>(a, s), units = a.Hkv * blocks;
    }
    __device__ __forceinline__ void segment(int tile) {
        h = unit / blocks, rb = unit - h * blocks;
        t0 = tile, t1 = (int)max(0ll, min((long long)nt, end - u0 - X));
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    __device__ __forceinline__ bool last() const { return end - (u0 + nt + X) <= X; }
    // The next segment; false at the end of the range.
    __device__ __forceinline__ bool next() {
        if (last()) return false;
        u0 += nt + X, later = true;
        if (++unit == units) {
            unit = 0;
            do {
                ++b;
                load();
            } while (nt == 0);
        }
        segment(0);
        return true;
    }
};

// A unit that goes on past the end of a CTA's range: what the join needs, one record a CTA.
struct KvBorder {
    int b, h, r0, rows;  // rows 0: the range ends between units
    int c0, n;           // the unit's CTAs are c0 .. c0 + n - 1
    int second;          // the unit begins within CTA c0's range, after another: its partial there is the second
    int pad;
};

// Record of this CTA's last segment, by one thread.
template <bool ATTN, int KT>
__device__ __forceinline__ KvBorder kv_border(const KvArgs& a, const KvSplit& split, const KvWalk<ATTN, KT>& w) {
    KvBorder k{};
    if (w.t1 == w.nt) return k;
    const long long first = w.u0 + w.X;
    k.b = w.b, k.h = w.h, k.r0 = w.rb * a.row_block, k.rows = min(a.row_block, w.s.nodes * a.G - k.r0);
    k.c0 = split.owner(first), k.n = split.owner(first + w.nt - 1) - k.c0 + 1;
    k.second = split.start(k.c0) < w.u0;
    return k;
}

// Every page of the sequence's entries is a page of the pool (all threads of a group of `n` ask, each
// a part; the caller joins the answers).
__device__ __forceinline__ bool kv_pages_ok(const KvArgs& a, const KvSeq& s, int tid, int n) {
    const int32_t* row = a.page_table + (int64_t)s.slot * a.max_pages;
    const int used = (s.len + a.page_size - 1) / a.page_size;
    bool ok = true;
    for (int i = tid; i < used; i += n) ok = ok && (uint32_t)row[i] < (uint64_t)a.num_pages;
    return ok;
}

// Outputs of rows that no unit computes: padding, refused sequences, nodes past a sequence's count; by
// `n` threads of each CTA, of which this is thread `i`. Error bits of refused sequences are set here,
// once a call.
__device__ __forceinline__ void kv_empty_rows(const KvArgs& a, const KvSeq* seq, int i, int n) {
    const int64_t row_bytes = (int64_t)a.d * dtype_size(a.dtype);
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && row_bytes % 16 == 0;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const KvSeq s = seq ? seq[b] : kv_seq<true>(a, b);
        if (s.err && i == 0) set_error(a.dev_err, s.err);
        if (s.nodes == a.T) continue;
        const int64_t r0 = ((int64_t)b * a.T + s.nodes) * a.Hq, r1 = ((int64_t)b + 1) * a.T * a.Hq;
        char* o = static_cast<char*>(a.out) + r0 * row_bytes;
        const int64_t bytes = (r1 - r0) * row_bytes;
        if (vec)
            for (int64_t x = (int64_t)i * 16; x < bytes; x += (int64_t)n * 16)
                *reinterpret_cast<uint4*>(o + x) = make_uint4(0, 0, 0, 0);
        else  // 2-byte words: a 16-bit output of odd d starts its rows on 2-byte boundaries
            for (int64_t x = (int64_t)i * 2; x < bytes; x += (int64_t)n * 2) *reinterpret_cast<uint16_t*>(o + x) = 0;
        if (a.lse)
            for (int64_t r = r0 + i; r < r1; r += n) a.lse[r] = -INFINITY;
    }
}

__device__ __forceinline__ float kv_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Floats of one partial: row_block rows of d outputs, their maxima and their sums (16-byte blocks). A sum
// of -1 says that the CTA met a page outside the pool: the unit's rows are those of a refused sequence.
__host__ __device__ inline int64_t kv_part_floats(int row_block, int d) { return ((int64_t)row_block * (d + 2) + 3) / 4 * 4; }

__host__ __device__ inline int64_t kv_part_bytes(int64_t grid, int row_block, int d) {
    return grid * 2 * kv_part_floats(row_block, d) * 4;
}

// The join kernel is launched while the attention kernel runs (programmatic launch): the attention
// kernel's blocks let it start, and every block of it waits here until the attention kernel has ended
// and its writes are visible.
__device__ __forceinline__ void kv_grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void kv_grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Eviction's move lists in the workspace: for unit (b, h) a count (-1: the sequence stays as it is),
// and after four words up to `cap` holes and as many fillers.
__host__ __device__ inline int64_t kv_moves_at(int64_t unit, int cap) {
    return unit * (4 + 2 * (int64_t)align_up(cap, 4));
}
// Most moves of a unit: a hole lies below the budget, a filler at or above it.
__host__ __device__ inline int kv_moves_cap(int max_pages, int page_size, int budget) {
    const int room = max_pages * page_size;
    const int over = room > budget ? room - budget : 0;
    return over < budget ? over : budget;
}

// Norm, rotation and append.
struct KvTurn {  // one side's rows
    const void* in;
    void* out;
    int64_t in_seq, in_node, in_head, out_seq, out_node, out_head;
    const float* norm;
    int64_t norm_head;
};

struct KvRotateArgs {
    KvTurn q, k, v;  // (in NULL: none; v: values, copied; of an append the keys and values go to the cache)
    const uint64_t* turns;
    const int32_t* axis;
    const int32_t* positions;
    float eps, offset;
    int rot, axes, interleaved;
    int tokens;  // B T, or the rows of an append
    int T, Hq, Hkv, d, dtype;
    int log_block;  // of the tokens of a block
};

// Compaction's workspace: held pages, a bit each; where each page above the border goes; the pages that move, in order.
struct KvPlan {
    uint32_t* bits;
    int32_t *to, *hole, *mover, *head;  // head: pages that move (-1: refused), pages held
    int words;
};
__host__ __device__ inline int64_t kv_plan_words(int64_t num_pages) { return (num_pages + 31) / 32; }
__host__ __device__ inline int64_t kv_plan_ints(int64_t num_pages) { return 8 + kv_plan_words(num_pages) + 3 * num_pages; }
__host__ __device__ inline KvPlan kv_plan(int32_t* ws, int64_t num_pages) {
    KvPlan p;
    p.words = (int)kv_plan_words(num_pages);
    p.head = ws, p.bits = reinterpret_cast<uint32_t*>(ws + 8);
    p.to = ws + 8 + p.words, p.hole = p.to + num_pages, p.mover = p.hole + num_pages;
    return p;
}

}  // namespace gdn
