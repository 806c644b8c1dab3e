// kv_prompt.cuh -- what the prompt attention kernels share: the division of packed
// causal prompts over a persistent grid, and rows that no unit computes.
//
// Units. The rows of a sequence and key head are its tokens' heads of the group,
// token by token (row = token * G + head). A unit is a block of RB of them (the call's
// row_block); its keys end behind its last token, so that blocks grow along a prompt.
//
// Division. All units in order (sequence, key head, block) make a line, a unit as
// long as its keys and a few more (the call's extra) that stand for what it costs beyond its
// tiles, and CTA c of `parts` takes [W c / parts, W (c + 1) / parts) of it: every CTA
// has the same work, whatever the lengths, and neighbours read the same keys. In
// units of a G-th key the length of block i is G (prefix + extra) + RB (i + 1), so
// its place on the line is a quadratic in i: a CTA finds its range without a walk. A
// unit that a border cuts is cut between tiles, and leaves one partial result a CTA
// (unnormalised outputs, maximum and sum), joined by kp_join_kernel (kv_prompt_join.cuh).
#pragma once

#include "kv_common.cuh"

namespace gdn {

struct KpSeq {
    int slot;   // -1: padding, or refused with an error bit
    int first;  // its first row
    int n, len;  // rows, entries
    int err;
    bool owned;  // the offsets are in order: its rows are its own
};

__device__ __forceinline__ KpSeq kp_seq(const KvArgs& a, int b) {
    KpSeq s{-1, 0, 0, 0, 0, true};
    const int first = a.cu[b], end = a.cu[b + 1], slot = a.slots[b];
    if (first < 0 || end < first || end > a.total) {
        s.err = GDN_DEVERR_SEQLEN, s.owned = false;
        return s;
    }
    s.first = first, s.n = end - first;
    if (slot < 0) return s;
    if (slot >= a.num_slots) {
        s.err = GDN_DEVERR_SLOT;
        return s;
    }
    const int len = a.lengths[slot];
    if (len < s.n || (int64_t)len > (int64_t)a.max_pages * a.page_size) {
        s.err = KV_DEVERR_LENGTH;
        return s;
    }
    s.slot = slot, s.len = len;
    return s;
}

// Blocks of a sequence, and the length of the line before block i of a key head.
__device__ __forceinline__ int kp_blocks(const KvArgs& a, const KpSeq& s) {
    return s.slot < 0 ? 0 : (int)((uint32_t)(s.n * a.G + a.row_block - 1) / (uint32_t)a.row_block);
}
__device__ __forceinline__ long long kp_before(const KvArgs& a, const KpSeq& s, long long i) {
    return i * ((long long)a.G * (s.len - s.n + a.extra)) + a.row_block * (i * (i + 1) / 2);
}
__device__ __forceinline__ long long kp_seq_cost(const KvArgs& a, const KpSeq& s) {
    return kp_before(a, s, kp_blocks(a, s)) * a.Hkv;
}

// A place between tiles: in sequence b, key head h, block i, ahead of tile t.
struct KpPlace {
    int b, h, i, t;
};

// What the scan over sequences leaves in shared memory: the CTA's range.
struct KpMark {
    long long off;  // from the beginning of sequence b's share of the line
    int b;          // a.B: the end of the line
};
template <int NT, int KEEP>
struct KpScan {
    static constexpr int keep = KEEP;
    KpSeq seq[KEEP];  // the batch's sequences, where there are at most KEEP (which is at most NT)
    long long warp_sum[NT / 32];
    KpMark mark[2];  // beginning and end of the range
    KpPlace place[2];  // and between which tiles they lie
    long long q;     // ranges: length, and how many are one longer
    int r, parts;
};

// Tiles of block `blk`: keys 0 .. prefix + last token.
template <int KT>
__device__ __forceinline__ int kp_tiles(const KvArgs& a, const KpSeq& x, int blk) {
    const int rows = (int)min((long long)x.n * a.G, (long long)(blk + 1) * a.row_block);
    return (x.len - x.n + (rows - 1) / a.G + KT) / KT;
}
// The place that a point of the line is cut at.
template <int KT>
__device__ __forceinline__ KpPlace kp_place(const KvArgs& a, const KpMark& m, const KpSeq& x) {
    const int nb = kp_blocks(a, x);
    const long long one = kp_before(a, x, nb);
    KpPlace p{m.b, (int)kv_div(m.off, one), 0, 0};
    const long long off = m.off - one * p.h;
    int lo = 0, hi = nb;  // the block that holds `off`
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (kp_before(a, x, mid) <= off) lo = mid;
        else hi = mid;
    }
    p.i = lo;
    const long long in = off - kp_before(a, x, lo) - (long long)a.extra * a.G;
    // (at the last tile at most: its CTA is the one that ends the unit)
    if (in > 0) p.t = (int)min(kv_div(in, (long long)KT * a.G), (long long)kp_tiles<KT>(a, x, lo) - 1);
    return p;
}

// By the whole block of NT threads: the division, and this CTA's range.
template <int KT, int NT, int KEEP>
__device__ __forceinline__ void kp_locate(const KvArgs& a, KpScan<NT, KEEP>& sc) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = a.B <= NT ? 1 : (a.B + NT - 1) / NT;
    const int b0 = (int)min((long long)a.B, (long long)tid * run), b1 = min(a.B, b0 + run);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
        const KpSeq s = kp_seq(a, b);
        if (a.B <= KEEP) sc.seq[b] = s;
        sum += kp_seq_cost(a, s);
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(FULL_MASK, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sc.warp_sum[warp] = inc;
    if (tid < 2) sc.mark[tid].b = a.B, sc.mark[tid].off = 0;
    __syncthreads();
    long long before = inc - sum, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sc.warp_sum[w];
        total += sc.warp_sum[w];
    }
    const long long most = kv_div(total, (long long)a.least * a.G);
    const int parts = (int)(most < 1 ? 1 : most < gridDim.x ? most : gridDim.x);
    const long long q = kv_div(total, parts);
    const int r = (int)(total - q * parts), c = blockIdx.x;
    if (tid == 0) sc.q = q, sc.r = r, sc.parts = parts;
    for (int side = 0; side < 2; ++side) {
        const int x = c + side;
        if (x > parts) break;
        const long long want = q * x + min(x, r);
        if (want >= before && want < before + sum) {
            long long at = before;
            int b = b0;
            for (; b < b1 - 1; ++b) {
                const long long n = kp_seq_cost(a, a.B <= KEEP ? sc.seq[b] : kp_seq(a, b));
                if (want < at + n) break;
                at += n;
            }
            sc.mark[side].b = b, sc.mark[side].off = want - at;
        }
    }
    __syncthreads();
    if (lane == 0 && warp < 2) {  // (beside one another: a place takes a search)
        const KpMark m = sc.mark[warp];
        if (m.b < a.B) sc.place[warp] = kp_place<KT>(a, m, a.B <= KEEP ? sc.seq[m.b] : kp_seq(a, m.b));
        else sc.place[warp] = KpPlace{a.B, 0, 0, 0};
    }
    __syncthreads();
}

// A walk along a CTA's segments: runs of tiles of one unit.
template <int KT>
struct KpWalk {
    const KvArgs& a;
    const KpSeq* seq;  // the batch's sequences in shared memory, or NULL
    KpPlace end;
    int b, h, i, blocks;
    KpSeq s;
    int nt, t0, t1;  // the unit's tiles, and the segment's

    __device__ __forceinline__ KpSeq get(int x) const { return seq ? seq[x] : kp_seq(a, x); }
    __device__ __forceinline__ bool before_end() const {
        return b < end.b || (b == end.b && (h < end.h || (h == end.h && i <= end.i)));
    }
    __device__ __forceinline__ void load() {
        s = get(b);
        blocks = kp_blocks(a, s);
    }
    // The segment of the current unit from tile t on; false if the range ends ahead of it.
    __device__ __forceinline__ bool segment(int t) {
        if (!before_end() || b >= a.B) return false;
        nt = kp_tiles<KT>(a, s, i), t0 = t;
        t1 = b == end.b && h == end.h && i == end.i ? min(end.t, nt) : nt;
        return true;
    }
    template <int NT, int KEEP>
    __device__ __forceinline__ KpWalk(const KvArgs& a_, const KpScan<NT, KEEP>& sc, bool& some)
        : a(a_), seq(a_.B <= KEEP ? sc.seq : nullptr) {
        t0 = t1 = nt = 0;
        some = false;
        if ((int)blockIdx.x >= sc.parts) return;
        const KpPlace from = sc.place[0];
        end = sc.place[1];
        b = from.b, h = from.h, i = from.i;
        if (b >= a.B) return;
        load();
        some = segment(from.t);
        if (some && t0 >= t1) some = next();
    }
    __device__ __forceinline__ bool step() {  // to the next unit
        if (++i == blocks) {
            i = 0;
            if (++h == a.Hkv) {
                h = 0;
                do {
                    if (++b >= a.B) return false;
                    load();
                } while (blocks == 0);
            }
        }
        return true;
    }
    // The next segment with a tile; false at the end of the range.
    __device__ __forceinline__ bool next() {
        do {
            if (!step() || !segment(0)) return false;
        } while (t0 >= t1);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    // Which of the CTA's two partials the segment's is: only its first segment begins inside a unit.
    __device__ __forceinline__ int later() const { return t0 == 0; }
    __device__ __forceinline__ int r0() const { return i * a.row_block; }
    __device__ __forceinline__ int rows() const { return min(a.row_block, s.n * a.G - r0()); }
};

// A unit cut by the end of the CTA's range in which it begins: what the join needs, one record a CTA.
struct KpBorder {
    int first, h, r0, rows, n;  // the sequence's first row, and CTAs of the unit: this one and n - 1 behind it (0: none)
    int pad[3];
};

// Writes this CTA's record: of the segment `w`, if the unit begins in it and goes on past the range (which is then at
// its end, sc.mark[1] inside the unit), else that there is none. By one thread.
template <int KT, int NT, int KEEP>
__device__ __forceinline__ void kp_border(const KvArgs& a, const KpScan<NT, KEEP>& sc, const KpWalk<KT>& w) {
    KpBorder k{};
    k.first = w.s.first, k.h = w.h, k.r0 = w.r0(), k.rows = w.rows(), k.n = 1;
    const long long u0 = kp_before(a, w.s, w.blocks) * w.h + kp_before(a, w.s, w.i);  // in its sequence's share
    const long long size = kp_before(a, w.s, w.i + 1) - kp_before(a, w.s, w.i), at = sc.mark[1].off - u0;
    const auto start = [&](int x) { return sc.q * x + min(x, sc.r); };
    const int c = blockIdx.x;
    // each CTA whose range begins inside the unit has one of its tiles: a range is as long as two tiles, and longer than
    // the last tile and what the line counts behind it (a block's rows that the sequence has no more)
    for (int x = c + 1; x < sc.parts; ++x) {
        ++k.n;
        if (at + start(x + 1) - start(c + 1) >= size) break;
    }
    static_cast<KpBorder*>(a.border)[blockIdx.x] = k;
}
__device__ __forceinline__ void kp_no_border(const KvArgs& a) { static_cast<KpBorder*>(a.border)[blockIdx.x].n = 0; }

// Rows of sequences that no unit computes (padding, refused), by `n` threads of each CTA, of which this is
// thread `i`. Error bits of refused sequences are set here, once a call.
__device__ __forceinline__ void kp_empty_rows(const KvArgs& a, const KpSeq* seq, int i, int n) {
    const int64_t row_bytes = (int64_t)a.Hq * a.d * dtype_size(a.dtype);
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && row_bytes % 16 == 0;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const KpSeq s = seq ? seq[b] : kp_seq(a, b);
        if (s.err && i == 0) set_error(a.dev_err, s.err);
        if (s.slot >= 0 || !s.owned) continue;
        char* o = static_cast<char*>(a.out) + s.first * row_bytes;
        const int64_t bytes = s.n * row_bytes;
        if (vec)
            for (int64_t x = (int64_t)i * 16; x < bytes; x += (int64_t)n * 16)
                *reinterpret_cast<uint4*>(o + x) = make_uint4(0, 0, 0, 0);
        else
            for (int64_t x = (int64_t)i * 2; x < bytes; x += (int64_t)n * 2) *reinterpret_cast<uint16_t*>(o + x) = 0;
        if (a.lse)
            for (int64_t r = (int64_t)s.first * a.Hq + i; r < ((int64_t)s.first + s.n) * a.Hq; r += n) a.lse[r] = -INFINITY;
    }
}

// Partials: column e of the outputs of a unit's places, then the rows' maxima and sums. A unit's rows lie in tiles of
// tile_rows, each in the first of tile_places places. A sum of -1 says that the CTA
// met a page outside the pool (or gave up): the unit's rows are those of a refused sequence.
__host__ __device__ inline int64_t kp_part_floats(int places, int d) { return (int64_t)places * (d + 2); }
__host__ __device__ inline int64_t kp_part_bytes(int64_t grid, int places, int d) {
    return grid * 2 * kp_part_floats(places, d) * 4;
}

}  // namespace gdn
