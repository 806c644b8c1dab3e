// kv_rotate.cuh -- norm of each head's row, position rotation, and the append of
// a prompt's keys and values to the paged cache.
//
// Mathematics. y = x rsqrt(mean x^2 + eps) (w + offset); pairs of y turned by
// position times a frequency. The frequency is a 64-bit fraction of a turn, so
// that the product's low 64 bits are that fraction's angle modulo a turn, exactly;
// its upper 32 bits, as a signed number, go to sincospif.
//
// Shape: a block takes a few tokens. Their angles' cosines and sines are formed
// once, into shared memory (rot / 2 pairs a token serve all its heads), beside the
// places of the entries; then groups of LP lanes take rows (query heads, key
// heads, values of a token), a lane eight elements. The two elements of a pair are
// the same register of two lanes where the halves are a multiple of eight (one
// shuffle each), or neighbours in one lane (interleaved). Other sizes and
// alignments take the scalar form: a warp a row, the row in shared memory.
// Bound by HBM: each element is read and written once. 20000 tokens of 32 + 8 heads (d =
// 128, bf16, 0.41 GB) take 78.5 us, 5.2 TB/s or 0.77 of the measured copy bandwidth; an
// append of 37000 tokens of 8 prompts with queries (fp16, 0.93 GB) 182 us, 5.1 TB/s. (A
// row's token, side and head found anew for each row took 267 instructions a warp and
// row, and 127 us; places, angles and weights now stay with a group of lanes.) In halves
// they take 86 us, in fp32 139 (5.9 TB/s). The rotation's 48 registers (for a fifth block
// a SM) spill 76 bytes of stores and 96 of loads a thread, 1.7% of its instructions.
// The scalar form is bound by its instructions, a 2-byte load and store an element of a
// lane: 20000 tokens take 427 us at d = 96 with 24 turned and 418 at d = 80 with 40, 0.7
// and 0.6 TB/s, where the vector form of the same rows takes 81 and 78 with all turned.
#pragma once

#include "kv_common.cuh"

namespace gdn {

namespace kvr {

constexpr int NT = 256, WARPS = NT / 32;
constexpr int MAX_TOKENS = 16;   // of a block
constexpr int MAX_PAIRS = 2048;  // cosines (and sines) of a block
constexpr int SEQS = 1024;       // offsets that the block keeps in shared memory
constexpr int LANE = 8;          // elements of a lane

// Eight elements of a row, as they lie.
template <typename ST>
struct Eight {
    static constexpr int N = sizeof(ST) / 2;
    uint4 w[N];
    __device__ __forceinline__ void clear() {
        for (int i = 0; i < N; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const ST* p) {
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(ST* p) const {
        for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void unpack(float* x) const {
        for (int i = 0; i < N; ++i) Store<ST>::unpack(w[i], x + i * Store<ST>::VEC);
    }
    __device__ __forceinline__ void pack(const float* x) {
        for (int i = 0; i < N; ++i) w[i] = Store<ST>::pack(x + i * Store<ST>::VEC);
    }
};

struct Place {
    int64_t k, v, w;  // element offsets of the entry of head 0; its weight
    int32_t stamp;
    int live;  // 1: all of it, 2: queries alone (its page is missing), 0: zeros, -1: no sequence's row
    int first;  // position where none are given
};

}  // namespace kvr

__device__ __forceinline__ float2 kv_cos_sin(const uint64_t turns, int position) {
    const uint64_t a = turns * (uint64_t)(int64_t)position;
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: halves of a turn
    return make_float2(c, s);
}

// Whether the call's offsets are in order, by the whole block; with B small they are left in `cu`.
template <int NT>
__device__ __forceinline__ bool kv_offsets_ok(const KvArgs& a, int* cu, int most) {
    bool ok = true;
    for (int b = threadIdx.x; b <= a.B; b += NT) {
        const int x = a.cu[b], next = a.cu[b < a.B ? b + 1 : b];
        ok = ok && x >= 0 && x <= next && next <= a.total;
        if (a.B < most) cu[b] = x;
    }
    return __syncthreads_and(ok);
}

// Where row t of an append goes, by one thread.
__device__ __forceinline__ kvr::Place kv_place(const KvArgs& c, const int* cu, int t) {
    kvr::Place p{0, 0, 0, 0, -1, 0};
    if (t < cu[0] || t >= cu[c.B]) return p;
    int lo = 0, hi = c.B;  // the last sequence that begins at or before t and holds a row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int slot = c.slots[lo], first = cu[lo], n = cu[lo + 1] - first, j = t - first;
    p.live = 0;
    if (slot < 0 || slot >= c.num_slots) return p;
    const int len = c.lengths[slot];
    if (len < 0 || (int64_t)len + n > (int64_t)c.max_pages * c.page_size) return p;
    const int e = len + j, pg = e / c.page_size, page = c.page_table[(int64_t)slot * c.max_pages + pg], at = e - pg * c.page_size;
    p.first = p.stamp = (c.counts ? c.counts[slot] : len) + j;
    p.live = 2;
    if ((uint32_t)page >= (uint64_t)c.num_pages) return p;
    p.live = 1;
    p.k = (int64_t)page * c.k.page + (int64_t)at * c.k.token, p.v = (int64_t)page * c.v.page + (int64_t)at * c.v.token;
    p.w = (int64_t)page * c.Hkv * c.page_size + at;
    return p;
}

// ST: element type; LP: lanes a row (eight elements a lane), or 0 for the scalar form; APPEND: c is the cache.
template <typename ST, int LP, bool APPEND>
__global__ void __launch_bounds__(kvr::NT, LP > 0 ? (APPEND ? 4 : 5) : 1) kv_rotate_kernel(const __grid_constant__ KvRotateArgs a, const __grid_constant__ KvArgs c) {
    using namespace kvr;
    __shared__ __align__(16) float s_cos[MAX_PAIRS], s_sin[MAX_PAIRS];
    __shared__ Place s_place[APPEND ? MAX_TOKENS : 1];
    __shared__ int s_cu[APPEND ? SEQS : 1];
    __shared__ float s_row[LP == 0 ? WARPS : 1][LP == 0 ? KV_MAX_D : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x << a.log_block, tokens = min(1 << a.log_block, a.tokens - t0), half = a.rot / 2;
    // rows of a token: queries, keys, values; row r is that of token r % 2^log_block
    const int nq = a.q.in ? a.Hq : 0, nk = a.k.in ? a.Hkv : 0, per = nq + nk + (a.v.in ? a.Hkv : 0), rows = per << a.log_block;
    const auto side_of = [&](int y) { return y < nq ? 0 : y < nq + nk ? 1 : 2; };
    const auto head_of = [&](int y, int side) { return y - (side == 0 ? 0 : side == 1 ? nq : nq + nk); };
    const auto turn_of = [&](int side) -> const KvTurn& { return side == 0 ? a.q : side == 1 ? a.k : a.v; };
    const auto offset = [&](int tok, int64_t seq, int64_t node) {
        if (a.T == 1) return tok * seq;  // (tokens in one stride)
        const int b = tok / a.T;
        return b * seq + (tok - b * a.T) * node;
    };
    const auto in_of = [&](int r) {
        const int y = r >> a.log_block, side = side_of(y);
        const KvTurn& s = turn_of(side);
        return static_cast<const ST*>(s.in) + offset(t0 + (r & ((1 << a.log_block) - 1)), s.in_seq, s.in_node) +
               (int64_t)head_of(y, side) * s.in_head;
    };
    const auto there = [&](int r) { return r < rows && (r & ((1 << a.log_block) - 1)) < tokens; };

    if constexpr (APPEND) {
        kv_grid_launch();
        if (!kv_offsets_ok<NT>(c, s_cu, SEQS)) return;
        if (tid < tokens) s_place[tid] = kv_place(c, c.B < SEQS ? s_cu : c.cu, t0 + tid);
        if (!a.positions) __syncthreads();
    }
    for (int i = tid; i < tokens * half; i += NT) {
        const int t = i / half, x = i - t * half;
        int ax = a.axis ? a.axis[x] : 0;
        if ((uint32_t)ax >= (uint32_t)a.axes) ax = 0;
        int pos;
        if (!APPEND || a.positions) pos = a.positions[(int64_t)ax * a.tokens + t0 + t];
        else pos = s_place[t].first;
        const float2 cs = kv_cos_sin(a.turns[x], pos);
        s_cos[i] = cs.x, s_sin[i] = cs.y;
    }
    __syncthreads();
    // where row r goes (NULL: nowhere), and whether as zeros
    const auto out_of = [&](int r, bool& zero) -> ST* {
        const int y = r >> a.log_block, side = side_of(y), t = r & ((1 << a.log_block) - 1), h = head_of(y, side);
        const KvTurn& s = turn_of(side);
        ST* out = static_cast<ST*>(s.out) + (int64_t)h * s.out_head;
        zero = false;
        if constexpr (APPEND) {
            const Place& p = s_place[t];
            zero = p.live == 0;
            if (side > 0) return p.live != 1 ? nullptr : out + (side == 1 ? p.k : p.v);
            if (p.live < 0) return nullptr;
        }
        return out + offset(t0 + t, s.out_seq, s.out_node);
    };
    if constexpr (LP > 0) {
        // A group of lanes stays with one token of the block: places, angles and weights are in registers, and the next
        // row is a step of whole heads away.
        constexpr int GROUPS = NT / LP, AHEAD = 2;
        const int sub = tid % LP, e0 = sub * LANE, group = tid / LP, t = group & ((1 << a.log_block) - 1), h0 = group >> a.log_block;
        const int step = GROUPS >> a.log_block;  // (a block has no more tokens than groups)
        const bool in = e0 < a.d && t < tokens, first = e0 < half, turned = e0 < a.rot;
        const int partner = first ? sub + half / LANE : turned ? sub - half / LANE : sub;
        const float mean = 1.f / (float)a.d;
        float co[LANE], si[LANE];  // of this lane's elements; interleaved: of its four pairs
#pragma unroll
        for (int e = 0; e < LANE; ++e) co[e] = 1.f, si[e] = 0.f;
        if (turned && t < tokens) {
            const int i = t * half + (a.interleaved ? e0 / 2 : first ? e0 : e0 - half);
#pragma unroll
            for (int e = 0; e < LANE; e += 4) {
                if (a.interleaved && e > 0) break;
                const float4 x = *reinterpret_cast<const float4*>(s_cos + i + e), y = *reinterpret_cast<const float4*>(s_sin + i + e);
                const float z = a.interleaved || !first ? 1.f : -1.f;  // (of halves: the other element's share, signed)
                co[e] = x.x, co[e + 1] = x.y, co[e + 2] = x.z, co[e + 3] = x.w;
                si[e] = z * y.x, si[e + 1] = z * y.y, si[e + 2] = z * y.z, si[e + 3] = z * y.w;
            }
        }
        const auto rows_of = [&](const KvTurn& s, int heads, int side) {
            const ST* from = static_cast<const ST*>(s.in) + offset(t0 + t, s.in_seq, s.in_node) + (int64_t)h0 * s.in_head + e0;
            ST* to = static_cast<ST*>(s.out) + (int64_t)h0 * s.out_head + e0;
            bool zero = false, write = in;
            if constexpr (APPEND) {
                const Place& p = s_place[t];
                zero = p.live == 0, write = in && (side > 0 ? p.live == 1 : p.live >= 0);
                if (side > 0) to += side == 1 ? p.k : p.v;
            }
            if (!APPEND || side == 0) to += offset(t0 + t, s.out_seq, s.out_node);
            const int64_t from_step = step * s.in_head, to_step = step * s.out_head;
            const bool norm = side < 2 && s.norm, turn = side < 2 && half > 0;
            float w[LANE];
            const auto weights = [&](int h) {
#pragma unroll
                for (int e = 0; e < LANE; e += 4) {
                    float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (in && h < heads) g = *reinterpret_cast<const float4*>(s.norm + (int64_t)h * s.norm_head + e0 + e);
                    w[e] = g.x + a.offset, w[e + 1] = g.y + a.offset, w[e + 2] = g.z + a.offset, w[e + 3] = g.w + a.offset;
                }
            };
            if (norm) weights(h0);
#pragma unroll 1
            for (int i = 0; i * step < heads; i += AHEAD) {  // (the same trips for every lane)
                Eight<ST> raw[AHEAD];
#pragma unroll
                for (int y = 0; y < AHEAD; ++y) {
                    raw[y].clear();
                    if (write && !zero && h0 + (i + y) * step < heads) raw[y].load(from);
                    from += from_step;
                }
#pragma unroll
                for (int y = 0; y < AHEAD; ++y) {
                    const int h = h0 + (i + y) * step;
                    if (norm || turn) {
                        float x[LANE];
                        raw[y].unpack(x);
                        if (norm) {
                            if (s.norm_head && i + y > 0) weights(h);
                            float ss = 0.f;
#pragma unroll
                            for (int e = 0; e < LANE; ++e) ss = fmaf(x[e], x[e], ss);
                            ss = group_sum<LP>(ss);
                            const float f = rsqrtf(ss * mean + a.eps);
#pragma unroll
                            for (int e = 0; e < LANE; ++e) x[e] *= f * w[e];
                        }
                        if (turn && a.interleaved) {
                            if (turned) {
#pragma unroll
                                for (int e = 0; e < LANE; e += 2) {
                                    const float p = x[e], q = x[e + 1];
                                    x[e] = p * co[e / 2] - q * si[e / 2], x[e + 1] = p * si[e / 2] + q * co[e / 2];
                                }
                            }
                        } else if (turn) {
#pragma unroll
                            for (int e = 0; e < LANE; ++e) {
                                const float o = __shfl_sync(FULL_MASK, x[e], partner, LP);
                                if (turned) x[e] = fmaf(o, si[e], x[e] * co[e]);
                            }
                        }
                        raw[y].pack(x);
                    }
                    if (zero) raw[y].clear();
                    if (write && h < heads) raw[y].store(to);
                    to += to_step;
                }
            }
        };
        if (nq) rows_of(a.q, a.Hq, 0);
        if (nk) rows_of(a.k, a.Hkv, 1);
        if (a.v.in) rows_of(a.v, a.Hkv, 2);
    } else {
        float* line = s_row[warp];
        for (int r = warp; r < rows; r += WARPS) {
            if (!there(r)) continue;
            const int y = r >> a.log_block, side = side_of(y), t = r & ((1 << a.log_block) - 1);
            const KvTurn& s = turn_of(side);
            bool zero;
            ST* out = out_of(r, zero);
            if (!out) continue;
            const ST* from = in_of(r);
            if (zero || side == 2 || (!s.norm && half == 0)) {
                for (int e = lane; e < a.d; e += 32) out[e] = zero ? ST(0.f) : from[e];
                continue;
            }
            float ss = 0.f;
            for (int e = lane; e < a.d; e += 32) {
                const float x = load_elem(from, e, Store<ST>::code);
                line[e] = x, ss = fmaf(x, x, ss);
            }
            ss = group_sum<32>(ss);
            __syncwarp();
            if (s.norm) {
                const float f = rsqrtf(ss / (float)a.d + a.eps);
                const float* norm = s.norm + (int64_t)head_of(y, side) * s.norm_head;
                for (int e = lane; e < a.d; e += 32) line[e] *= f * (norm[e] + a.offset);
                __syncwarp();
            }
            for (int e = lane; e < a.d; e += 32) {
                float z = line[e];
                if (e < a.rot) {
                    const bool one = a.interleaved ? (e & 1) == 0 : e < half;
                    const int i = a.interleaved ? e >> 1 : one ? e : e - half;
                    const float other = line[a.interleaved ? e ^ 1 : one ? e + half : e - half];
                    const float co = s_cos[t * half + i], si = s_sin[t * half + i];
                    z = one ? z * co - other * si : other * si + z * co;
                }
                store_elem(out, e, Store<ST>::code, z);
            }
            __syncwarp();
        }
    }
    if constexpr (APPEND) {
        if (c.weights)
            for (int i = tid; i < tokens * c.Hkv; i += NT) {
                const int t = i / c.Hkv, h = i - t * c.Hkv;
                const Place& p = s_place[t];
                if (p.live != 1) continue;
                const int64_t w = p.w + (int64_t)h * c.page_size;
                c.weights[w] = 0.f, c.stamps[w] = p.stamp;
            }
    }
}

// Behind an append: a warp a sequence looks at all its new pages, and its length and count grow.
constexpr int KV_GROW_NT = 128;
__global__ void __launch_bounds__(KV_GROW_NT) kv_grow_kernel(const __grid_constant__ KvArgs c) {
    kv_grid_wait();  // the rows are written, and nobody reads the lengths any more
    const bool ok = kv_offsets_ok<KV_GROW_NT>(c, nullptr, 0);
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(c.dev_err, GDN_DEVERR_SEQLEN);
        return;
    }
    const int lane = threadIdx.x & 31, b = blockIdx.x * (KV_GROW_NT / 32) + (threadIdx.x >> 5);
    if (b >= c.B) return;
    const int slot = c.slots[b], n = c.cu[b + 1] - c.cu[b];
    if (slot < 0) return;
    int err = 0, len = 0;
    if (slot >= c.num_slots) err = GDN_DEVERR_SLOT;
    if (!err) {
        len = c.lengths[slot];
        if (len < 0 || (int64_t)len + n > (int64_t)c.max_pages * c.page_size) err = KV_DEVERR_LENGTH;
    }
    if (!err && n > 0) {
        const int32_t* row = c.page_table + (int64_t)slot * c.max_pages;
        bool bad = false;
        for (int i = len / c.page_size + lane; i <= (len + n - 1) / c.page_size; i += 32)
            bad = bad || (uint32_t)row[i] >= (uint64_t)c.num_pages;
        if (__any_sync(FULL_MASK, bad)) err = KV_DEVERR_PAGE;
    }
    if (lane != 0) return;
    if (err) {
        set_error(c.dev_err, err);
    } else if (n > 0) {
        c.lengths[slot] = len + n;
        if (c.counts) c.counts[slot] += n;
    }
}

}  // namespace gdn
