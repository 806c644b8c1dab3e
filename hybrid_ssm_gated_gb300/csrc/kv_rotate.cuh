// kv_rotate.cuh -- norm of each head's row, position rotation, and the append of
// a prompt's keys and values to the paged cache.
//
// Mathematics. y = x rsqrt(mean x^2 + eps) (w + offset); pairs of y turned by
// position times a frequency. The frequency is a 64-bit fraction of a turn, so
// that the product's low 64 bits are the angle modulo a turn, off by 2^-65 turns
// a position; its upper 32 bits, as a signed number, go to sincospif.
//
// Shape: a block takes a few tokens. Their angles' cosines and sines are formed
// once, into shared memory (rot / 2 pairs a token serve all its heads), beside the
// places of the entries; then groups of LP lanes take rows (query heads, key
// heads, values of a token), a lane eight elements. The two elements of a pair are
// the same register of two lanes where the halves are a multiple of eight (one
// shuffle each), or neighbours in one lane (interleaved). Other sizes and
// alignments take the scalar form: a warp a row, the row in shared memory.
// Bound by HBM: each element is read and written once.
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
__global__ void __launch_bounds__(kvr::NT) kv_rotate_kernel(const __grid_constant__ KvRotateArgs a, const __grid_constant__ KvArgs c) {
    using namespace kvr;
    __shared__ __align__(16) float s_cos[MAX_PAIRS], s_sin[MAX_PAIRS];
    __shared__ Place s_place[APPEND ? MAX_TOKENS : 1];
    __shared__ int s_cu[APPEND ? SEQS : 1];
    __shared__ float s_row[LP == 0 ? WARPS : 1][LP == 0 ? KV_MAX_D : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * a.per_block, tokens = min(a.per_block, a.tokens - t0), half = a.rot / 2;
    if constexpr (APPEND) {
        kv_grid_launch();
        if (!kv_offsets_ok<NT>(c, s_cu, SEQS)) return;
        if (tid < tokens) s_place[tid] = kv_place(c, c.B < SEQS ? s_cu : c.cu, t0 + tid);
        __syncthreads();
    }
    for (int i = tid; i < tokens * half; i += NT) {
        const int t = i / half, x = i - t * half;
        int ax = a.axis ? a.axis[x] : 0;
        if ((uint32_t)ax >= (uint32_t)a.axes) ax = 0;
        int pos;
        if constexpr (APPEND) pos = a.positions ? a.positions[(int64_t)ax * a.tokens + t0 + t] : s_place[t].first;
        else pos = a.positions[(int64_t)ax * a.tokens + t0 + t];
        const float2 cs = kv_cos_sin(a.turns[x], pos);
        s_cos[i] = cs.x, s_sin[i] = cs.y;
    }
    __syncthreads();
    // rows of a token: queries, keys, values
    const int nq = a.q.in ? a.Hq : 0, nk = a.k.in ? a.Hkv : 0, per = nq + nk + (a.v.in ? a.Hkv : 0), rows = tokens * per;
    // row r: its token, kind and addresses (out NULL: nothing is written)
    struct Row {
        const ST* in;
        ST* out;
        const float* norm;
        int t;
        bool turn, zero;
    };
    const auto row_of = [&](int r) {
        Row x;
        x.t = r / per;
        const int y = r - x.t * per, side = y < nq ? 0 : y < nq + nk ? 1 : 2, h = side == 0 ? y : side == 1 ? y - nq : y - nq - nk;
        const KvTurn& s = side == 0 ? a.q : side == 1 ? a.k : a.v;
        const int tok = t0 + x.t;
        const int64_t b = APPEND ? 0 : tok / a.T, j = APPEND ? tok : tok - b * a.T;
        x.in = static_cast<const ST*>(s.in) + b * s.in_seq + j * s.in_node + (int64_t)h * s.in_head;
        x.norm = s.norm ? s.norm + (int64_t)h * s.norm_head : nullptr;
        x.turn = side < 2 && (s.norm || half > 0), x.zero = false;  // (else it is moved as it is)
        x.out = static_cast<ST*>(s.out) + b * s.out_seq + j * s.out_node + (int64_t)h * s.out_head;
        if constexpr (APPEND) {
            const Place& p = s_place[x.t];
            if (side > 0)
                x.out = p.live != 1 ? nullptr
                                    : static_cast<ST*>(s.out) + (side == 1 ? p.k : p.v) + (int64_t)h * s.out_head;
            else if (p.live < 0)
                x.out = nullptr;
            x.zero = p.live == 0;
        }
        return x;
    };
    if constexpr (LP > 0) {
        constexpr int GROUPS = NT / LP, AHEAD = 2;
        const int sub = tid % LP, e0 = sub * LANE;
        const bool in = e0 < a.d, first = e0 < half, turned = e0 < a.rot;
        const int partner = first ? sub + half / LANE : turned ? sub - half / LANE : sub;
        for (int r0 = tid / LP; r0 - tid / LP < rows; r0 += GROUPS * AHEAD) {  // (the same trips for every lane)
            Row row[AHEAD];
            Eight<ST> raw[AHEAD];
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                row[y] = row_of(min(r0 + y * GROUPS, rows - 1));
                if (r0 + y * GROUPS >= rows) row[y].out = nullptr;
                raw[y].clear();
                if (in && row[y].out && !row[y].zero) raw[y].load(row[y].in + e0);
            }
#pragma unroll
            for (int y = 0; y < AHEAD; ++y) {
                const Row& w = row[y];
                float x[LANE];
                raw[y].unpack(x);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < LANE; ++e) ss = fmaf(x[e], x[e], ss);
                ss = group_sum<LP>(ss);
                if (w.norm && in) {
                    const float f = rsqrtf(ss / (float)a.d + a.eps);
#pragma unroll
                    for (int e = 0; e < LANE; e += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(w.norm + e0 + e);
                        x[e] *= f * (g.x + a.offset), x[e + 1] *= f * (g.y + a.offset);
                        x[e + 2] *= f * (g.z + a.offset), x[e + 3] *= f * (g.w + a.offset);
                    }
                }
                if (a.interleaved) {
                    if (turned && w.turn) {
                        const int i = w.t * half + e0 / 2;
                        const float4 co = *reinterpret_cast<const float4*>(s_cos + i), si = *reinterpret_cast<const float4*>(s_sin + i);
                        const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                        for (int e = 0; e < LANE; e += 2) {
                            const float p = x[e], q = x[e + 1];
                            x[e] = p * c4[e / 2] - q * s4[e / 2], x[e + 1] = p * s4[e / 2] + q * c4[e / 2];
                        }
                    }
                } else {
                    const int i = w.t * half + e0 - (first || !turned ? 0 : half);
#pragma unroll
                    for (int e = 0; e < LANE; e += 4) {
                        float o[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) o[z] = __shfl_sync(FULL_MASK, x[e + z], partner, LP);
                        if (turned && w.turn) {
                            const float4 co = *reinterpret_cast<const float4*>(s_cos + i + e);
                            const float4 si = *reinterpret_cast<const float4*>(s_sin + i + e);
                            const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                x[e + z] = x[e + z] * c4[z] + (first ? -o[z] : o[z]) * s4[z];
                        }
                    }
                }
                if (w.turn) raw[y].pack(x);
                if (in && w.out) raw[y].store(w.out + e0);
            }
        }
    } else {
        float* line = s_row[warp];
        for (int r = warp; r < rows; r += WARPS) {
            const Row w = row_of(r);
            if (!w.out) continue;
            float ss = 0.f;
            for (int e = lane; e < a.d; e += 32) {
                const float x = w.zero ? 0.f : load_elem(w.in, e, Store<ST>::code);
                line[e] = x, ss = fmaf(x, x, ss);
            }
            ss = group_sum<32>(ss);
            __syncwarp();
            if (!w.turn && !w.zero) {
                for (int e = lane; e < a.d; e += 32) w.out[e] = w.in[e];
                __syncwarp();
                continue;
            }
            if (w.norm) {
                const float f = rsqrtf(ss / (float)a.d + a.eps);
                for (int e = lane; e < a.d; e += 32) line[e] *= f * (w.norm[e] + a.offset);
                __syncwarp();
            }
            for (int e = lane; e < a.d; e += 32) {
                float z = line[e];
                if (e < a.rot && !w.zero) {
                    const bool one = a.interleaved ? (e & 1) == 0 : e < half;
                    const int i = a.interleaved ? e >> 1 : one ? e : e - half;
                    const float other = line[a.interleaved ? e ^ 1 : one ? e + half : e - half];
                    const float co = s_cos[w.t * half + i], si = s_sin[w.t * half + i];
                    z = one ? z * co - other * si : other * si + z * co;
                }
                store_elem(w.out, e, Store<ST>::code, w.zero ? 0.f : z);
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
