// kv_tc.cuh -- attention of drafted nodes over the paged cache on the tcgen05
// tensor cores (16-bit caches whose pages hold a multiple of 8 entries and
// whose rows the TMA engine can address).
//
// Mathematics. The transposed form of one-pass attention: for a tile of 128
// keys and NR query rows, S^T = K Q^T (128 x NR), P^T = 2^{c S^T - m} with a
// reference m per row, O^T += V^T P^T (d x NR). The rows of a unit are the
// MMAs' N, so a decode step's handful of rows costs 16 columns, not a padded
// block of 128, and a thread owns one key: its softmax work is NR elements
// whatever the number of rows, and its share of the row sums stays in
// registers until the unit ends.
//
// The reference. m is not the running maximum but one that lags: as long as
// no score of a tile exceeds m by more than REF_SLACK (in powers of two), the
// tile's weights are formed against the old m, which is exact (numerator and
// denominator carry the same factor) and stays far inside the range of fp16
// (2^8). So the cross-thread maximum, and the rescaling of the accumulator in
// tensor memory, happen on a unit's first tile and where the maximum really
// moves; otherwise a tile costs one barrier, which carries the vote.
//
// Kernel shape: persistent, one CTA per SM:
//   softmax    NG groups of four warps (two up to 32 rows, four above: 16 or 32
//              rows a thread keep scores and sums in registers); group g owns
//              NR / NG query rows (columns of S^T and O^T), thread key
//              (warp % 4) * 32 + lane = its tensor-memory lane;
//   loads      one warp: K and V tiles by TMA into a ring of stages of 128 keys
//              x 128 elements (64 where d <= 64), 128-byte swizzle, boxes of as
//              many keys as a page and the tile share; page indices two tiles
//              ahead;
//   MMAs       one thread issues them: S^T of tile i + 1 before O^T of tile i,
//              so that the tensor cores work while tile i's weights form.
// K is the A operand as it lies (K-major); V is the A operand of the second
// product transposed (MN-major); P^T is written by its threads, 16 bytes for
// eight rows, in the unswizzled MN-major layout, which a warp fills without
// bank conflicts. The drafted nodes are the unit's last tile.
#pragma once

#include <cuda.h>

#include "gdn_tcgen05.cuh"
#include "kv_common.cuh"

namespace gdn {

namespace kvt {

constexpr int KT = 128;       // keys a tile
// groups of softmax warps, and all warps, for a block of NR rows
__host__ __device__ constexpr int groups(int NR) { return NR > 32 ? 4 : 2; }
__host__ __device__ constexpr int threads(int NR) { return (4 * groups(NR) + 2) * 32; }
constexpr int LEAST = 1;      // tiles a CTA at least
constexpr int BOX = 64;       // elements of d in one TMA box (128 bytes)
constexpr int BOX_BYTES = KT * BOX * 2;
constexpr float REF_NONE = -3.0e38f;  // reference of a row without a key yet
constexpr float REF_SLACK = 8.f;
constexpr int MAX_STAGES = 14;

struct Maps {
    CUtensorMap k, v, kn, vn;
};

// Small shared-memory state of a CTA.
template <int NR>
struct __align__(16) State {
    float nref[NR];           // reference of each row, negated: -m
    float factor[NR];         // rescaling factor of a moved reference; at the end 1 / l
    float warp_max[4][NR];    // maxima by warp quadrant; at the end sums
    uint32_t mask[2][NR];     // mask words of each row
    int64_t row[NR];          // row of out and lse, -1 where the unit has none
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], q_full, v_ok, drain;
    int64_t q_at[NR];         // element offset of each row's query
    KvScan<threads(NR)> scan;
    int gave_up[4], v_stage;
    uint32_t tmem;
};

template <int NR>
__host__ __device__ constexpr int p_bytes() {
    return KT * NR * 2;
}
// Bytes ahead of the ring: queries, two weight buffers, state; the ring follows at a multiple of 1024.
template <int NR>
__host__ __device__ constexpr int fixed_bytes(int boxes) {
    return boxes * NR * 128 + 2 * p_bytes<NR>();
}
template <int NR>
__host__ __device__ constexpr int smem_bytes(int boxes, int stages) {
    return 1024 + fixed_bytes<NR>(boxes) + stages * (boxes > 1 ? 2 : 1) * BOX_BYTES + (int)sizeof(State<NR>);
}

// Operand descriptors. K-major, 128-byte swizzle: rows of 128 bytes, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)swizzle << 61;
}
constexpr uint32_t SW128 = 2, SW_NONE = 0;

// Instruction descriptor, kind::f16: FP32 accumulator; A and B both bf16 (1) or both f16 (0); M = 128.
__device__ __forceinline__ uint32_t idesc(uint32_t type, bool a_mn, bool b_mn, int N) {
    return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(KT >> 4) << 24);
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Barrier of one softmax group (128 threads), and the same with a vote.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ bool group_any(int g, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + g)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <typename ST>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
    static constexpr uint32_t type = 1, exp_mask = 0x7f80u;
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    __device__ static __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Half16<__half> {
    static constexpr uint32_t type = 0, exp_mask = 0x7c00u;
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
    __device__ static __forceinline__ __half round(float x) { return __float2half_rn(x); }
};

// Row sums of 32 (or N < 32) rows over a warp's threads: lane r holds row r's.
template <int N>
__device__ __forceinline__ float sum_rows(float* l, int lane) {
    constexpr int M = N < 32 ? N : 32;
    float x[M];
#pragma unroll
    for (int r = 0; r < M; ++r) x[r] = l[r];
    float y = reduce_scatter<M>(x, lane & (M - 1));
#pragma unroll
    for (int o = M; o < 32; o <<= 1) y += __shfl_xor_sync(FULL_MASK, y, o);
    return y;
}

// Eight 16-bit values with those that are not finite replaced by zero.
template <typename ST>
__device__ __forceinline__ uint4 clear_odd(uint4 x) {
    constexpr uint32_t e = Half16<ST>::exp_mask;
    uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((u[i] & e) == e) u[i] &= 0xffff0000u;
        if ((u[i] >> 16 & e) == e) u[i] &= 0x0000ffffu;
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Whether this thread's share of the nodes' values (all 128 threads of a group ask) is not all finite.
template <typename ST>
__device__ __forceinline__ bool odd_values(const KvArgs& a, int nodes, int b, int h, int gt) {
    constexpr uint32_t m = Half16<ST>::exp_mask;
    const ST* v = static_cast<const ST*>(a.vn.p) + (int64_t)b * a.vn.seq + (int64_t)h * a.vn.head;
    bool odd = false;
    const int per = (a.d + 63) / 64 * 8, n = nodes * per;
#pragma unroll 4
    for (int i = gt; i < n; i += 128) {
        const int j = i / per, e = (i - j * per) * 8;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (e < a.d) x = *reinterpret_cast<const uint4*>(v + (int64_t)j * a.vn.node + e);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) odd = odd || (u[y] & m) == m || (u[y] >> 16 & m) == m;
    }
    return odd;
}

// The values that clear_odd took out, added to the rows' outputs where the row attends the node.
template <typename ST, int N>
__device__ __noinline__ void add_odd(const KvArgs& a, int nodes, int b, int h, int e, const uint32_t* lo, const uint32_t* hi,
                                     float* o) {
    for (int j = 0; j < nodes; ++j) {
        const float v = load_elem(a.vn.p, (int64_t)b * a.vn.seq + (int64_t)j * a.vn.node + (int64_t)h * a.vn.head + e,
                                  Store<ST>::code);
        if (isfinite(v)) continue;
        for (int x = 0; x < N; ++x)
            if ((j < 32 ? lo[x] >> j : hi[x] >> (j - 32)) & 1) o[x] += v;
    }
}

// x * c + y on two values at a time
__device__ __forceinline__ float2 fma2(float2 x, float2 c, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(c.x), "f"(c.y), "f"(y.x), "f"(y.y));
    return r;
}

}  // namespace kvt

// boxes: 64-element boxes of d; stages: of the ring; box_rows: keys of one TMA box.
template <typename ST, int NR>
__global__ void __launch_bounds__(kvt::threads(NR), 1)
    kv_attn_tc_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ kvt::Maps maps, const int boxes,
                      const int stages, const int box_rows) {
    using namespace kvt;
    using H = Half16<ST>;
    constexpr int NG = groups(NR), NRH = NR / NG, NT = threads(NR), SM_WARPS = 4 * NG;
    constexpr int LOAD_WARP = SM_WARPS, MMA_WARP = SM_WARPS + 1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int pairs = (boxes + 1) >> 1;  // 128-element halves of d
    const int stage_bytes = (boxes > 1 ? 2 : 1) * BOX_BYTES;
    unsigned char* sQ = smem;
    unsigned char* sP = sQ + boxes * NR * 128;
    unsigned char* ring = smem + fixed_bytes<NR>(boxes);
    State<NR>& st = *reinterpret_cast<State<NR>*>(ring + stages * stage_bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr uint32_t TM_S = 0, TM_O = 2 * NR;  // tensor memory: two buffers of S^T, then O^T by halves of d
    constexpr uint32_t TM_COLS = NR * 4;

    kv_grid_launch();
    if (warp == LOAD_WARP) {
        if (lane < 4) {
            const CUtensorMap* m = lane == 0 ? &maps.k : lane == 1 ? &maps.v : lane == 2 ? &maps.kn : &maps.vn;
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
        }
        if (lane < stages) mbar_init(&st.full[lane], 1), mbar_init(&st.empty[lane], 1);
        if (lane < 2) {
            mbar_init(&st.s_full[lane], 1), mbar_init(&st.s_empty[lane], SM_WARPS);
            mbar_init(&st.p_full[lane], SM_WARPS), mbar_init(&st.p_empty[lane], 1);
        }
        if (lane == 2) mbar_init(&st.q_full, SM_WARPS), mbar_init(&st.v_ok, 1), mbar_init(&st.drain, 1);
        if (lane < 4) st.gave_up[lane] = 0;
        fence_barrier_init();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&st.tmem)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before();
    const KvSplit split = kv_locate<true, KT, NT>(a, st.scan, gridDim.x, LEAST);
    tc::fence_after();
    const uint32_t tmem = st.tmem;
    const bool busy = split.busy(blockIdx.x);

    if (warp == LOAD_WARP && busy) {
        // ------------------------------------------------------------ loads
        KvWalk<true, KT> w(a, split, st.scan);
        uint32_t n_block = 0;
        int stage = 0, round = 0;
        bool ok = true;
        const int per_tile = KT / box_rows;
        do {
            const int n = w.t1 - w.t0;
            const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
            // page of this lane's box in tile t
            const auto page_of = [&](int t) {
                const int e = t * KT + lane * box_rows;
                return lane < per_tile && e < w.s.len && t < w.t1 ? table[e / a.page_size] : 0;
            };
            int p_prev = 0, p_cur = page_of(w.t0), p_next = page_of(w.t0 + 1);
            const auto load = [&](int t, int page, const CUtensorMap* map, const CUtensorMap* map_new) {
                const bool tree = t == w.nt - 1;
                const int live = tree ? 0 : min(KT, w.s.len - t * KT);
                const int used = (live + box_rows - 1) / box_rows;  // boxes with an entry
                const int e = t * KT + lane * box_rows, place = e % a.page_size;
                for (int p = 0; p < pairs && ok; ++p) {
                    ok = __all_sync(FULL_MASK, mbar_wait(&st.empty[stage], (round & 1) ^ 1));
                    if (!ok) break;
                    const int nb = min(2, boxes - 2 * p);
                    unsigned char* dst = ring + stage * stage_bytes;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&st.full[stage], (tree ? a.T : used * box_rows) * 128 * nb);
                    __syncwarp();
                    if (tree) {
                        if (lane < nb)
                            tma_load(dst + lane * BOX_BYTES, map_new, (2 * p + lane) * BOX, 0, w.h, w.b, &st.full[stage]);
                    } else if (lane < used) {
                        for (int x = 0; x < nb; ++x)
                            tma_load(dst + x * BOX_BYTES + lane * box_rows * 128, map, (2 * p + x) * BOX, place, w.h, page,
                                     &st.full[stage]);
                    }
                    ++n_block;
                    if (++stage == stages) stage = 0, ++round;
                }
            };
            load(w.t0, p_cur, &maps.k, &maps.kn);
            for (int i = 0; i < n && ok; ++i) {
                const int t = w.t0 + i;
                const int p_far = page_of(t + 2);
                p_prev = p_cur, p_cur = p_next, p_next = p_far;
                if (i + 1 < n) load(t + 1, p_cur, &maps.k, &maps.kn);
                load(t, p_prev, &maps.v, &maps.vn);
            }
        } while (ok && w.next());
        if (!ok) {
            if (lane == 0) set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
            // the copies in flight land before the CTA ends
            const int last = n_block < (uint32_t)stages ? (int)n_block : stages;
            for (int i = 0; i < last; ++i) {
                const uint32_t blk = n_block - 1 - i;
                mbar_wait(&st.full[blk % stages], (blk / stages) & 1);
            }
        }
    } else if (warp == MMA_WARP && busy) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0) {
            KvWalk<true, KT> w(a, split, st.scan);
            const uint32_t id_s = idesc(H::type, false, false, NR), id_o = idesc(H::type, true, true, NR);
            const uint32_t aQ = smem_addr(sQ), aP = smem_addr(sP), aR = smem_addr(ring);
            int stage = 0, round = 0;
            uint32_t n_s = 0, n_o = 0, seg = 0;  // tiles of S^T and O^T so far, segments
            bool ok = true;
            const int ksteps = (min(a.d, BOX) + 15) / 16;  // of one box (a box past the first is read whole)
            const auto step = [&]() {
                if (++stage == stages) stage = 0, ++round;
            };
            const auto scores = [&]() {  // S^T of the next tile
                const int buf = n_s & 1;
                if (n_s >= 2) ok = ok && mbar_wait(&st.s_empty[buf], ((n_s >> 1) - 1) & 1);
                for (int p = 0; p < pairs && ok; ++p) {
                    ok = mbar_wait(&st.full[stage], round & 1);
                    if (!ok) break;
                    tc::fence_after();
                    const int nb = min(2, boxes - 2 * p);
                    for (int x = 0; x < nb; ++x)
                        for (int k = 0; k < ksteps; ++k)
                            mma(tmem + TM_S + buf * NR, desc(aR + stage * stage_bytes + x * BOX_BYTES + k * 32, 16, 1024, SW128),
                                desc(aQ + (2 * p + x) * NR * 128 + k * 32, 16, 1024, SW128), id_s, p + x + k > 0);
                    tc::commit(&st.empty[stage]);
                    step();
                }
                if (ok) tc::commit(&st.s_full[buf]);
                ++n_s;
            };
            do {
                const int n = w.t1 - w.t0;
                ok = ok && mbar_wait(&st.q_full, seg & 1);
                if (!ok) break;
                ++seg;
                tc::fence_after();
                scores();
                for (int i = 0; i < n && ok; ++i) {
                    if (i + 1 < n) scores();
                    const int buf = n_o & 1, t = w.t0 + i;
                    const bool tree = t == w.nt - 1, part = tree || w.s.len - t * KT < KT;
                    if (part) {  // the softmax threads clear the rows of V past the last key
                        int s2 = stage, r2 = round;
                        for (int p = 0; p < pairs && ok; ++p) {
                            ok = mbar_wait(&st.full[s2], r2 & 1);
                            if (++s2 == stages) s2 = 0, ++r2;
                        }
                        st.v_stage = stage;
                        if (ok) mbar_arrive(&st.v_ok);
                    }
                    ok = ok && mbar_wait(&st.p_full[buf], (n_o >> 1) & 1);
                    if (!ok) break;
                    tc::fence_after();
                    for (int p = 0; p < pairs && ok; ++p) {
                        ok = mbar_wait(&st.full[stage], round & 1);
                        if (!ok) break;
                        tc::fence_after();
                        // A: 128 elements of d (the second 64 in the stage's second box; where there is
                        // none, the first again: its lanes are not read)
                        const uint32_t lbo = boxes - 2 * p > 1 ? BOX_BYTES : 0;
                        for (int k = 0; k < KT / 16; ++k)
                            mma(tmem + TM_O + p * NR, desc(aR + stage * stage_bytes + k * 2048, lbo, 1024, SW128),
                                desc(aP + buf * p_bytes<NR>() + k * 256, 128, KT * 16, SW_NONE), id_o, i + k > 0);
                        tc::commit(&st.empty[stage]);
                        step();
                    }
                    if (ok) tc::commit(&st.p_empty[buf]);
                    ++n_o;
                }
            } while (ok && w.next());
            if (!ok) {
                set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
                tc::commit(&st.drain);  // MMAs in flight end before tensor memory is freed
                mbar_wait(&st.drain, 0);
            }
        }
        __syncwarp();
    } else if (warp < SM_WARPS && busy) {
        // ------------------------------------------------------------ softmax
        const int g = warp >> 2, quad = warp & 3, key = quad * 32 + lane, gt = tid & 127, g0 = g * NRH;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const float c2 = a.scale * LOG2E;
        const int64_t part_floats = kv_part_floats(NR, a.d);
        KvWalk<true, KT> w(a, split, st.scan);
        uint32_t n_t = 0, n_v = 0;  // tiles so far, v_ok rounds so far
        int checked = -1;
        bool pages_bad = false, failed = false, stop = false;  // stop: the whole group gives up
        float l[NRH];
        do {
            const int rows = min(NR, w.s.nodes * a.G - w.rb * NR), r_first = w.rb * NR, n = w.t1 - w.t0;
            // ---- row tables and queries of the group's rows
            if (gt < NRH) {
                const int r = g0 + gt, node = (r_first + r) / a.G, x = w.h * a.G + (r_first + r) - node * a.G;
                const bool in = r < rows;
                st.nref[r] = -REF_NONE;
                st.row[r] = in ? ((int64_t)w.b * a.T + node) * a.Hq + x : -1;
                st.q_at[r] = (int64_t)w.b * a.q.seq + (int64_t)node * a.q.node + (int64_t)x * a.q.head;
                const uint64_t m = in ? a.mask[(int64_t)w.b * a.T + node] : 0;
                st.mask[0][r] = (uint32_t)m, st.mask[1][r] = (uint32_t)(m >> 32);
            }
            group_sync(g);
            {
                // 16-byte pieces, eight of a row's box; a thread's loads all go out before the first is stored
                constexpr int N = (NRH * 8 + 127) / 128;
                for (int x = 0; x < boxes; ++x) {
                    uint4 v[N];
#pragma unroll
                    for (int y = 0; y < N; ++y) {
                        const int i = gt + y * 128, r = g0 + (i >> 3), e = x * BOX + (i & 7) * 8;
                        v[y] = make_uint4(0, 0, 0, 0);
                        if (i < NRH * 8 && r < rows && e < a.d)
                            v[y] = *reinterpret_cast<const uint4*>(static_cast<const ST*>(a.q.p) + st.q_at[r] + e);
                    }
#pragma unroll
                    for (int y = 0; y < N; ++y) {
                        const int i = gt + y * 128, r = g0 + (i >> 3);
                        if (i < NRH * 8)
                            *reinterpret_cast<uint4*>(sQ + x * NR * 128 + r * 128 + (((i & 7) ^ (r & 7)) << 4)) = v[y];
                    }
                }
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&st.q_full);
            if (checked != w.b) {
                pages_bad = group_any(g, !kv_pages_ok(a, w.s, gt, 128));
                if (pages_bad && tid == 0) set_error(a.dev_err, KV_DEVERR_PAGE);
                checked = w.b;
            }
            bool odd = false;  // a node's value is not finite
#pragma unroll
            for (int r = 0; r < NRH; ++r) l[r] = 0.f;

            for (int i = 0; i < n; ++i, ++n_t) {
                const int t = w.t0 + i, buf = n_t & 1;
                const bool tree = t == w.nt - 1;
                const int live = tree ? w.s.nodes : min(KT, w.s.len - t * KT);
                if (tree) odd = group_any(g, odd_values<ST>(a, w.s.nodes, w.b, w.h, gt));
                float s[NRH];
                failed = failed || !mbar_wait(&st.s_full[buf], (n_t >> 1) & 1);
                tc::fence_after();
                tc::tmem_ld<NRH>(tmem + lane_base + TM_S + buf * NR + g0, s);
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&st.s_empty[buf]);
                float c = c2;
                if (live < KT) {  // the scaled scores, -inf where the row does not see the key
                    c = 1.f;
#pragma unroll
                    for (int r = 0; r < NRH; ++r) {
                        const bool seen = key < live && (!tree || (st.mask[quad & 1][g0 + r] >> lane & 1));
                        s[r] = seen ? s[r] * c2 : -INFINITY;
                    }
                }
                const float2 cc = make_float2(c, c);
                float over = -INFINITY;  // the largest exponent against the references
#pragma unroll
                for (int r = 0; r < NRH; r += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(&st.nref[g0 + r]);
                    const float2 x = fma2(make_float2(s[r], s[r + 1]), cc, make_float2(m.x, m.y));
                    const float2 y = fma2(make_float2(s[r + 2], s[r + 3]), cc, make_float2(m.z, m.w));
                    over = fmaxf(over, fmaxf(fmaxf(x.x, x.y), fmaxf(y.x, y.y)));
                }
                if (failed) st.gave_up[g] = 1;
                if (group_any(g, failed || over > REF_SLACK)) {
                    if (st.gave_up[g]) {
                        stop = true;
                        break;
                    }
                    // the tile's maxima, new references
#pragma unroll
                    for (int r = 0; r < NRH; ++r) {
                        const float x = warp_max(s[r] * c);
                        if (lane == (r & 31)) st.warp_max[quad][g0 + r] = x;
                    }
                    group_sync(g);
                    if (gt < NRH) {
                        const int r = g0 + gt;
                        const float old = -st.nref[r];
                        const float m = fmaxf(fmaxf(fmaxf(st.warp_max[0][r], st.warp_max[1][r]),
                                                    fmaxf(st.warp_max[2][r], st.warp_max[3][r])), old);
                        st.factor[r] = kv_ex2(old - m), st.nref[r] = -m;
                    }
                    group_sync(g);
                    if (i > 0) {  // the sums and the accumulator, once the last tile's product is in it
#pragma unroll
                        for (int r = 0; r < NRH; r += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(&st.factor[g0 + r]);
                            l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
                        }
                        const uint32_t p = n_t - 1;
                        failed = failed || !mbar_wait(&st.p_empty[p & 1], (p >> 1) & 1);
                        tc::fence_after();
                        for (int hf = 0; hf < pairs; ++hf)
#pragma unroll
                            for (int r = 0; r < NRH; r += 8) {
                                float o[8];
                                const uint32_t at = tmem + lane_base + TM_O + hf * NR + g0 + r;
                                tc::tmem_ld<8>(at, o);
                                const float4 f0 = *reinterpret_cast<const float4*>(&st.factor[g0 + r]);
                                const float4 f1 = *reinterpret_cast<const float4*>(&st.factor[g0 + r + 4]);
                                o[0] *= f0.x, o[1] *= f0.y, o[2] *= f0.z, o[3] *= f0.w;
                                o[4] *= f1.x, o[5] *= f1.y, o[6] *= f1.z, o[7] *= f1.w;
                                tc::tmem_st<8>(at, o);
                            }
                        tc::fence_before();
                    }
                }
                // weights: FP32 sums, rounded once to the cache's type for the product with the values
                if (n_t >= 2) failed = failed || !mbar_wait(&st.p_empty[buf], ((n_t >> 1) - 1) & 1);
                unsigned char* dst = sP + buf * p_bytes<NR>() + g * (NRH / 8) * (KT * 16) + key * 16;
#pragma unroll
                for (int r = 0; r < NRH; r += 8) {
                    uint32_t u[4];
#pragma unroll
                    for (int x = 0; x < 8; x += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(&st.nref[g0 + r + x]);
                        const float2 y = fma2(make_float2(s[r + x], s[r + x + 1]), cc, make_float2(m.x, m.y));
                        const float2 z = fma2(make_float2(s[r + x + 2], s[r + x + 3]), cc, make_float2(m.z, m.w));
                        const float p0 = kv_ex2(y.x), p1 = kv_ex2(y.y), p2 = kv_ex2(z.x), p3 = kv_ex2(z.y);
                        l[r + x] += p0, l[r + x + 1] += p1, l[r + x + 2] += p2, l[r + x + 3] += p3;
                        u[x / 2] = H::pack(p0, p1), u[x / 2 + 1] = H::pack(p2, p3);
                    }
                    *reinterpret_cast<uint4*>(dst + (r / 8) * (KT * 16)) = make_uint4(u[0], u[1], u[2], u[3]);
                }
                if (live < KT) {
                    // Rows of V past the last key become zero (0 x NaN would reach the sums), and so do a
                    // node's values that are not finite: the epilogue adds them to the rows that attend it.
                    failed = failed || !mbar_wait(&st.v_ok, n_v & 1);
                    ++n_v;
                    for (int x = g; x < boxes; x += NG) {
                        int stage = st.v_stage + (x >> 1);
                        if (stage >= stages) stage -= stages;
                        uint4* row = reinterpret_cast<uint4*>(ring + stage * stage_bytes + (x & 1) * BOX_BYTES + key * 128);
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            if (key >= live) row[y ^ (lane & 7)] = make_uint4(0, 0, 0, 0);  // (order against bank conflicts)
                            else if (tree && odd) row[y] = clear_odd<ST>(row[y]);
                        }
                    }
                }
                tc::fence_async_smem();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&st.p_full[buf]);
            }
            if (stop) break;
            // ---- row sums over the group's threads, then the outputs
            const float own = sum_rows<NRH>(l, lane);
            if (lane < NRH) st.warp_max[quad][g0 + lane] = own;
            group_sync(g);
            const bool whole = w.whole();
            float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later) * part_floats;
            if (gt < NRH) {
                const int r = g0 + gt;
                const float sum = pages_bad ? 0.f : st.warp_max[0][r] + st.warp_max[1][r] + st.warp_max[2][r] + st.warp_max[3][r];
                st.factor[r] = pages_bad ? 0.f : whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                if (st.row[r] >= 0) {
                    if (!whole)
                        part[NR * a.d + r] = -st.nref[r], part[NR * a.d + NR + r] = sum;
                    else if (a.lse)
                        a.lse[st.row[r]] = sum == 0.f ? -INFINITY : (log2f(sum) - st.nref[r]) * LN2;
                }
            }
            group_sync(g);
            failed = failed || !mbar_wait(&st.p_empty[(n_t - 1) & 1], ((n_t - 1) >> 1) & 1);
            tc::fence_after();
            for (int hf = 0; hf < pairs; ++hf) {
                const int e = hf * 128 + key;
                float o[NRH];
                __syncwarp();
                tc::tmem_ld<NRH>(tmem + lane_base + TM_O + hf * NR + g0, o);
                if (e < a.d) {
                    if (odd) add_odd<ST, NRH>(a, w.s.nodes, w.b, w.h, e, &st.mask[0][g0], &st.mask[1][g0], o);
                    if (whole) {
                        ST* out = static_cast<ST*>(a.out) + e;
#pragma unroll
                        for (int r = 0; r < NRH; ++r) {
                            const int64_t row = st.row[g0 + r];
                            const float f = st.factor[g0 + r];
                            if (row >= 0) out[row * a.d] = H::round(f == 0.f ? 0.f : o[r] * f);
                        }
                    } else {
                        float* x = part + (int64_t)g0 * a.d + e;
#pragma unroll
                        for (int r = 0; r < NRH; ++r)
                            if (g0 + r < rows) x[r * a.d] = st.factor[g0 + r] == 0.f ? 0.f : o[r];
                    }
                }
            }
            tc::fence_before();
            if (tid == 0 && w.last()) static_cast<KvBorder*>(a.border)[blockIdx.x] = kv_border(a, split, w);
            group_sync(g);  // the row tables are read
        } while (w.next());
        if (failed && lane == 0) set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
    }
    if (!busy && tid == 0) static_cast<KvBorder*>(a.border)[blockIdx.x].rows = 0;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    kv_empty_rows<NT>(a);
    if (warp == MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
}

}  // namespace gdn
