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
// The sum over tiles. The tensor cores keep O^T in FP32 but cut each product
// off at about 2^-25 of what the accumulator holds, always towards zero: over
// 131072 entries the outputs came out 0.12% (equal weights) to 0.39% (one leader)
// too small, and in proportion over more. So O^T is a sum over FOLD tiles (2048
// entries, 2^-14 at most), and is then added to a second one in tensor memory,
// by the softmax threads, which round to nearest. (FOLD 16 and 32 take the same
// time: nothing where HBM bounds, 2% of the 64-node tree below.)
//
// The reference. m is not the running maximum but one that lags: as long as
// no score of a tile exceeds the maximum that m was formed from by more than
// REF_SLACK (in powers of two), the tile's weights are formed against the old
// m, which is exact (numerator and denominator carry the same factor). So the
// cross-thread maximum, and the rescaling of the accumulator in tensor memory,
// happen on a unit's first tile and where the maximum really moves; otherwise a
// tile costs one barrier, which carries the vote.
//
// Weights in fp16. Their range ends at 2^16 above and at steps of 2^-24 below.
// Weights against the maximum itself would use eight powers of two above 1 and
// lose, in the product with V but not in the sum, what lies under 2^-25: 131071
// entries of 2^-25.2 below a leader are 0.3% of its row. So m lies seven powers
// of two under the maximum (Half16::lift): the largest weight is 2^7 to 2^15,
// and what is rounded to nothing lies under 2^-32 of the maximum: 2^20 such
// entries together are under half an fp16 unit of rounding. bf16 has FP32's
// range and no lift.
//
// Kernel shape: persistent, one CTA per SM:
//   softmax    NG groups of four warps (two up to 32 rows, four above); group g
//              owns NR / NG query rows (columns of S^T and O^T), thread key
//              (warp % 4) * 32 + lane = its tensor-memory lane;
//   K, V       a warp each: tiles by TMA into a ring of stages of 128 keys x 128
//              elements (64 where d <= 64), 128-byte swizzle, boxes of as many
//              keys as a page and the tile share. A warp needs about 80 cycles a
//              box: with pages of 16 entries one warp for both took 4400 cycles
//              a tile, where HBM takes 2800. The K warp also writes the tables
//              of a segment's rows ahead of the softmax warps, and looks at the
//              pages that it loads;
//   S^T, O^T   a warp each, one elected thread of which issues the products from
//              uniform registers. The S^T warp loads a segment's queries beside
//              the last one's end and runs up to two tiles ahead, so that the
//              tensor cores work while weights form.
// Each ring has one producer and one consumer, both in tile order: a barrier's
// phase is never more than one ahead of its waiter. (In one ring for both, K
// could reach a stage two rounds ahead of V, and a parity wait passes then.)
// K is the A operand as it lies (K-major); V is the A operand of the second
// product transposed (MN-major); P^T is written by its threads, 16 bytes for
// eight rows, in the unswizzled MN-major layout, which a warp fills without
// bank conflicts. The drafted nodes are the unit's last tile.
//
// Bound and measurement (GB300, whole calls with the join). Up to 64 rows a key
// head: HBM. A decode step of 64 sequences of up to 8192 tokens (32 / 8 heads,
// d = 128, bf16, 1.32 GB) takes 205 us, 6.5 TB/s or 0.97 of the measured copy
// bandwidth; 16-node trees over 32 x 4096 tokens (0.33 GB) 72 us, 0.69, of which
// some 20 us are start, the units' ends and the join. Above 128 rows a key head
// each block of 128 is a unit that reads all keys: a 64-node tree over 131072
// tokens (256 rows, 0.54 GB, 137 GFLOP) takes 184 us, 745 TFLOP/s, and reads
// 1.08 GB from HBM (161 us of it; the softmax warps' chain, 2800 cycles a tile
// where HBM takes 2900 and the products 1200, is close behind). Short calls are
// latency: 10 us of steps (lengths, first tiles, maxima, outputs) and the join's
// 4.
// Measured and not taken: exponents before the vote instead of after it (the 64-
// node tree 208 -> 248 us); a look at the next tile beside this one's exponents
// with three buffers of S^T (179 -> 185, the 16-node trees 72 -> 76); two weight
// buffers at 128 rows, which leave K a ring of one stage (179 -> 211).
#pragma once

#include <cuda.h>

#include "gdn_tcgen05.cuh"
#include "kv_common.cuh"

namespace gdn {

namespace kvt {

constexpr int KT = 128;       // keys a tile
// groups of softmax warps, and all warps, for a block of NR rows
__host__ __device__ constexpr int groups(int NR) { return NR > 32 ? 4 : 2; }
__host__ __device__ constexpr int threads(int NR) { return (4 * groups(NR) + 4) * 32; }
constexpr int LEAST = 2;      // of the line a CTA at least
constexpr int BOX = 64;       // elements of d in one TMA box (128 bytes)
constexpr int BOX_BYTES = KT * BOX * 2;
constexpr float REF_NONE = -3.0e38f;  // reference of a row without a key yet
constexpr float REF_SLACK = 8.f;      // how far scores may rise above a reference's own maximum
constexpr float FUSED_MOST = 16777216.f;  // references up to which exponents are formed in one rounding
constexpr int FOLD = 16;  // tiles of one sum in tensor memory
constexpr int MAX_STAGES = 14;

struct Maps {
    CUtensorMap k, v, kn, vn, q;
};

// What a segment's rows are, written by the K warp ahead of the softmax warps.
template <int NR>
struct __align__(16) Table {
    uint32_t mask[2][NR];  // mask words of each row
    int64_t row[NR];       // row of out and lse
    int64_t q_at[NR];      // element offset of its query
    int odd;               // a node's value is not finite
    int bad;               // a page of the segment lies outside the pool
};

// Small shared-memory state of a CTA.
template <int NR>
struct __align__(16) State {
    float nref[NR];           // reference of each row, negated: -m (m: its maximum, less Half16::lift)
    float factor[NR];         // rescaling factor of a moved reference; at the end 1 / l
    float warp_max[4][NR];    // maxima by warp quadrant; at the end sums
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];  // the K ring's stages, then the V ring's
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], q_full, v_ok, drain[2];
    Table<NR> table[2];       // of this segment and the next
    uint64_t table_full[2], table_empty[2], seg_loaded[2];
    KvScan<threads(NR)> scan;
    KvSplit split;            // (for refuse_range alone: nothing of it stays in registers)
    int gave_up[4], big[4], v_stage;
    int stopped;  // a wait ran out
    uint32_t tmem;
#ifdef GDN_TEST_STALL
    uint64_t never;
#endif
};

template <int NR>
__host__ __device__ constexpr int p_bytes() {
    return KT * NR * 2;
}
// Bytes ahead of the rings: queries and weight buffers; the rings follow at a multiple of 1024, then the state.
template <int NR>
__host__ __device__ constexpr int fixed_bytes(int boxes, int p_bufs) {
    return boxes * NR * 128 + p_bufs * p_bytes<NR>();
}
template <int NR>
__host__ __device__ constexpr int smem_bytes(int boxes, int p_bufs, int stages) {
    return 1024 + fixed_bytes<NR>(boxes, p_bufs) + stages * (boxes > 1 ? 2 : 1) * BOX_BYTES + (int)sizeof(State<NR>);
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

// Issued by one thread of a converged warp (all of whose threads call it with the same operands, which
// so stay in uniform registers: a lone thread needed 110 cycles a product).
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
        : "memory");
}
// The barrier's arrival once the products issued so far by the same thread are done (as mma).
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
}
// A value that every thread of the warp holds, as one the compiler knows to be so.
template <typename T>
__device__ __forceinline__ T uniform(T x) {
    return __shfl_sync(FULL_MASK, x, 0);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(FULL_MASK, mbar_wait(bar, parity));
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Waits for a load warp's own copies: the last ones into the stages of its ring, of which `stage` would be
// the next to fill, for the time `round`.
__device__ __forceinline__ void landed(uint64_t* full, int first, int end, int stage, uint32_t round) {
#pragma unroll 1
    for (int s = first; s < end; ++s) {
        const uint32_t n = s < stage ? round + 1 : round;
        if (n > 0) mbar_wait(&full[s], (n - 1) & 1);
    }
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
    static constexpr float lift = 0.f;  // log2 of the weight of a score at the reference's maximum
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    __device__ static __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Half16<__half> {
    static constexpr uint32_t type = 0, exp_mask = 0x7c00u;
    static constexpr float lift = 7.f;
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
    __device__ static __forceinline__ __half round(float x) { return __float2half_rn(x); }
};

// Whether one of eight 16-bit values is not finite.
template <typename ST>
__device__ __forceinline__ bool has_odd(const uint4& x) {
    constexpr uint32_t e = Half16<ST>::exp_mask;
    bool odd = false;
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) odd = odd || (u[i] & e) == e || (u[i] >> 16 & e) == e;
    return odd;
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

// The values that clear_odd took out, added to the rows' outputs where the row attends the node.
template <typename ST>
__device__ __noinline__ void add_odd(const KvArgs& a, int nodes, int b, int h, int e, const uint32_t* lo, const uint32_t* hi,
                                     float* o) {
    for (int j = 0; j < nodes; ++j) {
        const float v = load_elem(a.vn.p, (int64_t)b * a.vn.seq + (int64_t)j * a.vn.node + (int64_t)h * a.vn.head + e,
                                  Store<ST>::code);
        if (isfinite(v)) continue;
        for (int x = 0; x < 8; ++x)
            if ((j < 32 ? lo[x] >> j : hi[x] >> (j - 32)) & 1) o[x] += v;
    }
}

// Two floats in one 64-bit register, for the packed instructions; the register is the variable, so that
// operands that serve many of them are put together once.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float x, float y) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 parts(Two x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ Two fma2(Two x, Two c, Two y) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(c), "l"(y));
    return r;
}
__device__ __forceinline__ Two add2(Two x, Two y) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ Two mul2(Two x, Two y) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

// Row sums of N (up to 32) rows over a warp's threads: lane r holds row r's.
template <int N>
__device__ __forceinline__ float sum_rows(const Two* l, int lane) {
    float x[N];
#pragma unroll
    for (int r = 0; r < N; r += 2) x[r] = parts(l[r / 2]).x, x[r + 1] = parts(l[r / 2]).y;
    float y = reduce_scatter<N>(x, lane & (N - 1));
#pragma unroll
    for (int o = N; o < 32; o <<= 1) y += __shfl_xor_sync(FULL_MASK, y, o);
    return y;
}

// The largest of three (a NaN among them is dropped).
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// What a CTA leaves whose waits ran out, by the whole block: the rows of its range as those of a refused
// sequence. Units that it shares with other CTAs get partials that say so, and the join a record as ever (the
// workspace is not initialised: what it held would be taken for one).
template <int NR>
__device__ __noinline__ void refuse_range(const KvArgs& a, const State<NR>& st) {
    const KvSplit split = st.split;
    bool some;
    KvWalk<true, KT> w(a, split, st.scan, some);
    if (!some) return;
    do {
        const int r0 = w.rb * NR, rows = min(NR, w.s.nodes * a.G - r0);
        if (w.whole()) {
            for (int i = threadIdx.x; i < rows * a.d; i += threads(NR)) {
                const int r = i / a.d, node = (r0 + r) / a.G, hq = w.h * a.G + (r0 + r) - node * a.G;
                const int64_t row = ((int64_t)w.b * a.T + node) * a.Hq + hq;
                store_elem(a.out, row * a.d + (i - r * a.d), a.dtype, 0.f);
                if (a.lse && i == r * a.d) a.lse[row] = -INFINITY;
            }
        } else {
            float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later) * kv_part_floats(NR, a.d) + NR * a.d;
            for (int r = threadIdx.x; r < rows; r += threads(NR)) part[r] = REF_NONE, part[NR + r] = -1.f;
        }
        if (threadIdx.x == 0 && w.last()) static_cast<KvBorder*>(a.border)[blockIdx.x] = kv_border(a, split, w);
    } while (w.next());
}

}  // namespace kvt

// boxes: 64-element boxes of d; k_stages, v_stages: of the rings; p_bufs: weight buffers (1 or 2: one where
// a second would cost a stage; the product of a tile is done long before the next one's weights);
// box_rows: keys of one TMA box.
template <typename ST, int NR>
__global__ void __launch_bounds__(kvt::threads(NR), 1)
    kv_attn_tc_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ kvt::Maps maps, const int boxes,
                      const int k_stages, const int v_stages, const int p_bufs, const int box_rows) {
    using namespace kvt;
    using H = Half16<ST>;
    constexpr int NG = groups(NR), NRH = NR / NG, NT = threads(NR), SM_WARPS = 4 * NG;
    constexpr int K_WARP = SM_WARPS, V_WARP = SM_WARPS + 1, S_WARP = SM_WARPS + 2, O_WARP = SM_WARPS + 3;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int pairs = (boxes + 1) >> 1;  // 128-element halves of d
    const int stage_bytes = (boxes > 1 ? 2 : 1) * BOX_BYTES;
    unsigned char* sQ = smem;
    unsigned char* sP = sQ + boxes * NR * 128;
    unsigned char* ring = smem + fixed_bytes<NR>(boxes, p_bufs);
    const int stages = k_stages + v_stages, pb = p_bufs - 1;  // tile n's weights: buffer n & pb, its use n >> pb
    State<NR>& st = *reinterpret_cast<State<NR>*>(ring + stages * stage_bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr uint32_t TM_S = 0, TM_O = 2 * NR;  // tensor memory: two buffers of S^T, then O^T by halves of d,
    const uint32_t TM_F = TM_O + pairs * NR;     // then the sum of its folds, alike
    const uint32_t TM_COLS = NR * (pairs > 1 ? 8 : 4);

    kv_grid_launch();
    if (warp == K_WARP) {
        if (lane < 5) {
            const CUtensorMap* m = lane == 0 ? &maps.k : lane == 1 ? &maps.v : lane == 2 ? &maps.kn : lane == 3 ? &maps.vn : &maps.q;
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
        }
        if (lane < stages) mbar_init(&st.full[lane], 1), mbar_init(&st.empty[lane], 1);
        if (lane < 2) {
            mbar_init(&st.s_full[lane], 1), mbar_init(&st.s_empty[lane], SM_WARPS);
            mbar_init(&st.p_full[lane], SM_WARPS), mbar_init(&st.p_empty[lane], 1);
            mbar_init(&st.table_full[lane], 1), mbar_init(&st.table_empty[lane], SM_WARPS), mbar_init(&st.seg_loaded[lane], 1);
        }
        if (lane == 2) mbar_init(&st.q_full, 1), mbar_init(&st.v_ok, 1), mbar_init(&st.drain[0], 1), mbar_init(&st.drain[1], 1);
        if (lane < 4) st.gave_up[lane] = 0, st.big[lane] = 0;
        if (lane == 0) st.stopped = 0;
#ifdef GDN_TEST_STALL
        if (lane == 0) mbar_init(&st.never, 1);
#endif
        fence_barrier_init();
    }
    if (warp == O_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&st.tmem)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before();
    const KvSplit split = kv_locate<true, KT, NT>(a, st.scan, gridDim.x, LEAST);
    tc::fence_after();
    const uint32_t tmem = st.tmem;
    bool busy;
    KvWalk<true, KT> w(a, split, st.scan, busy);
    if (tid == 0) st.split = split;

    if ((warp == K_WARP || warp == V_WARP) && busy) {
        // ------------------------------------------------------------ loads
        const bool keys = warp == K_WARP;
        const CUtensorMap *map = keys ? &maps.k : &maps.v, *map_new = keys ? &maps.kn : &maps.vn;
        const int first = keys ? 0 : k_stages, end = keys ? k_stages : stages;
        int stage = first;
        uint32_t round = 0;
        bool ok = true;
        const int per_tile = KT / box_rows, step_pages = KT / a.page_size, step_places = KT - step_pages * a.page_size;
        uint32_t seg = 0;
        do {
            const int n = w.t1 - w.t0, side = seg & 1;
            const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
            bool bad = false;
            // this lane's box of the next tile: its page (one tile ahead) and place
            const int e0 = w.t0 * KT + lane * box_rows;
            int pg = e0 / a.page_size, place = e0 - pg * a.page_size, e = e0;
            const auto look = [&]() { return lane < per_tile && e < w.s.len ? table[pg] : 0; };
            int page = look();
            const auto rows_table = [&]() {  // for the softmax warps and the queries' loads
                if (seg >= 2) ok = warp_wait(&st.table_empty[side], ((seg >> 1) - 1) & 1);
                Table<NR>& tb = st.table[side];
                const int r_first = w.rb * NR, rows = min(NR, w.s.nodes * a.G - r_first);
#pragma unroll 1
                for (int r = lane; r < NR; r += 32) {
                    const int x = r_first + min(r, rows - 1), node = x / a.G, hq = w.h * a.G + x - node * a.G;
                    const uint64_t m = a.mask[(int64_t)w.b * a.T + node];
                    tb.mask[0][r] = (uint32_t)m, tb.mask[1][r] = (uint32_t)(m >> 32);
                    tb.row[r] = ((int64_t)w.b * a.T + node) * a.Hq + hq;
                    tb.q_at[r] = (int64_t)w.b * a.q.seq + (int64_t)node * a.q.node + (int64_t)hq * a.q.head;
                }
                if (lane == 0) tb.odd = 0, tb.bad = 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&st.table_full[side]);
            };
            if (keys && seg > 0) rows_table();
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const int t = w.t0 + i;
                const bool tree = t == w.nt - 1;
                bad = bad || (uint32_t)page >= (uint64_t)a.num_pages;
                const int used = tree ? 0 : (min(KT, w.s.len - t * KT) + box_rows - 1) / box_rows;  // boxes with an entry
                const int this_page = page, this_place = place;
                e += KT, pg += step_pages, place += step_places;
                if (place >= a.page_size) place -= a.page_size, ++pg;
                page = look();
#pragma unroll 1
                for (int p = 0; p < pairs; ++p) {
                    ok = __all_sync(FULL_MASK, mbar_wait(&st.empty[stage], (round & 1) ^ 1));
                    if (!ok) break;
                    const int nb = min(2, boxes - 2 * p);
                    uint64_t* full = &st.full[stage];
                    unsigned char* dst = ring + stage * stage_bytes;
                    if (lane == 0) mbar_arrive_expect_tx(full, (tree ? a.T : used * box_rows) * 128 * nb);
                    __syncwarp();
                    if (tree) {
                        if (lane < nb) tma_load(dst + lane * BOX_BYTES, map_new, (2 * p + lane) * BOX, 0, w.h, w.b, full);
                    } else if (lane < used) {
                        tma_load(dst + lane * box_rows * 128, map, 2 * p * BOX, this_place, w.h, this_page, full);
                        if (nb > 1)
                            tma_load(dst + BOX_BYTES + lane * box_rows * 128, map, (2 * p + 1) * BOX, this_place, w.h,
                                     this_page, full);
                    }
                    if (++stage == end) stage = first, ++round;
                }
                if (keys && seg == 0 && i == 0) rows_table();  // (the first loads go ahead of it)
            }
            if (keys) {
                bad = __any_sync(FULL_MASK, bad);
                if (lane == 0) {
                    if (bad) st.table[side].bad = 1, set_error(a.dev_err, KV_DEVERR_PAGE);
                    mbar_arrive(&st.seg_loaded[side]);
                }
            }
            ++seg;
        } while (ok && w.next());
        if (!ok && lane == 0) st.stopped = 1, set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
        landed(st.full, first, end, stage, round);
    } else if ((warp == S_WARP || warp == O_WARP) && busy) {
        // ------------------------------------------------------------ MMAs
        const bool outs = warp == O_WARP;
        const uint32_t id = outs ? idesc(H::type, true, true, NR) : idesc(H::type, false, false, NR);
        const uint32_t aQ = smem_addr(sQ), aP = smem_addr(sP), aR = smem_addr(ring), tm = uniform(tmem);
        const int first = outs ? k_stages : 0, end = outs ? stages : k_stages;
        int stage = first;
        uint32_t round = 0, n_t = 0, seg = 0, asked = 0;  // asked: copies of queries
        bool ok = true;
        do {
            const int n = uniform(w.t1 - w.t0);
            // the tile whose V has rows that the softmax threads clear: the cache's last one, if it is not
            // full, and the nodes'
            const int t0 = uniform(w.t0), short_t = uniform(w.s.len % KT ? w.nt - 2 : w.nt - 1), tree_t = uniform(w.nt - 1);
            if (!outs) {
                // the queries, once the last segment's products have read theirs: by TMA where the block holds
                // whole nodes (nodes past the count may be there too: their columns are not looked at) ...
                const int side = seg & 1, r_first = w.rb * NR;
                if (n_t > 0) ok = warp_wait(&st.s_full[(n_t - 1) & 1], ((n_t - 1) >> 1) & 1);
                if (NR % a.G == 0) {
                    if (lane == 0 && ok) {
                        mbar_arrive_expect_tx(&st.q_full, boxes * NR * 128);
#pragma unroll 1
                        for (int x = 0; x < boxes; ++x)
                            tma_load(sQ + x * NR * 128, &maps.q, x * BOX, w.h * a.G, r_first / a.G, w.b, &st.q_full);
                    }
                    __syncwarp();
                    asked += ok;
                    ok = ok && warp_wait(&st.q_full, seg & 1);
                } else {  // ... else by the lanes, eight loads of one out before the first is stored
                    ok = ok && warp_wait(&st.table_full[side], (seg >> 1) & 1);
                    const Table<NR>& tb = st.table[side];
                    const int rows = min(NR, w.s.nodes * a.G - r_first), c = lane & 7;
#pragma unroll 1
                    for (int x = 0; x < boxes && ok; ++x) {
                        const bool in = x * BOX + c * 8 < a.d;
#pragma unroll 1
                        for (int r0 = lane >> 3; r0 < NR; r0 += 32) {
                            uint4 v[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const int r = r0 + 4 * y;
                                v[y] = make_uint4(0, 0, 0, 0);
                                if (r < rows && in)
                                    v[y] = *reinterpret_cast<const uint4*>(static_cast<const ST*>(a.q.p) + tb.q_at[r] + x * BOX +
                                                                           c * 8);
                            }
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const int r = r0 + 4 * y;
                                if (r < NR) *reinterpret_cast<uint4*>(sQ + x * NR * 128 + r * 128 + ((c ^ (r & 7)) << 4)) = v[y];
                            }
                        }
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                }
            }
            ++seg;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i, ++n_t) {
                const int buf = n_t & (outs ? pb : 1), t = t0 + i;
                if (outs) {
                    if (t == tree_t || t == short_t) {
                        int s2 = stage;
                        uint32_t r2 = round;
#pragma unroll 1
                        for (int p = 0; p < pairs && ok; ++p) {
                            ok = warp_wait(&st.full[s2], r2 & 1);
                            if (++s2 == end) s2 = first, ++r2;
                        }
                        if (ok && lane == 0) st.v_stage = stage, mbar_arrive(&st.v_ok);
                        __syncwarp();
                    }
                    ok = ok && warp_wait(&st.p_full[buf], (n_t >> pb) & 1);
                } else if (n_t >= 2) {
                    ok = warp_wait(&st.s_empty[buf], ((n_t >> 1) - 1) & 1);
                }
#pragma unroll 1
                for (int p = 0; p < pairs && ok; ++p) {
                    ok = warp_wait(&st.full[stage], round & 1);
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t in = aR + stage * stage_bytes;
                    const int nb = min(2, boxes - 2 * p);
                    if (outs) {
                        // A: 128 elements of d (the second 64 in the stage's second box; where there is
                        // none, the first again: its lanes are not read)
                        const uint64_t da = desc(in, nb > 1 ? BOX_BYTES : 0, 1024, SW128);
                        const uint64_t db = desc(aP + buf * p_bytes<NR>(), 128, KT * 16, SW_NONE);
#pragma unroll
                        for (int k = 0; k < KT / 16; ++k)
                            mma(tm + TM_O + p * NR, da + k * (2048 >> 4), db + k * (256 >> 4), id, i % FOLD + k > 0);
                    } else {
                        const uint64_t da = desc(in, 16, 1024, SW128), db = desc(aQ + 2 * p * NR * 128, 16, 1024, SW128);
#pragma unroll
                        for (int k = 0; k < BOX / 16; ++k)  // (past the end of d both operands are zero)
                            mma(tm + TM_S + buf * NR, da + k * (32 >> 4), db + k * (32 >> 4), id, p + k > 0);
                        if (nb > 1) {
#pragma unroll
                            for (int k = 0; k < BOX / 16; ++k)
                                mma(tm + TM_S + buf * NR, da + (BOX_BYTES >> 4) + k * (32 >> 4),
                                    db + (NR * 128 >> 4) + k * (32 >> 4), id, true);
                        }
                    }
                    commit(&st.empty[stage]);
                    if (++stage == end) stage = first, ++round;
                }
                if (ok) commit(outs ? &st.p_empty[buf] : &st.s_full[buf]);
            }
        } while (ok && w.next());
        // products and copies in flight end before tensor memory is freed and the CTA leaves, also where it is the
        // softmax warps that gave up (else nobody waits here for long: they have waited for these)
        if (!ok && lane == 0) st.stopped = 1, set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
        if (asked) mbar_wait(&st.q_full, (asked - 1) & 1);
        commit(&st.drain[outs]);
        mbar_wait(&st.drain[outs], 0);
        __syncwarp();
    } else if (warp < SM_WARPS && busy) {
        // ------------------------------------------------------------ softmax
        const int g = warp >> 2, quad = warp & 3, key = quad * 32 + lane, gt = tid & 127, g0 = g * NRH;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        // (a scale of zero as the smallest normal number: -inf times it stays -inf)
        const float c2 = a.scale == 0.f ? 1.1754944e-38f : a.scale * LOG2E;
        const int64_t part_floats = kv_part_floats(NR, a.d);
        uint32_t n_t = 0, n_v = 0, seg = 0;  // tiles, v_ok rounds and segments so far
        bool failed = false, stop = false;   // stop: the whole group gives up
        Two l[NRH / 2];  // this key's share of the rows' sums
        if (gt < NRH) st.nref[g0 + gt] = -REF_NONE;
        group_sync(g);
        do {
            const int rows = min(NR, w.s.nodes * a.G - w.rb * NR), n = w.t1 - w.t0, side = seg & 1;
            Table<NR>& tb = st.table[side];
            failed = failed || !mbar_wait(&st.table_full[side], (seg >> 1) & 1);
#pragma unroll
            for (int r = 0; r < NRH / 2; ++r) l[r] = 0;
            bool big = false;

            for (int i = 0; i < n; ++i, ++n_t) {
                const int t = w.t0 + i, buf = n_t & 1;
                const bool tree = t == w.nt - 1;
                const int live = tree ? w.s.nodes : min(KT, w.s.len - t * KT);
                const uint32_t tm_s = tmem + lane_base + TM_S + buf * NR + g0;
                const bool dead = key >= live;  // no key in this thread's row of the tile
                failed = failed || !mbar_wait(&st.s_full[buf], (n_t >> 1) & 1);
#ifdef GDN_TEST_STALL
                if (blockIdx.x == gridDim.x / 2 && g == 0 && n_t == 1) failed = failed || !mbar_wait(&st.never, 0);
#endif
                tc::fence_after();
                if (tree) {  // scores that a row does not see, made such that the scaled ones are -inf
                    const float never = c2 > 0.f ? -INFINITY : INFINITY;
#pragma unroll 1
                    for (int r = 0; r < NRH; r += 8) {
                        float x[8];
                        tc::tmem_ld<8>(tm_s + r, x);
                        const uint4 m0 = *reinterpret_cast<const uint4*>(&tb.mask[quad & 1][g0 + r]);
                        const uint4 m1 = *reinterpret_cast<const uint4*>(&tb.mask[quad & 1][g0 + r + 4]);
                        const uint32_t m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            if (dead || !(m[y] >> lane & 1)) x[y] = never;
                        tc::tmem_st<8>(tm_s + r, x);
                    }
                }
                // Exponents c s - m are fused, one rounding: exact enough while a product's own rounding is under
                // one. Where a reference is larger, the segment goes on with scores that are scaled first, so
                // that the largest exponent is zero still.
                bool again = false;
                const auto scale_tile = [&]() {
#pragma unroll 1
                    for (int r = 0; r < NRH; r += 8) {
                        float x[8];
                        tc::tmem_ld<8>(tm_s + r, x);
#pragma unroll
                        for (int y = 0; y < 8; ++y) x[y] *= c2;
                        tc::tmem_st<8>(tm_s + r, x);
                    }
                };
                if (big) scale_tile();
                // sixteen scores at a time: 32 beside the 32 sums do not fit the registers of 20 warps, and are
                // read from tensor memory a second time below
                constexpr int CH = NRH < 16 ? NRH : 16;
                float s[CH];
                const float cf = big ? 1.f : c2;
                float over = -INFINITY;  // the largest exponent against the references
#pragma unroll
                for (int r0 = 0; r0 < NRH; r0 += CH) {
                    tc::tmem_ld<CH>(tm_s + r0, s);
#pragma unroll
                    for (int r = 0; r < CH; r += 4) {
                        // (one at a time: pairs cost two moves each out of the registers that tensor memory fills)
                        const float4 m = *reinterpret_cast<const float4*>(&st.nref[g0 + r0 + r]);
                        over = max3(max3(over, fmaf(s[r], cf, m.x), fmaf(s[r + 1], cf, m.y)), fmaf(s[r + 2], cf, m.z),
                                    fmaf(s[r + 3], cf, m.w));
                    }
                }
                if (dead) over = -INFINITY;
                if (failed) st.gave_up[g] = 1;
                if (group_any(g, failed || over > REF_SLACK + H::lift)) {
                    if (st.gave_up[g]) {
                        stop = true;
                        break;
                    }
                    // the tile's maxima, new references (the scores read once more, in a short loop: a unit
                    // comes here once or twice, and long straight code costs its fetch)
#pragma unroll 1
                    for (int r = 0; r < NRH; r += 8) {
                        float x[8];
                        tc::tmem_ld<8>(tm_s + r, x);
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            x[y] = warp_max(dead ? -INFINITY : big ? x[y] : x[y] * c2);
                            if (lane == y) st.warp_max[quad][g0 + r + y] = x[y];
                        }
                    }
                    group_sync(g);
                    if (gt < NRH) {
                        const int r = g0 + gt;
                        const float old = -st.nref[r];
                        float m = fmaxf(fmaxf(st.warp_max[0][r], st.warp_max[1][r]),
                                        fmaxf(st.warp_max[2][r], st.warp_max[3][r]));
                        m = fmaxf(m - H::lift, old);
                        if (fabsf(m) > FUSED_MOST && m > REF_NONE) st.big[g] = 1;
                        st.factor[r] = kv_ex2(old - m), st.nref[r] = -m;
                    }
                    group_sync(g);
                    if (!big && st.big[g]) big = true, again = true, scale_tile();
                    if (i > 0) {  // the sums and the accumulator, once the last tile's product is in it
#pragma unroll
                        for (int r = 0; r < NRH; r += 2) {
                            l[r / 2] = mul2(l[r / 2], *reinterpret_cast<const Two*>(&st.factor[g0 + r]));
                        }
                        const uint32_t p = n_t - 1;
                        failed = failed || !mbar_wait(&st.p_empty[p & pb], (p >> pb) & 1);
                        tc::fence_after();
                        const int blocks = i > FOLD ? 2 * pairs : pairs;  // O^T's, and its folds'
#pragma unroll 1
                        for (int hf = 0; hf < blocks; ++hf)
#pragma unroll 1
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
                    }
                }
                // weights: FP32 sums, rounded once to the cache's type for the product with the values
                const int pbuf = n_t & pb;
                unsigned char* dst = sP + pbuf * p_bytes<NR>() + g * (NRH / 8) * (KT * 16) + key * 16;
                const float ce = big ? 1.f : c2;
                uint32_t u[NRH / 2];
#pragma unroll
                for (int r0 = 0; r0 < NRH; r0 += CH) {
                    if (NRH > CH || again) tc::tmem_ld<CH>(tm_s + r0, s);
                    if (r0 + CH >= NRH) {  // the scores are read
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&st.s_empty[buf]);
                    }
                    if (!dead) {
#pragma unroll
                        for (int r = 0; r < CH; r += 8) {
#pragma unroll
                            for (int x = 0; x < 8; x += 4) {
                                const int i2 = (r0 + r + x) / 2;
                                const float4 m = *reinterpret_cast<const float4*>(&st.nref[g0 + r0 + r + x]);
                                const float p0 = kv_ex2(fmaf(s[r + x], ce, m.x)), p1 = kv_ex2(fmaf(s[r + x + 1], ce, m.y));
                                const float p2 = kv_ex2(fmaf(s[r + x + 2], ce, m.z)), p3 = kv_ex2(fmaf(s[r + x + 3], ce, m.w));
                                l[i2] = add2(l[i2], two(p0, p1)), l[i2 + 1] = add2(l[i2 + 1], two(p2, p3));
                                u[i2] = H::pack(p0, p1), u[i2 + 1] = H::pack(p2, p3);
                            }
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < CH / 2; ++r) u[r0 / 2 + r] = 0;
                    }
                }
                // the buffer is free once the product of the tile that used it is done: with one buffer that
                // product runs beside the exponentials above
                if (n_t >= (uint32_t)p_bufs) failed = failed || !mbar_wait(&st.p_empty[pbuf], ((n_t >> pb) - 1) & 1);
#pragma unroll
                for (int r = 0; r < NRH / 2; r += 4)
                    *reinterpret_cast<uint4*>(dst + (r / 4) * (KT * 16)) = make_uint4(u[r], u[r + 1], u[r + 2], u[r + 3]);
                if (i > 0 && i % FOLD == 0) {  // O^T into its folds; this tile's product begins a new one
                    const uint32_t p = n_t - 1;
                    failed = failed || !mbar_wait(&st.p_empty[p & pb], (p >> pb) & 1);
                    tc::fence_after();
#pragma unroll 1
                    for (int hf = 0; hf < pairs; ++hf)
#pragma unroll 1
                        for (int r = 0; r < NRH; r += 8) {
                            float o[8], f[8];
                            const uint32_t at = tmem + lane_base + hf * NR + g0 + r;
                            __syncwarp();
                            tc::tmem_ld<8>(at + TM_O, o);
                            if (i > FOLD) {
                                tc::tmem_ld<8>(at + TM_F, f);
#pragma unroll
                                for (int y = 0; y < 8; ++y) o[y] += f[y];
                            }
                            tc::tmem_st<8>(at + TM_F, o);
                        }
                }
                if (live < KT) {
                    // Rows of V past the last key become zero (0 x NaN would reach the sums), and so do a
                    // node's values that are not finite: the epilogue adds them to the rows that attend it.
                    failed = failed || !mbar_wait(&st.v_ok, n_v & 1);
                    ++n_v;
                    for (int x = g; x < boxes && !failed; x += NG) {  // (v_stage is not there if the wait ran out)
                        int stage = st.v_stage + (x >> 1);
                        if (stage >= stages) stage -= v_stages;
                        uint4* row = reinterpret_cast<uint4*>(ring + stage * stage_bytes + (x & 1) * BOX_BYTES + key * 128);
#pragma unroll 1
                        for (int y = 0; y < 8; ++y) {
                            const int c = y ^ (lane & 7);  // (an order without bank conflicts)
                            if (dead) row[c] = make_uint4(0, 0, 0, 0);
                            else if (tree && has_odd<ST>(row[c])) row[c] = clear_odd<ST>(row[c]), tb.odd = 1;
                        }
                    }
                    __threadfence_block();  // tb.odd, for every group once the product is done
                }
                tc::fence_async_smem();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&st.p_full[pbuf]);
            }
            if (stop) break;
            // ---- row sums over the group's threads, then the outputs
            const float own = sum_rows<NRH>(l, lane);
            if (lane < NRH) st.warp_max[quad][g0 + lane] = own;
            group_sync(g);
            const bool whole = w.whole();
            float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later) * part_floats;
            failed = failed || !mbar_wait(&st.seg_loaded[side], (seg >> 1) & 1);
            const bool bad = tb.bad;
            if (gt < NRH) {
                const int r = g0 + gt;
                const float sum = bad ? 0.f : st.warp_max[0][r] + st.warp_max[1][r] + st.warp_max[2][r] + st.warp_max[3][r];
                st.factor[r] = bad ? 0.f : whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                if (r < rows) {
                    if (!whole)
                        part[NR * a.d + r] = -st.nref[r], part[NR * a.d + NR + r] = bad ? -1.f : sum;
                    else if (a.lse)
                        a.lse[tb.row[r]] = sum == 0.f ? -INFINITY : (log2f(sum) - st.nref[r]) * LN2;
                }
                st.nref[r] = -REF_NONE;  // for the next segment
                st.big[g] = 0;
            }
            group_sync(g);
            failed = failed || !mbar_wait(&st.p_empty[(n_t - 1) & pb], ((n_t - 1) >> pb) & 1);
            tc::fence_after();
            const bool odd = w.t1 == w.nt && tb.odd;
#pragma unroll 1
            for (int i = 0; i < pairs * (NRH / 8); ++i) {
                const int hf = i / (NRH / 8), r0 = g0 + (i - hf * (NRH / 8)) * 8, e = hf * 128 + key;
                float o[8];
                __syncwarp();
                tc::tmem_ld<8>(tmem + lane_base + TM_O + hf * NR + r0, o);
                if (n > FOLD) {
                    float f[8];
                    tc::tmem_ld<8>(tmem + lane_base + TM_F + hf * NR + r0, f);
#pragma unroll
                    for (int x = 0; x < 8; ++x) o[x] += f[x];
                }
                if (e >= a.d || r0 >= rows) continue;
                if (odd) add_odd<ST>(a, w.s.nodes, w.b, w.h, e, &tb.mask[0][r0], &tb.mask[1][r0], o);
                const float4 f0 = *reinterpret_cast<const float4*>(&st.factor[r0]);
                const float4 f1 = *reinterpret_cast<const float4*>(&st.factor[r0 + 4]);
                const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                if (whole) {
                    ST* out = static_cast<ST*>(a.out) + e;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (r0 + x < rows) out[tb.row[r0 + x] * a.d] = H::round(f[x] == 0.f ? 0.f : o[x] * f[x]);
                } else {
                    float* out = part + (int64_t)r0 * a.d + e;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (r0 + x < rows) out[x * a.d] = f[x] == 0.f ? 0.f : o[x];
                }
            }
            tc::fence_before();
            if (tid == 0 && w.last()) static_cast<KvBorder*>(a.border)[blockIdx.x] = kv_border(a, split, w);
            if (failed) st.gave_up[g] = 1;
            group_sync(g);  // the sums and factors are read
            stop = st.gave_up[g];
            if (lane == 0) mbar_arrive(&st.table_empty[side]);
            ++seg;
        } while (!stop && w.next());
        if (stop && lane == 0) st.stopped = 1, set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
    }
    if (warp == S_WARP) kv_empty_rows(a, a.B <= NT ? st.scan.seq : nullptr, lane, 32);
    if (!busy && tid == 0) static_cast<KvBorder*>(a.border)[blockIdx.x].rows = 0;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == O_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
    if (st.stopped) refuse_range<NR>(a, st);
}

}  // namespace gdn
