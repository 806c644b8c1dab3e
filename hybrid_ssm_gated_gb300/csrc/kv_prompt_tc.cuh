// kv_prompt_tc.cuh -- causal attention of packed prompts over the paged cache on the
// tcgen05 tensor cores (16-bit caches whose pages hold a multiple of 8 entries and
// whose rows the TMA engine can address; up to 128 query heads a key head).
//
// Mathematics. One pass over tiles of 128 (QT = 1: 64) keys for tiles of 128 query rows: S = Q K^T
// (128 x 128), P = 2^{c S - m} with a reference m a row, O += P V (128 x d). A thread
// owns a row: its 128 scores of a tile come from tensor memory into its registers, and
// maximum, sum and weights need no other thread. The weights go back to tensor memory,
// over the scores, as the A operand of the second product.
//
// The reference lags behind the row's maximum, and weights in fp16 are lifted by seven
// powers of two, as in kv_tc.cuh. O is a sum over FOLD tiles in tensor memory (whose
// FP32 sums are cut off towards zero), which the softmax threads then add, rounding to
// nearest, to a sum in the CTA's partial in the workspace: tensor memory is full.
//
// Kernel shape: persistent, one CTA a SM;
//   QT = 2 (d up to 128): a unit is two tiles of query rows, which share each tile of
//     keys and values; while one tile's weights form, the tensor cores work for the
//     other one. Tensor memory: two S (P over them), two O.
//   QT = 1 (d above 128, and calls with few units): one tile, two buffers of S in turn.
//   softmax    four warps a tile of rows, thread = row = tensor-memory lane;
//   K, V       a warp each: tiles by TMA into a ring of stages of a tile's keys x 128
//              elements, boxes of as many keys as a page and the tile share;
//              the V warp loads a unit's queries too, once the last one's products have
//              read theirs (whole tokens: a tile of rows holds as many as have their G
//              heads in it);
//   products   two warps, an elected thread of each. QT = 2: one a tile of rows, which
//              issues all of its products in order: S right behind the last product that
//              reads the P it is written over, waiting for nobody (the tensor cores take a
//              thread's products in the order of their issue). QT = 1: one for S, one
//              for O. (A commit holds a thread up for 120 to 210 cycles, one right behind
//              another for 12: a thread for both tiles of rows took 4100 cycles a tile of
//              keys where the products take 2048, one for S and O of one tile 2800 where
//              they take 1280.)
// A tile's chain is S, softmax, O, S ...: what bounds the kernel is its latency. So the
// weights' first half is formed against the last tile's reference while the maximum is
// still looked for (it is formed again where that moved the reference), and is given to
// the tensor cores while the second half is formed.
// Bound and measurement (GB300, whole calls with the join). QT = 2: a tile of 256 rows by
// 128 keys takes some 3300 cycles where its products take 2048: the two tiles' blocks
// (O of one's last weights, then S of its next keys: 1100 to 1250 cycles) and the way
// from one thread of products to the other, 300 each. 20000 tokens (32 / 8 heads, d =
// 128, bf16, 3.28 TFLOP) take 2.23 ms, 1470 TFLOP/s or 0.75 of the measured rate (tensor
// pipe 50% active at 6000 tokens); chunks of up to 512 tokens behind up to 8192 for 15
// sequences (fp16, 0.40 TFLOP) 403 to 407 us, 990: half-filled last units (whose empty
// second tile is computed all the same), and 5 to 9 us a unit's beginning and end. The
// chain does not shorten with d: 8192 tokens of 32 / 8 heads take 427 us at d = 128 (1289
// TFLOP/s), 401 at 96, 394 at 80, 378 at 64 (726). QT = 1: 8192 tokens of 16 / 2 heads,
// d = 256, 492 to 510 us, 1077 to 1117 TFLOP/s; 16000 of them 1773 us, 1183; 8192 at d =
// 192 415 us (995), at 136 414. 700 of d = 256 30 us: latency, of which the beginning
// (lengths, places, first loads) is 6, a unit's end 3, the join 7.
// Registers: QT = 2 spills 644 bytes a thread of stores and 552 of loads at its 168,
// 1.2% of the instructions that 6000 tokens issue. QT = 1 (200 registers) spills nothing.
// Measured and not taken (20000 tokens): sixteen softmax warps, two threads a row (2700
// us: 96 registers); one thread of products for both tiles (2690); the turn passed on
// ahead of S (2630) or amid it (2300 to 2440); weights given over at once (2460) or in
// three parts (2680); scalar instead of packed exponents' arithmetic (2640).
// A tile of which some row sees a part ("mixed") has its values looked through by the
// softmax threads: rows of V past the sequence's end become zero, and so does what is
// not finite (0 x NaN would reach rows that do not see it); the epilogue adds the
// latter to the rows that do.
#pragma once

#include "kv_prompt.cuh"
#include "kv_tc.cuh"

namespace gdn {

namespace kpt {

using kvt::BOX;
constexpr int TILE = 128;  // rows of a tile
// Keys of a tile: at d = 256 a tile of 128 of keys and one of values leave room for no second one beside the queries, and
// the next keys' way from L2 was the kernel's period (4700 cycles a tile); 64 leave two. (N = 64 costs a product of S 48
// cycles instead of 32.)
__host__ __device__ constexpr int keys_of(int QT) { return QT == 2 ? 128 : 64; }
constexpr int KEEP = 32;   // sequences that the scan keeps
constexpr int MAX_STAGES = 12;
constexpr float MOST = 32768.f;  // sum of the weights of half a tile, at most (each then fits fp16)
// Entries of one sum in tensor memory: what its products' cut-off costs (2^-21 of the sum a product of 16 keys at most)
// stays under half of half a unit of the outputs' type.
template <typename ST>
__host__ __device__ constexpr int fold_keys() { return 4096; }
template <>
__host__ __device__ constexpr int fold_keys<__nv_bfloat16>() { return 16384; }
__host__ __device__ constexpr int threads(int QT) { return (4 * QT + 4) * 32; }

struct Maps {
    CUtensorMap k, v, q;
};

template <int QT>
struct __align__(16) State {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];  // the K ring's stages, then the V ring's
    uint64_t s_full[2], o_done[2], p_full[2][2], q_full, q_free, v_ok, v_clean, drain[2], turn[2];
    uint64_t seg_open[2], seg_loaded[2], seg_free[2];
    KpScan<threads(QT), KEEP> scan;
    int bad[2], odd[2];  // of this segment and the next: a page outside the pool; a value that is not finite
    int v_stage, stopped;
    uint32_t tmem;
#ifdef GDN_TEST_STALL
    uint64_t never;
#endif
};

template <int QT>
__host__ __device__ constexpr int stage_bytes(int boxes) { return (boxes > 1 ? 2 : 1) * keys_of(QT) * BOX * 2; }
template <int QT>
__host__ __device__ constexpr int smem_bytes(int boxes, int stages) {
    return 1024 + QT * boxes * TILE * 128 + stages * stage_bytes<QT>(boxes) + (int)sizeof(State<QT>);
}

// Operand descriptors of the 128-byte swizzle, 1024 bytes between groups of eight rows: the upper word is the same for
// all, the lower one holds address and leading offset.
constexpr uint32_t DESC_HI = (1024 >> 4) | 1u << 14 | kvt::SW128 << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3FFFF) >> 4 | (lbo >> 4) << 16; }

// One thread of a converged warp.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r != 0;
}

// A product, by one thread; A in shared memory, or in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"((uint32_t)accumulate), "n"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"((uint32_t)accumulate), "n"(DESC_HI)
        : "memory");
}

// Sixteen words to consecutive columns of this thread's lane; in tensor memory once st_wait returns.
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The values of a row's mixed tiles that are not finite, added to its outputs where the row sees the entry (entries
// `from` to `last`): output e is out[e * step], of type `dtype`.
template <typename ST>
__device__ __noinline__ void add_odd(const KvArgs& a, const int32_t* table, int h, int from, int last, void* out, int64_t step,
                                     int dtype) {
    for (int e = from; e <= last; ++e) {
        const int pg = e / a.page_size, page = table[pg];
        if ((uint32_t)page >= (uint64_t)a.num_pages) continue;
        const int64_t at = kv_at(a.v, page, h, e - pg * a.page_size);
        for (int x = 0; x < a.d; ++x) {
            const float v = load_elem(a.v.p, at + x, Store<ST>::code);
            if (!isfinite(v)) store_elem(out, x * step, dtype, load_elem(out, x * step, dtype) + v);
        }
    }
}

// Four pieces of each of four lanes (a lane's piece i its row's) turned, so that piece k of a lane is of row k and all
// lie next to one another.
__device__ __forceinline__ void turn4(uint4 (&x)[4], int lane) {
#pragma unroll
    for (int b = 1; b < 4; b <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & b) continue;
            const bool up = lane & b;
            uint4& lo = x[i];
            uint4& hi = x[i | b];
            uint4 y = up ? lo : hi;
            y.x = __shfl_xor_sync(FULL_MASK, y.x, b), y.y = __shfl_xor_sync(FULL_MASK, y.y, b);
            y.z = __shfl_xor_sync(FULL_MASK, y.z, b), y.w = __shfl_xor_sync(FULL_MASK, y.w, b);
            if (up) lo = y;
            else hi = y;
        }
}

// What a CTA leaves whose waits ran out, by the whole block: the rows of its range as those of a refused sequence.
template <int QT>
__device__ __noinline__ void refuse_range(const KvArgs& a, const State<QT>& st) {
    constexpr int NT = threads(QT), PLACES = QT * TILE, KT = keys_of(QT);
    bool some;
    KpWalk<KT> w(a, st.scan, some);
    if (!some) return;
    do {
        const int r0 = w.r0(), rows = w.rows();
        if (w.whole()) {
            for (int64_t i = threadIdx.x; i < (int64_t)rows * a.d; i += NT) {
                const int r = (int)(i / a.d), x = r0 + r, tok = x / a.G;
                const int64_t row = (int64_t)(w.s.first + tok) * a.Hq + w.h * a.G + (x - tok * a.G);
                store_elem(a.out, row * a.d + (i - (int64_t)r * a.d), a.dtype, 0.f);
                if (a.lse && i == (int64_t)r * a.d) a.lse[row] = -INFINITY;
            }
        } else {
            float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later()) * kp_part_floats(PLACES, a.d) + (int64_t)PLACES * a.d;
            for (int r = threadIdx.x; r < PLACES; r += NT) part[r] = -INFINITY, part[PLACES + r] = -1.f;
            if (threadIdx.x == 0 && w.t0 == 0) kp_border(a, st.scan, w);
        }
    } while (w.next());
}

}  // namespace kpt

// boxes: 64-element boxes of d; k_stages, v_stages: of the rings; box_rows: keys of one TMA box.
template <typename ST, int QT>
__global__ void __launch_bounds__(kpt::threads(QT), 1)
    kv_prompt_tc_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ kpt::Maps maps, const int boxes,
                        const int k_stages, const int v_stages, const int box_rows) {
    using namespace kpt;
    using kvt::idesc, kvt::warp_wait, kvt::tma_load;
    using kvt::Two, kvt::two, kvt::fma2, kvt::add2, kvt::parts, kvt::max3;
    using H = kvt::Half16<ST>;
    constexpr int KT = keys_of(QT), FOLD = fold_keys<ST>() / KT, BOX_BYTES = KT * BOX * 2, HALF = KT / 2;
    constexpr int NT = threads(QT), SM_WARPS = 4 * QT, PLACES = QT * TILE;
    constexpr int K_WARP = SM_WARPS, V_WARP = SM_WARPS + 1, M_WARP = SM_WARPS + 2;
    constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int pairs = (boxes + 1) >> 1, one_stage = stage_bytes<QT>(boxes), stages = k_stages + v_stages;
    unsigned char* sQ = smem;
    unsigned char* ring = smem + QT * boxes * TILE * 128;
    State<QT>& st = *reinterpret_cast<State<QT>*>(ring + stages * one_stage);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.tile_rows;  // rows of a tile: whole tokens

    kv_grid_launch();
    if (warp == K_WARP) {
        if (lane < 3) {
            const CUtensorMap* m = lane == 0 ? &maps.k : lane == 1 ? &maps.v : &maps.q;
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
        }
        if (lane < stages) mbar_init(&st.full[lane], 1), mbar_init(&st.empty[lane], QT);
        if (lane < 2) {
            mbar_init(&st.s_full[lane], 1), mbar_init(&st.o_done[lane], 1);
            mbar_init(&st.p_full[lane][0], 4), mbar_init(&st.p_full[lane][1], 4);
            mbar_init(&st.seg_open[lane], 1), mbar_init(&st.seg_loaded[lane], 1), mbar_init(&st.seg_free[lane], SM_WARPS);
            st.bad[lane] = st.odd[lane] = 0;
        }
        if (lane == 2) {
            mbar_init(&st.q_full, 1), mbar_init(&st.q_free, QT), mbar_init(&st.v_ok, 1), mbar_init(&st.v_clean, SM_WARPS);
            mbar_init(&st.drain[0], 1), mbar_init(&st.drain[1], 1), st.stopped = 0;
            mbar_init(&st.turn[0], 1), mbar_init(&st.turn[1], 1);
        }
#ifdef GDN_TEST_STALL
        if (lane == 0) mbar_init(&st.never, 1);
#endif
        fence_barrier_init();
    }
    if (warp == M_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&st.tmem)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) kp_no_border(a);
    tc::fence_before();
    kp_locate<KT>(a, st.scan);
    tc::fence_after();
    const uint32_t tmem = st.tmem;
    bool busy;
    KpWalk<KT> w(a, st.scan, busy);
    // the first tile of the unit that some row sees a part of only
    const auto first_mixed = [&]() { return (w.s.len - w.s.n + w.r0() / a.G + 1) / KT; };

    // (of two tiles' kernel) registers to the threads that hold a row of scores: 256 x 216 + 128 x 72 of the launch's
    // 384 x 168
    if (warp >= SM_WARPS) {
    if constexpr (QT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if ((warp == K_WARP || warp == V_WARP) && busy) {
        // ------------------------------------------------------------ loads
        const bool keys = warp == K_WARP;
        const CUtensorMap* map = keys ? &maps.k : &maps.v;
        const int first = keys ? 0 : k_stages, end = keys ? k_stages : stages;
        int stage = first;
        uint32_t round = 0, seg = 0, asked = 0;
        bool ok = true;
        const int per_tile = KT / box_rows, step_pages = KT / a.page_size, step_places = KT - step_pages * a.page_size;
        do {
            const int side = seg & 1;
            const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
            bool bad = false;
            // this lane's box of the next tile: its page (one tile ahead) and place
            int e = w.t0 * KT + lane * box_rows, pg = e / a.page_size, place = e - pg * a.page_size;
            const auto look = [&]() { return lane < per_tile && e < w.s.len ? table[pg] : 0; };
            int page = look();
            if (!keys) {  // the unit's queries
                if (seg > 0) ok = warp_wait(&st.q_free, (seg - 1) & 1);
                if (ok) {
                    if (lane == 0) mbar_arrive_expect_tx(&st.q_full, QT * boxes * per * 128);
                    __syncwarp();
                    if (lane < QT * boxes) {
                        const int j = lane / boxes, x = lane - j * boxes;
                        tma_load(sQ + (j * boxes + x) * TILE * 128, &maps.q, x * BOX, w.h * a.G,
                                 w.s.first + w.r0() / a.G + j * (per / a.G), 0, &st.q_full);
                    }
                    __syncwarp();
                    ++asked;
                }
            }
            if (keys) {
                if (seg >= 2) {
                    ok = warp_wait(&st.seg_free[side], ((seg >> 1) - 1) & 1);
                    if (lane == 0) st.bad[side] = st.odd[side] = 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&st.seg_open[side]);
            }
#pragma unroll 1
            for (int t = w.t0; t < w.t1 && ok; ++t) {
                bad = bad || (uint32_t)page >= (uint64_t)a.num_pages;
                const int used = (min(KT, w.s.len - t * KT) + box_rows - 1) / box_rows;  // boxes with an entry
                const int this_page = page, this_place = place;
                e += KT, pg += step_pages, place += step_places;
                if (place >= a.page_size) place -= a.page_size, ++pg;
                page = look();
#pragma unroll 1
                for (int p = 0; p < pairs; ++p) {
                    ok = warp_wait(&st.empty[stage], (round & 1) ^ 1);
                    if (!ok) break;
                    const int nb = min(2, boxes - 2 * p);
                    uint64_t* full = &st.full[stage];
                    unsigned char* dst = ring + stage * one_stage;
                    if (lane == 0) mbar_arrive_expect_tx(full, used * box_rows * 128 * nb);
                    __syncwarp();
                    if (lane < used) {
                        tma_load(dst + lane * box_rows * 128, map, 2 * p * BOX, this_place, w.h, this_page, full);
                        if (nb > 1)
                            tma_load(dst + BOX_BYTES + lane * box_rows * 128, map, (2 * p + 1) * BOX, this_place, w.h,
                                     this_page, full);
                    }
                    if (++stage == end) stage = first, ++round;
                }
            }
            if (keys) {
                bad = __any_sync(FULL_MASK, bad);
                if (lane == 0) {
                    if (bad) st.bad[side] = 1, set_error(a.dev_err, KV_DEVERR_PAGE);
                    mbar_arrive(&st.seg_loaded[side]);
                }
            }
            ++seg;
        } while (ok && w.next());
        if (!ok && lane == 0) st.stopped = 1, set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
        kvt::landed(st.full, first, end, stage, round);
        if (asked) mbar_wait(&st.q_full, (asked - 1) & 1);
    } else if ((warp == M_WARP || warp == M_WARP + 1) && busy) {
        // ------------------------------------------------------------ products
        // (one thread, and one that the compiler knows to be alone: elsewhere a product took 107 cycles to issue, for
        // operands that might differ from thread to thread)
        if (elected()) {
            const int j = warp - M_WARP;
            const uint32_t id_s = idesc(H::type, false, false, KT), aQ = smem_addr(sQ) + (QT == 2 ? j * boxes * TILE * 128 : 0), aR = smem_addr(ring);
            int ks = 0, vs = k_stages;  // the rings' next stages
            uint32_t k_round = 0, v_round = 0, n_t = 0, n_v = 0, seg = 0;
            bool ok = true;
            // The two tiles take turns at the tensor cores, so that one's weights form while the other's products run (left
            // alone they fall into step and wait for both).
            uint32_t turns = 0;
            const auto my_turn = [&]() {
                if (QT == 2 && (j == 1 || turns > 0)) ok = ok && mbar_wait(&st.turn[j], (j == 1 ? turns : turns - 1) & 1);
                ++turns;
            };
            const auto pass = [&]() {
                if (QT == 2) mbar_arrive(&st.turn[j ^ 1]);
            };
            const auto k_there = [&]() {
                int sk = ks;
                uint32_t rk = k_round;
                for (int p = 0; p < pairs && ok; ++p) {
                    ok = mbar_wait(&st.full[sk], rk & 1);
                    if (++sk == k_stages) sk = 0, ++rk;
                }
                tc::fence_after();
            };
            const auto scores = [&](int buf) {  // S into buffer `buf`, from the K stages at ks, which are there
                const uint32_t to = tmem + TM_S + buf * KT;
                int sk = ks;
#pragma unroll 1
                for (int p = 0; p < pairs; ++p) {
                    const int nb = min(2, boxes - 2 * p);
                    const uint32_t db = desc_lo(aR + sk * one_stage, 16), da = desc_lo(aQ + 2 * p * TILE * 128, 16);
#pragma unroll 1
                    for (int x = 0; x < nb; ++x) {
                        const int steps = min(BOX / 16, (a.d - (2 * p + x) * BOX + 15) / 16);
                        const uint32_t da_x = da + x * (TILE * 128 >> 4), db_x = db + x * (BOX_BYTES >> 4);
                        if (steps == BOX / 16) {
#pragma unroll
                            for (int k = 0; k < BOX / 16; ++k)
                                mma_ss(to, da_x + k * (32 >> 4), db_x + k * (32 >> 4), id_s, p + x + k > 0);
                        } else {
#pragma unroll 1
                            for (int k = 0; k < steps; ++k)
                                mma_ss(to, da_x + k * (32 >> 4), db_x + k * (32 >> 4), id_s, p + x + k > 0);
                        }
                    }
                    if (++sk == k_stages) sk = 0;
                }
                pass();  // (ahead of the commits, which hold this thread up)
                tc::commit(&st.s_full[buf]);
                for (int p = 0; p < pairs; ++p) {
                    tc::commit(&st.empty[ks]);
                    if (++ks == k_stages) ks = 0, ++k_round;
                }
            };
            do {
                const int n = w.t1 - w.t0, t0 = w.t0, mixed = first_mixed();
                if (QT == 2 || j == 0) ok = ok && mbar_wait(&st.q_full, seg & 1);
                if constexpr (QT == 1) {
                    if (j == 0) {
#pragma unroll 1
                        for (int i = 0; i < n && ok; ++i, ++n_t) {
                            k_there();
                            if (n_t >= 2) ok = ok && mbar_wait(&st.o_done[n_t & 1], ((n_t >> 1) - 1) & 1);
                            if (!ok) break;
                            tc::fence_after();
                            scores(n_t & 1);
                            if (i + 1 == n) tc::commit(&st.q_free);
                        }
                        ++seg;
                        continue;
                    }
                } else {
                    if (ok) k_there();
                    my_turn();
                    if (ok) {
                        scores(j);
                        if (n == 1) tc::commit(&st.q_free);
                    }
                }
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i, ++n_t) {
                    const bool more = i + 1 < n;
                    const int buf = QT == 2 ? j : n_t & 1;
                    const uint32_t use = QT == 2 ? n_t : n_t >> 1;
                    if (QT == 2 && more) k_there();
                    int sp = vs;
                    uint32_t rp = v_round;
                    for (int p = 0; p < pairs && ok; ++p) {
                        ok = mbar_wait(&st.full[sp], rp & 1);
                        if (++sp == stages) sp = k_stages, ++rp;
                    }
                    if (ok && t0 + i >= mixed) {  // the softmax threads look the values through
                        if (j == (QT == 2 ? 0 : 1)) st.v_stage = vs, mbar_arrive(&st.v_ok);
                        ok = mbar_wait(&st.v_clean, n_v & 1);
                        ++n_v;
                    }
                    my_turn();
#pragma unroll 1
                    for (int half = 0; half < 2 && ok; ++half) {
                        ok = mbar_wait(&st.p_full[buf][half], use & 1);
                        if (!ok) break;
                        tc::fence_after();
                        sp = vs;
#pragma unroll 1
                        for (int p = 0; p < pairs; ++p) {
                            const int nb = min(2, boxes - 2 * p), N = min(128, (a.d - p * 128 + 15) / 16 * 16);
                            const uint32_t id = idesc(H::type, false, true, N), to = tmem + TM_O + (QT == 2 ? j : p) * 128;
                            const uint32_t from = tmem + TM_S + buf * KT + half * (HALF / 2);
                            const uint32_t db = desc_lo(aR + sp * one_stage + half * HALF * 128, nb > 1 ? BOX_BYTES : 0);
#pragma unroll
                            for (int k = 0; k < HALF / 16; ++k) mma_ts(to, from + k * 8, db + k * (2048 >> 4), id, i % FOLD + half + k > 0);
                            if (++sp == stages) sp = k_stages;
                        }
                    }
                    if (!ok) break;
                    if (QT == 2 && more) {
                        scores(j);
                        if (i + 2 == n) tc::commit(&st.q_free);
                    } else {
                        pass();
                        tc::commit(&st.o_done[buf]);
                    }
                    for (int p = 0; p < pairs; ++p) {
                        tc::commit(&st.empty[vs]);
                        if (++vs == stages) vs = k_stages, ++v_round;
                    }
                }
                ++seg;
            } while (ok && w.next());
            // products in flight end before tensor memory is freed and the CTA leaves, whoever gave up
            if (!ok) st.stopped = 1, set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
            tc::commit(&st.drain[j]);
            mbar_wait(&st.drain[j], 0);
        }
        __syncwarp();
    }
    if (warp == V_WARP) kp_empty_rows(a, a.B <= KEEP ? st.scan.seq : nullptr, lane, 32);
    } else {
    if constexpr (QT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    if (busy) {
        // ------------------------------------------------------------ softmax
        const int g = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tm_o = lane_base + TM_O + g * 128;
        const bool flip = a.scale < 0.f;
        // (a scale of zero as the smallest normal number: -inf times it stays -inf)
        const float c2 = a.scale == 0.f ? 1.1754944e-38f : fabsf(a.scale) * LOG2E;
        const bool vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
        uint32_t n_t = 0, n_v = 0, seg = 0;
        bool ok = true;
        // Tile x's product with V is done. (Of two tiles of rows: the next S, which is there, lay behind it, and
        // only a segment's last product has a barrier of its own.)
        const auto done = [&](uint32_t x, bool end) {
            bool y = true;
            if (QT == 1) y = warp_wait(&st.o_done[x & 1], (x >> 1) & 1);
            else if (end) y = warp_wait(&st.o_done[g], seg & 1);
            tc::fence_after();
            return y;
        };
        do {
            const int n = w.t1 - w.t0, side = seg & 1, prefix = w.s.len - w.s.n, rows = w.rows(), r0 = w.r0();
            const int mine = g * per + r;  // row of the unit
            const bool live = r < per && mine < rows;
            const int x = r0 + (live ? mine : r < per ? rows - 1 : min(g * per, rows - 1)), tok = x / a.G, last = prefix + tok;
            const int mixed = first_mixed();
            float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later()) * kp_part_floats(PLACES, a.d) + g * TILE + r;
            float m = -INFINITY, nref = 0.f, l = 0.f, folded = -INFINITY;  // reference (unscaled), lift - c m, sum; m of the fold
            bool big = false, taken = false;
            ok = ok && warp_wait(&st.seg_open[side], (seg >> 1) & 1);
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i, ++n_t) {
                const int t = w.t0 + i, buf = QT == 2 ? g : n_t & 1;
                const uint32_t tm_s = lane_base + TM_S + buf * KT;
                ok = warp_wait(&st.s_full[buf], (QT == 2 ? n_t : n_t >> 1) & 1);
#ifdef GDN_TEST_STALL
                if (blockIdx.x == gridDim.x / 2 && warp == 0 && n_t == 1) ok = ok && warp_wait(&st.never, 0);
#endif
                if (!ok) break;
                tc::fence_after();
                float s[KT];
                tc::tmem_ld<64>(tm_s, s);
                if constexpr (KT == 128) tc::tmem_ld<64>(tm_s + 64, s + 64);
                if (flip) {
#pragma unroll
                    for (int y = 0; y < KT; ++y) s[y] = -s[y];
                }
                if (t >= mixed) {
                    const int lim = last - t * KT;
#pragma unroll
                    for (int y = 0; y < KT; ++y)
                        if (y > lim) s[y] = -INFINITY;
                }
                if (i > 0 && i % FOLD == 0) {  // the sum in tensor memory joins the folds; this tile's product begins a new one
                    ok = done(n_t - 1, false);
                    const float f = folded == -INFINITY ? 1.f : kv_ex2((folded - m) * c2);
#pragma unroll 1
                    for (int e = 0; e < a.d; e += 8) {
                        float o[8], old[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) old[y] = i > FOLD ? part[(e + y) * PLACES] : 0.f;
                        tc::tmem_ld<8>(tm_o + e, o);
#pragma unroll
                        for (int y = 0; y < 8; ++y) part[(e + y) * PLACES] = fmaf(old[y], f, o[y]);
                    }
                    folded = m;
                }
                // Exponents c s - m are fused, one rounding: exact enough while a product's own rounding is under one. A
                // row whose reference became larger takes it off the scores first (`taken`; big: some row of the warp).
                float from = nref;
                if (big) {
                    const float base = taken ? m : 0.f;
                    if (taken) from = H::lift;
#pragma unroll
                    for (int y = 0; y < KT; ++y) s[y] -= base;
                }
                // weights: FP32 sums, rounded once to the cache's type for the product with the values
                Two sum[2];
                const auto weights = [&](int h) {  // of 32 keys
                    const Two cc = two(c2, c2), nn = two(from, from);
                    uint32_t u[16];
#pragma unroll
                    for (int y = 0; y < 32; y += 2) {
                        const float2 z = parts(fma2(two(s[h * 32 + y], s[h * 32 + y + 1]), cc, nn));
                        const float p0 = kv_ex2(z.x), p1 = kv_ex2(z.y);
                        sum[y / 2 & 1] = add2(sum[y / 2 & 1], two(p0, p1));
                        u[y / 2] = H::pack(p0, p1);
                    }
                    st16(tm_s + h * 16, u);
                };
                const auto weights_of = [&](int half) {
#pragma unroll
                    for (int h = 0; h < HALF / 32; ++h) weights(half * (HALF / 32) + h);
                };
                sum[0] = sum[1] = 0;
                weights_of(0);
                // A new reference where the maximum has left the old one behind (not for places without a row: what they
                // hold is anything). No weight is larger than their sum: the first half's largest need not be looked for.
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int y = HALF; y < KT; y += 8)
#pragma unroll
                    for (int z = 0; z < 4; ++z) top[z] = max3(top[z], s[y + 2 * z], s[y + 2 * z + 1]);
                const float upper = max3(max3(top[0], top[1], top[2]), top[3], top[3]);
                const float2 half = parts(add2(sum[0], sum[1]));
                const bool need = live && (m == -INFINITY || half.x + half.y > MOST ||
                                           fmaf(upper, c2, from) > kvt::REF_SLACK + H::lift);
                if (__any_sync(FULL_MASK, need)) {
                    float f = 1.f, mx = upper;
#pragma unroll
                    for (int y = 0; y < HALF; y += 2) mx = max3(mx, s[y], s[y + 1]);
                    float shift = 0.f;
                    if (need && mx > (taken ? 0.f : m)) {  // (a row's result depends on no other row)
                        f = m == -INFINITY ? 1.f : kv_ex2((taken ? -mx : m - mx) * c2);
                        m = taken ? m + mx : mx, nref = fmaf(-m, c2, H::lift), l *= f;
                        if (taken) shift = mx;
                    }
                    if (!taken && fabsf(nref) > kvt::FUSED_MOST) taken = true, shift = m;
                    from = taken ? H::lift : nref;
                    if (__any_sync(FULL_MASK, taken)) {
                        big = true;
#pragma unroll
                        for (int y = 0; y < KT; ++y) s[y] -= shift;
                    }
                    if (i % FOLD != 0) {
                        ok = ok && done(n_t - 1, false);
#pragma unroll 1
                        for (int e = 0; e < a.d; e += 8) {
                            float o[8];
                            tc::tmem_ld<8>(tm_o + e, o);
#pragma unroll
                            for (int y = 0; y < 8; ++y) o[y] *= f;
                            tc::tmem_st<8>(tm_o + e, o);
                        }
                    }
                    sum[0] = sum[1] = 0;
                    weights_of(0);
                }
                if (t >= mixed) {
                    // rows of V, a key each: the boxes are shared out over the groups, four pieces of a row at a time
                    ok = ok && warp_wait(&st.v_ok, n_v & 1);
                    ++n_v;
                    const int key = r % KT;
                    const bool dead = t * KT + key >= w.s.len;
#pragma unroll 1
                    for (int b = ok ? g + r / KT : boxes; b < boxes; b += QT * (TILE / KT)) {
                        int stage = st.v_stage + (b >> 1);
                        if (stage >= stages) stage -= v_stages;
                        uint4* row = reinterpret_cast<uint4*>(ring + stage * one_stage + (b & 1) * BOX_BYTES + key * 128);
#pragma unroll 1
                        for (int c0 = 0; c0 < 8; c0 += 4) {  // (piece c ^ lane: an order without bank conflicts)
                            uint4 v[4];
                            bool bad_one = dead;
#pragma unroll
                            for (int y = 0; y < 4; ++y) v[y] = row[(c0 + y) ^ (lane & 7)];
#pragma unroll
                            for (int y = 0; y < 4; ++y) bad_one = bad_one || kvt::has_odd<ST>(v[y]);
                            if (!bad_one) continue;
#pragma unroll 1
                            for (int y = 0; y < 4; ++y) {
                                uint4* at = &row[(c0 + y) ^ (lane & 7)];
                                if (dead) *at = make_uint4(0, 0, 0, 0);
                                else if (kvt::has_odd<ST>(*at)) *at = kvt::clear_odd<ST>(*at), st.odd[side] = 1;
                            }
                        }
                    }
                    __threadfence_block();
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&st.v_clean);
                }
                const auto publish = [&](int half) {
                    st_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&st.p_full[buf][half]);
                };
                publish(0);
                weights_of(1);
                publish(1);
                const float2 all = parts(add2(sum[0], sum[1]));
                l += all.x + all.y;
            }
            if (!ok) break;
            // ------------------------------------------------------------ outputs
            ok = done(n_t - 1, true) && warp_wait(&st.seg_loaded[side], (seg >> 1) & 1);
            if (!ok) break;
            const bool bad = st.bad[side], odd = st.odd[side], whole = w.whole(), fold = n > FOLD;
            const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
            const float back = folded == -INFINITY ? 1.f : kv_ex2((folded - m) * c2);
            const float inv = bad || l == 0.f ? 0.f : 1.f / l;
            const int64_t to = (int64_t)(w.s.first + tok) * a.Hq + w.h * a.G + (x - tok * a.G);
            int64_t to4[4];  // where the rows of this lane's group of four go (-1: nowhere)
#pragma unroll
            for (int y = 0; y < 4; ++y) to4[y] = __shfl_sync(FULL_MASK, live ? to * a.d : -1, (lane & ~3) + y);
            const bool none = inv == 0.f, some_none = __any_sync(FULL_MASK, none);
            float old[32];
            const auto folds = [&](int e) {  // of 32 outputs
#pragma unroll
                for (int y = 0; y < 32; ++y) old[y] = e + y < a.d ? part[(e + y) * PLACES] : 0.f;
            };
            if (fold) folds(0);
#pragma unroll 1
            for (int e = 0; e < a.d; e += 32) {
                float o[32];
                const int cols = min(32, a.d - e);
                tc::tmem_ld<32>(tm_o + e, o);
                if (fold) {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = fmaf(old[y], back, o[y]);
                    if (e + 32 < a.d) folds(e + 32);
                }
                if (!whole) {
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (y < cols) part[(e + y) * PLACES] = bad ? 0.f : o[y];
                    continue;
                }
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] *= inv;
                if (some_none) {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = none ? 0.f : o[y];
                }
                if (vec) {
                    uint4 z[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) z[y] = Store<ST>::pack(o + 8 * y);
                    turn4(z, lane);
                    const int at = e + (lane & 3) * 8;
                    if (at < a.d) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            if (to4[y] >= 0) *reinterpret_cast<uint4*>(static_cast<ST*>(a.out) + to4[y] + at) = z[y];
                    }
                } else if (live) {
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (y < cols) static_cast<ST*>(a.out)[to * a.d + e + y] = H::round(o[y]);
                }
            }
            tc::fence_before();
            if (live) {
                if (!whole) {
                    float* stat = part + (int64_t)PLACES * a.d;
                    stat[0] = m == -INFINITY ? -INFINITY : -nref, stat[PLACES] = bad ? -1.f : l;
                } else if (a.lse) {
                    a.lse[to] = bad || l == 0.f ? -INFINITY : (log2f(l) - nref) * LN2;
                }
            }
            if (odd && !bad) {
                __syncwarp();  // (the row's outputs are other lanes' stores)
                const int from = max(mixed, w.t0) * KT, end = min(last, w.t1 * KT - 1);
                if (live && whole) add_odd<ST>(a, table, w.h, from, end, static_cast<ST*>(a.out) + to * a.d, 1, Store<ST>::code);
                else if (live) add_odd<ST>(a, table, w.h, from, end, part, PLACES, GDN_F32);
            }
            if (tid == 0 && w.t0 == 0 && !whole) kp_border(a, st.scan, w);
            __syncwarp();
            if (lane == 0) mbar_arrive(&st.seg_free[side]);
            ++seg;
        } while (w.next());
        if (!ok && lane == 0) st.stopped = 1, set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
    }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == M_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
    if (st.stopped) refuse_range<QT>(a, st);
}

}  // namespace gdn
