// kv_weights_tc.cuh -- accumulation of attention weight per cache entry on the
// tcgen05 tensor cores (16-bit caches, as kv_tc.cuh).
//
// Mathematics. S^T = K Q^T for a tile of 128 keys and NR rows of the accepted
// path (node-major); with the rows' log-sum-exps known, the thread that owns a
// key adds 2^{(scale s - lse) log2 e} over its NR columns and updates the one
// weight it owns: no maximum, no sum across threads, no atomics.
//
// Bound: the keys' bytes (d x 2 a key and head, and 8 for the weight). Paths of up
// to 4 nodes over 64 sequences of up to 8192 entries (32 / 8 heads, d = 128,
// fp16, 0.66 GB): 115 us, 5.8 TB/s or 0.86 of the measured copy bandwidth (FP32
// pipe: 1040 us). Shape:
// persistent, one CTA per SM; one warp loads K tiles by TMA into a ring that
// fills shared memory, one thread issues the MMAs, two groups of four warps
// take tiles in turn, each with a buffer of S^T in tensor memory, so that one
// group's exponentials run beside the other's wait. Paths with more than 128
// rows take their blocks of rows one after another over the CTA's tiles (the
// keys come from L2 then).
#pragma once

#include "kv_tc.cuh"

namespace gdn {

namespace kvw {

using kvt::BOX;
using kvt::BOX_BYTES;
using kvt::KT;
constexpr int NT = 384, GROUPS = 2, SM_WARPS = 4 * GROUPS;
constexpr int K_WARP = SM_WARPS, S_WARP = SM_WARPS + 1;

template <int NR>
struct __align__(16) State {
    float nlse[NR];    // -lse of each row; -inf where the block has none, or its lse is -inf (its weights are 0)
    int64_t q_at[NR];  // element offset of each row's query
    uint64_t full[kvt::MAX_STAGES], empty[kvt::MAX_STAGES];
    uint64_t s_full[2], s_empty[2], q_full, q_empty, drain;
    KvScan<NT> scan;
    uint32_t tmem;
#ifdef GDN_TEST_STALL
    uint64_t never;
#endif
};

// Barrier of the eight weight warps.
__device__ __forceinline__ void all_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ bool any_of(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

template <int NR>
__host__ __device__ constexpr int smem_bytes(int boxes, int stages) {
    return 1024 + boxes * NR * 128 + stages * (boxes > 1 ? 2 : 1) * BOX_BYTES + (int)sizeof(State<NR>);
}

}  // namespace kvw

template <typename ST, int NR>
__global__ void __launch_bounds__(kvw::NT, 1)
    kv_weights_tc_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ CUtensorMap map, const int boxes,
                         const int stages, const int box_rows) {
    using namespace kvw;
    using kvt::desc;
    using H = kvt::Half16<ST>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int pairs = (boxes + 1) >> 1, stage_bytes = (boxes > 1 ? 2 : 1) * BOX_BYTES;
    unsigned char* sQ = smem;
    unsigned char* ring = smem + boxes * NR * 128;
    State<NR>& st = *reinterpret_cast<State<NR>*>(ring + stages * stage_bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr uint32_t TM_COLS = 2 * NR < 32 ? 32 : 2 * NR;

    if (warp == K_WARP) {
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
        if (lane < stages) mbar_init(&st.full[lane], 1), mbar_init(&st.empty[lane], 1);
        if (lane < 2) mbar_init(&st.s_full[lane], 1), mbar_init(&st.s_empty[lane], 4);
        if (lane == 2) mbar_init(&st.q_full, SM_WARPS), mbar_init(&st.q_empty, 1), mbar_init(&st.drain, 1);
#ifdef GDN_TEST_STALL
        if (lane == 3) mbar_init(&st.never, 1);
#endif
        fence_barrier_init();
    }
    if (warp == S_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&st.tmem)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before();
    const KvSplit split = kv_locate<false, KT, NT>(a, st.scan, gridDim.x, 1);
    tc::fence_after();
    const uint32_t tmem = st.tmem;
    bool busy;
    KvWalk<false, KT> w(a, split, st.scan, busy);

    if (warp == K_WARP && busy) {
        // ------------------------------------------------------------ loads
        int stage = 0;
        uint32_t round = 0;
        bool ok = true;
        const int per_tile = KT / box_rows, step_pages = KT / a.page_size, step_places = KT - step_pages * a.page_size;
        do {
            const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
            const int blocks = (w.s.nodes * a.G + NR - 1) / NR;
#pragma unroll 1
            for (int rb = 0; rb < blocks && ok; ++rb) {
                int e = w.t0 * KT + lane * box_rows, pg = e / a.page_size, place = e - pg * a.page_size;
                const auto look = [&]() { return lane < per_tile && e < w.s.len ? table[pg] : 0; };
                int page = look();
#pragma unroll 1
                for (int t = w.t0; t < w.t1 && ok; ++t) {
                    const int used = (min(KT, w.s.len - t * KT) + box_rows - 1) / box_rows;  // boxes with an entry
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
                        unsigned char* dst = ring + stage * stage_bytes + lane * box_rows * 128;
                        if (lane == 0) mbar_arrive_expect_tx(full, used * box_rows * 128 * nb);
                        __syncwarp();
                        if (lane < used) {
                            kvt::tma_load(dst, &map, 2 * p * BOX, this_place, w.h, this_page, full);
                            if (nb > 1)
                                kvt::tma_load(dst + BOX_BYTES, &map, (2 * p + 1) * BOX, this_place, w.h, this_page, full);
                        }
                        if (++stage == stages) stage = 0, ++round;
                    }
                }
            }
        } while (ok && w.next());
        if (!ok && lane == 0) set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
        kvt::landed(st.full, 0, stages, stage, round);
    } else if (warp == S_WARP && busy) {
        // ------------------------------------------------------------ MMAs
        const uint32_t id = kvt::idesc(H::type, false, false, NR);
        const uint32_t aQ = smem_addr(sQ), aR = smem_addr(ring), tm = kvt::uniform(tmem);
        int stage = 0;
        uint32_t round = 0, n_t = 0, seg = 0;
        bool ok = true;
        do {
            const int blocks = kvt::uniform((w.s.nodes * a.G + NR - 1) / NR), n = kvt::uniform(w.t1 - w.t0);
#pragma unroll 1
            for (int rb = 0; rb < blocks && ok; ++rb) {
                ok = kvt::warp_wait(&st.q_full, seg & 1);
                ++seg;
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i, ++n_t) {
                    const int buf = n_t & 1;
                    if (n_t >= 2) ok = kvt::warp_wait(&st.s_empty[buf], ((n_t >> 1) - 1) & 1);
#pragma unroll 1
                    for (int p = 0; p < pairs && ok; ++p) {
                        ok = kvt::warp_wait(&st.full[stage], round & 1);
                        if (!ok) break;
                        tc::fence_after();
                        const uint64_t da = desc(aR + stage * stage_bytes, 16, 1024, kvt::SW128),
                                       db = desc(aQ + 2 * p * NR * 128, 16, 1024, kvt::SW128);
#pragma unroll
                        for (int k = 0; k < BOX / 16; ++k)
                            kvt::mma(tm + buf * NR, da + k * (32 >> 4), db + k * (32 >> 4), id, p + k > 0);
                        if (boxes - 2 * p > 1) {
#pragma unroll
                            for (int k = 0; k < BOX / 16; ++k)
                                kvt::mma(tm + buf * NR, da + (BOX_BYTES >> 4) + k * (32 >> 4),
                                         db + (NR * 128 >> 4) + k * (32 >> 4), id, true);
                        }
                        kvt::commit(&st.empty[stage]);
                        if (++stage == stages) stage = 0, ++round;
                    }
                    if (ok) kvt::commit(&st.s_full[buf]);
                }
                if (ok) kvt::commit(&st.q_empty);  // the queries are read
            }
        } while (ok && w.next());
        if (!ok && lane == 0) set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
        kvt::commit(&st.drain);  // products in flight end before tensor memory is freed, whoever gave up
        mbar_wait(&st.drain, 0);
        __syncwarp();
    } else if (warp < SM_WARPS && busy) {
        // ------------------------------------------------------------ weights
        const int g = warp >> 2, quad = warp & 3, key = quad * 32 + lane, wt = tid & 255;
        const uint32_t tm_s = tmem + ((uint32_t)(quad * 32) << 16) + g * NR;
        const kvt::Two log2e = kvt::two(LOG2E, LOG2E);
        uint32_t n_t = 0, seg = 0;
        int checked = -1;
        // A warp whose wait ran out takes part in the barriers and in nothing else: it neither frees a buffer
        // nor hands over queries, so that the other roles' waits run out too and no weight is formed from a
        // product that nobody waited for.
        bool good = true, failed = false;
        do {
            const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
            const int rows_all = w.s.nodes * a.G, blocks = (rows_all + NR - 1) / NR;
            if (checked != w.b) {  // the path's nodes and the sequence's pages are in range
                int bad = kv_pages_ok(a, w.s, wt, 256) ? 0 : KV_DEVERR_PAGE;
                if (wt < w.s.nodes && (uint32_t)a.path[(int64_t)w.b * a.P + wt] >= (uint32_t)a.T) bad |= KV_DEVERR_NODES;
                if (bad) set_error(a.dev_err, bad);
                good = !any_of(bad != 0);
                checked = w.b;
            }
#pragma unroll 1
            for (int rb = 0; rb < blocks; ++rb, ++seg) {
                // ---- row tables and queries, once the last block's are read
                if (seg > 0) failed = failed || !kvt::warp_wait(&st.q_empty, (seg - 1) & 1);
                all_sync();  // nobody reads the last block's table any more
                const int rows = min(NR, rows_all - rb * NR);
                if (wt < NR) {
                    const int r = rb * NR + min(wt, rows - 1), j = r / a.G, hq = w.h * a.G + r - j * a.G;
                    const int node = good ? a.path[(int64_t)w.b * a.P + j] : 0;
                    const float lse = a.lse_in[((int64_t)w.b * a.T + node) * a.Hq + hq];
                    st.nlse[wt] = wt < rows && lse != -INFINITY ? -lse : -INFINITY;
                    st.q_at[wt] = (int64_t)w.b * a.q.seq + (int64_t)node * a.q.node + (int64_t)hq * a.q.head;
                }
                all_sync();
                constexpr int N = (NR * 8 + 255) / 256;
                for (int x = 0; x < boxes && !failed; ++x) {
                    uint4 v[N];
#pragma unroll
                    for (int y = 0; y < N; ++y) {
                        const int i = wt + y * 256, r = i >> 3, e = x * BOX + (i & 7) * 8;
                        v[y] = make_uint4(0, 0, 0, 0);
                        if (i < NR * 8 && r < rows && e < a.d)
                            v[y] = *reinterpret_cast<const uint4*>(static_cast<const ST*>(a.q.p) + st.q_at[r] + e);
                    }
#pragma unroll
                    for (int y = 0; y < N; ++y) {
                        const int i = wt + y * 256, r = i >> 3;
                        if (i < NR * 8)
                            *reinterpret_cast<uint4*>(sQ + x * NR * 128 + r * 128 + (((i & 7) ^ (r & 7)) << 4)) = v[y];
                    }
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0 && !failed) mbar_arrive(&st.q_full);
                // ---- this group's tiles
#pragma unroll 1
                for (int t = w.t0; t < w.t1; ++t, ++n_t) {
                    if ((int)(n_t & 1) != g) continue;
                    const int e = t * KT + key, pg = e / a.page_size;
                    const bool live = e < w.s.len && good;
                    float* x = a.weights;
                    float old = 0.f;
                    if (live) {
                        x += ((int64_t)table[pg] * a.Hkv + w.h) * a.page_size + (e - pg * a.page_size);
                        old = *x;
                    }
                    // rows of nodes before entry e's own do not see it
                    const int unseen = max(0, e - (w.s.len - w.s.nodes)) * a.G - rb * NR;
                    failed = failed || !kvt::warp_wait(&st.s_full[g], (n_t >> 1) & 1);
#ifdef GDN_TEST_STALL
                    if (blockIdx.x == gridDim.x / 2 && g == 0 && n_t == 2) failed = failed || !kvt::warp_wait(&st.never, 0);
#endif
                    if (failed) continue;
                    tc::fence_after();
                    // Columns that add nothing (past the block's rows, or of a row without a log-sum-exp) do so by
                    // their exponent of -inf. That is 0 for every finite score; a score that is not (0 x inf for
                    // the zero queries of a column without a row) makes it NaN, and the sum with it. So a sum that
                    // is NaN is formed again with those columns selected away, and no other needs the selection.
                    kvt::Two sum;
                    float total;
                    bool select = false;
                    while (true) {
                        sum = 0;
#pragma unroll 1
                        for (int r = 0; r < NR; r += 16) {
                            float s[16];
                            tc::tmem_ld<16>(tm_s + r, s);
#pragma unroll
                            for (int y = 0; y < 16; y += 4) {
                                const float4 m = *reinterpret_cast<const float4*>(&st.nlse[r + y]);
                                // the exponent is formed before it is scaled to base 2: a weight near one keeps a
                                // small one
                                const float x0 = fmaf(s[y], a.scale, m.x), x1 = fmaf(s[y + 1], a.scale, m.y);
                                const float x2 = fmaf(s[y + 2], a.scale, m.z), x3 = fmaf(s[y + 3], a.scale, m.w);
                                float2 u = kvt::parts(kvt::mul2(kvt::two(x0, x1), log2e));
                                float2 v = kvt::parts(kvt::mul2(kvt::two(x2, x3), log2e));
                                u = make_float2(kv_ex2(u.x), kv_ex2(u.y)), v = make_float2(kv_ex2(v.x), kv_ex2(v.y));
                                if (unseen > 0 || select) {
                                    if (r + y < unseen || m.x == -INFINITY) u.x = 0.f;
                                    if (r + y + 1 < unseen || m.y == -INFINITY) u.y = 0.f;
                                    if (r + y + 2 < unseen || m.z == -INFINITY) v.x = 0.f;
                                    if (r + y + 3 < unseen || m.w == -INFINITY) v.y = 0.f;
                                }
                                sum = kvt::add2(sum, kvt::add2(kvt::two(u.x, u.y), kvt::two(v.x, v.y)));
                            }
                        }
                        total = kvt::parts(sum).x + kvt::parts(sum).y;
                        if (select || !__any_sync(FULL_MASK, live && total != total)) break;
                        select = true;
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&st.s_empty[g]);
                    if (live) *x = fmaf(old, rb == 0 ? a.decay : 1.f, total);
                }
            }
        } while (w.next());
        if (failed && lane == 0) set_error(a.dev_err, GDN_DEVERR_TIMEOUT);
    } else if (warp == SM_WARPS + 2) {
        for (int b = blockIdx.x + lane * gridDim.x; b < a.B; b += 32 * gridDim.x) {
            const KvSeq s = a.B <= NT ? st.scan.seq[b] : kv_seq<false>(a, b);
            if (s.err) set_error(a.dev_err, s.err);
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == S_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
}

}  // namespace gdn
