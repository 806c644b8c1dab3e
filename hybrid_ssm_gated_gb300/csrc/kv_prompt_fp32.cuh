// kv_prompt_fp32.cuh -- causal attention of packed prompts over the paged cache on
// the FP32 pipe: any cache dtype, head size up to 256, page size and stride. It
// serves fp32 caches, whose scores and outputs keep FP32 products, and 16-bit caches
// that the tensor-core kernel's copies cannot address.
//
// Mathematics. One pass over the keys with a running maximum m and sum l a row
// (base-2 exponents); a tile's products with the values are summed by themselves and
// then added to the rescaled outputs, so that long sums are not rounded to the steps
// of what they have become.
//
// Shape: 128 threads, units of 64 rows, tiles of 64 keys, queries, keys, values and
// weights in shared memory as FP32. Threads form a 16 x 8 grid: eight rows by four
// keys of the scores, then the same eight rows by four outputs (of each 64 of d; by one
// of up to 16 that are left over), so that a row's maximum, sum and rescaling stay with
// its 16 threads. The keys of the
// next tile are on their way (cp.async where the cache is FP32 and its rows allow
// 16-byte copies) while weights and outputs form, the values while scores form.
// Bound by latency at two warps a scheduler (199 registers and 82 KB at d = 80: two CTAs
// a SM): 47% of issue slots, 34% of the FP32 pipe and 38% of shared memory's are used; for
// each instruction that it issues a warp waits 0.74 cycles for shared-memory loads, 0.56
// for its last instruction and 0.32 for the next one's code. Three prompts of up to 1200 rows (8 / 4 heads, d = 80, 3.4
// GFLOP) take 176 us, 19 TFLOP/s, where four rows by four keys of 256 threads took 192;
// 2000 tokens take 164 us at d = 64, 249 at 96, 343 at 128, 748 at 256 (22 to 25 TFLOP/s).
// What 16-bit caches that TMA cannot address cost: 1200 tokens of 8 / 4 heads, d = 128,
// 166 us in pages of 4 entries and 22 on the tensor cores in pages of 16. (255 registers
// from d = 81 on; above 208 they spill 176 bytes.)
#pragma once

#include "kv_attn.cuh"
#include "kv_prompt.cuh"

namespace gdn {

namespace kpg {

constexpr int RB = 64, KT = 64, NT = 128, R = 8;  // R: rows of a thread

struct Layout {
    int dp, pitch, off_k, off_v, off_p, off_at, off_q_at, off_scan, off_bad, bytes;
};
__host__ __device__ inline Layout layout(int d) {
    Layout L;
    L.dp = align_up(d, 4);
    L.pitch = L.dp + 4;  // the threads of a 16-byte load's phase meet distinct banks
    L.off_k = RB * L.pitch * 4;
    L.off_v = L.off_k + KT * L.pitch * 4;
    L.off_p = L.off_v + KT * L.pitch * 4;
    L.off_at = L.off_p + RB * (KT + 4) * 4;
    L.off_q_at = L.off_at + 2 * 2 * KT * 8;
    L.off_scan = L.off_q_at + RB * 8;
    L.off_bad = L.off_scan + (int)sizeof(KpScan<NT, NT>);
    L.bytes = L.off_bad + 16;
    return L;
}

}  // namespace kpg

// NC: blocks of 64 outputs; TAIL: and up to 16 more.
template <typename ST, int NC, bool TAIL>
__global__ void __launch_bounds__(kpg::NT) kv_prompt_kernel(const __grid_constant__ KvArgs a, const int vec) {
    using namespace kpg;
    extern __shared__ __align__(128) unsigned char smem[];
    const Layout L = layout(a.d);
    float* sQ = reinterpret_cast<float*>(smem);
    float* sK = reinterpret_cast<float*>(smem + L.off_k);
    float* sV = reinterpret_cast<float*>(smem + L.off_v);
    float* sP = reinterpret_cast<float*>(smem + L.off_p);
    int64_t(*s_at)[2][KT] = reinterpret_cast<int64_t(*)[2][KT]>(smem + L.off_at);  // [buffer][k, v]: rows of a tile
    int64_t* s_q = reinterpret_cast<int64_t*>(smem + L.off_q_at);
    KpScan<NT, NT>& sc = *reinterpret_cast<KpScan<NT, NT>*>(smem + L.off_scan);
    int& s_bad = *reinterpret_cast<int*>(smem + L.off_bad);  // a page of the segment lies outside the pool
    constexpr int PP = KT + 4;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, pitch = L.pitch, d4 = L.dp / 4;
    const float c2 = a.scale * LOG2E;
    kv_grid_launch();
    kp_locate<KT>(a, sc);
    bool busy;
    KpWalk<KT> w(a, sc, busy);
    kp_empty_rows(a, a.B <= NT ? sc.seq : nullptr, tid, NT);
    if (tid == 0) kp_no_border(a);
    if (!busy) return;
    do {
        const int rows = w.rows(), r0 = w.r0(), prefix = w.s.len - w.s.n, top = min(w.s.len, w.nt * KT);
        const int32_t* table = a.page_table + (int64_t)w.s.slot * a.max_pages;
        __syncthreads();  // the last segment's reads of shared memory
        if (tid == 0) s_bad = 0;
        if (tid < RB) {
            const int x = r0 + min(tid, rows - 1), tok = x / a.G;
            s_q[tid] = (int64_t)(w.s.first + tok) * a.q.node + (int64_t)(w.h * a.G + x - tok * a.G) * a.q.head;
        }
        __syncthreads();
        const auto look = [&](int t) {  // the rows of tile t, by 64 threads
            if (tid < KT) {
                const int e = t * KT + tid;
                int64_t k = 0, v = 0;
                if (t < w.t1 && e < w.s.len) {
                    const int pg = e / a.page_size, page = table[pg];
                    if ((uint32_t)page >= (uint64_t)a.num_pages) s_bad = 1;
                    else k = kv_at(a.k, page, w.h, e - pg * a.page_size), v = kv_at(a.v, page, w.h, e - pg * a.page_size);
                }
                s_at[t & 1][0][tid] = k, s_at[t & 1][1][tid] = v;
            }
        };
        const auto load = [&](float* dst, const KvPages& from, int t, int side) {
            const int64_t* at = s_at[t & 1][side];
            const int n = s_bad ? 0 : min(KT, top - t * KT);  // (a pool without a page has no row to read)
            kv_load_rows<ST, NT>(dst, pitch, L.dp, KT, n, from.p, a.d, vec, [&](int r) { return at[r]; });
            cp_async_commit();
        };
        look(w.t0);
        kv_load_rows<ST, NT>(sQ, pitch, L.dp, RB, rows, a.q.p, a.d, vec, [&](int r) { return s_q[r]; });
        cp_async_commit();
        __syncthreads();
        load(sK, a.k, w.t0, 0);
        load(sV, a.v, w.t0, 1);
        look(w.t0 + 1);
        int last[R];  // each row's last entry
        float m[R], l[R], o[NC > 0 ? NC : 1][R][4], ot[TAIL ? R : 1];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int x = r0 + min(ty * R + i, rows - 1);
            last[i] = prefix + x / a.G, m[i] = -INFINITY, l[i] = 0.f;
            if (TAIL) ot[i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][i][e] = 0.f;
        }
        const int first_last = prefix + r0 / a.G;  // the first row's
        for (int t = w.t0; t < w.t1; ++t) {
            cp_async_wait<1>();
            __syncthreads();
            float s[R][4] = {};
#pragma unroll 2
            for (int e = 0; e < d4; ++e) {
                float4 q[R], k[4];
#pragma unroll
                for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4*>(sQ + (ty * R + i) * pitch + e * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * pitch + e * 4);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) kv_dot4(s[i][j], q[i], k[j]);
            }
            float f[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float top_s = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = t * KT + tx + 16 * j <= last[i] ? s[i][j] * c2 : -INFINITY;
                    top_s = fmaxf(top_s, s[i][j]);
                }
#pragma unroll
                for (int x = 8; x; x >>= 1) top_s = fmaxf(top_s, __shfl_xor_sync(FULL_MASK, top_s, x));
                const float mn = fmaxf(m[i], top_s), base = mn == -INFINITY ? 0.f : mn;
                f[i] = kv_ex2(m[i] - base), m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = kv_ex2(s[i][j] - base), sum += s[i][j];
                    sP[(ty * R + i) * PP + tx + 16 * j] = s[i][j];
                }
#pragma unroll
                for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, x);
                l[i] = fmaf(l[i], f[i], sum);
            }
            __syncthreads();  // the keys are read, the weights written
            if (t + 1 < w.t1) load(sK, a.k, t + 1, 0);
            else cp_async_commit();
            cp_async_wait<1>();
            // Values of entries that a row does not see must not reach it, not even as 0 x infinity: where one is
            // not finite in a tile that some row sees a part of, weights of unseen entries are left out.
            bool odd = false;
            if (t * KT + KT - 1 > first_last) {
                __syncthreads();
                for (int i = tid; i < KT * L.dp; i += NT) {
                    const int r = i / L.dp;
                    odd = odd || !isfinite(sV[r * pitch + i - r * L.dp]);
                }
                odd = __syncthreads_or(odd);
            } else {
                __syncthreads();
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int e = c * 64 + tx * 4;
                float acc[R][4] = {};
                if (e < L.dp) {
                    if (!odd) {
#pragma unroll 2
                        for (int k = 0; k < KT; k += 4) {
                            float4 p[R];
#pragma unroll
                            for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(sP + (ty * R + i) * PP + k);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float4 v = *reinterpret_cast<const float4*>(sV + (k + y) * pitch + e);
#pragma unroll
                                for (int i = 0; i < R; ++i) {
                                    const float x = y == 0 ? p[i].x : y == 1 ? p[i].y : y == 2 ? p[i].z : p[i].w;
                                    acc[i][0] = fmaf(x, v.x, acc[i][0]), acc[i][1] = fmaf(x, v.y, acc[i][1]);
                                    acc[i][2] = fmaf(x, v.z, acc[i][2]), acc[i][3] = fmaf(x, v.w, acc[i][3]);
                                }
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int k = 0; k < KT; ++k) {
                            const float4 v = *reinterpret_cast<const float4*>(sV + k * pitch + e);
#pragma unroll
                            for (int i = 0; i < R; ++i) {
                                if (t * KT + k > last[i]) continue;
                                const float x = sP[(ty * R + i) * PP + k];
                                acc[i][0] = fmaf(x, v.x, acc[i][0]), acc[i][1] = fmaf(x, v.y, acc[i][1]);
                                acc[i][2] = fmaf(x, v.z, acc[i][2]), acc[i][3] = fmaf(x, v.w, acc[i][3]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[c][i][y] = fmaf(o[c][i][y], f[i], acc[i][y]);
            }
            if constexpr (TAIL) {
                float acc[R] = {};
                const int e = NC * 64 + tx;
                if (e < L.dp) {
                    if (!odd) {
#pragma unroll 2
                        for (int k = 0; k < KT; k += 4) {
                            float v[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) v[y] = sV[(k + y) * pitch + e];
#pragma unroll
                            for (int i = 0; i < R; ++i) {
                                const float4 p = *reinterpret_cast<const float4*>(sP + (ty * R + i) * PP + k);
                                acc[i] = fmaf(p.x, v[0], fmaf(p.y, v[1], fmaf(p.z, v[2], fmaf(p.w, v[3], acc[i]))));
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int k = 0; k < KT; ++k)
#pragma unroll
                            for (int i = 0; i < R; ++i)
                                if (t * KT + k <= last[i]) acc[i] = fmaf(sP[(ty * R + i) * PP + k], sV[k * pitch + e], acc[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i) ot[i] = fmaf(ot[i], f[i], acc[i]);
            }
            __syncthreads();  // values and weights are read
            if (t + 1 < w.t1) load(sV, a.v, t + 1, 1);
            else cp_async_commit();
            look(t + 2);
        }
        __syncthreads();
        const bool bad = s_bad, whole = w.whole();
        float* part = a.part + ((int64_t)blockIdx.x * 2 + w.later()) * kp_part_floats(RB, a.d);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = ty * R + i;
            if (r >= rows) break;
            const bool none = bad || l[i] == 0.f;
            const float inv = none ? 0.f : 1.f / l[i];
            const int x = r0 + r, tok = x / a.G;
            const int64_t to = (int64_t)(w.s.first + tok) * a.Hq + w.h * a.G + (x - tok * a.G);
            const auto put = [&](int e, float v) {
                if (e >= a.d) return;
                if (whole) store_elem(a.out, to * a.d + e, Store<ST>::code, none ? 0.f : v * inv);
                else part[(int64_t)e * RB + r] = v;
            };
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int y = 0; y < 4; ++y) put(c * 64 + tx * 4 + y, o[c][i][y]);
            if (TAIL) put(NC * 64 + tx, ot[i]);
            if (tx != 0) continue;
            if (!whole) part[RB * a.d + r] = m[i], part[RB * a.d + RB + r] = bad ? -1.f : l[i];
            else if (a.lse) a.lse[to] = none ? -INFINITY : (m[i] + log2f(l[i])) * LN2;
        }
        if (tid == 0) {
            if (bad) set_error(a.dev_err, KV_DEVERR_PAGE);
            if (w.t0 == 0 && !whole) kp_border(a, sc, w);
        }
    } while (w.next());
}

}  // namespace gdn
