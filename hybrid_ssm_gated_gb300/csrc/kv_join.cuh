// kv_join.cuh -- joins the partial results of units whose key tiles span CTAs:
// with m = max m_c, out = sum_c 2^{m_c - m} O_c / sum_c 2^{m_c - m} l_c.
//
// Bound by latency: a few megabytes at most, read once, in three dependent loads
// (the border's record; maxima, sums and the first outputs; further outputs). So
// a job is one row's 128 outputs (16 bytes a lane), many small blocks share a
// border, and the code is short: it is fetched once a call. 4 us behind a short
// call, 6 behind 152 CTAs with 64 rows each. (A warp a row with a factor formed
// at every load took 55 us for 32 rows in 7 parts; four jobs a warp in straight
// code 10 us.)
#pragma once

#include "kv_common.cuh"

namespace gdn {

namespace kvj {

constexpr int NT = 128, WARPS = NT / 32;
constexpr int SHARE = 8;  // blocks a border
constexpr int AHEAD = 2;  // parts whose outputs are asked for before the maxima are known

}  // namespace kvj

// Blocks SHARE i .. SHARE i + SHARE - 1 stand at the end of CTA i's range (`parts` is known on the device
// only, so there are blocks for every CTA of the attention kernel but the last); those at a unit's inner
// borders share its jobs.
__global__ void __launch_bounds__(kvj::NT) kv_join_kernel(const __grid_constant__ KvArgs a) {
    using namespace kvj;
    __shared__ float4 sums[WARPS][32];
    const int i = blockIdx.x / SHARE, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    kv_grid_wait();  // the partials are written
    const KvBorder k = static_cast<const KvBorder*>(a.border)[i];
    if (k.rows == 0) return;
    const int RB = a.row_block, rows = k.rows, r0 = k.r0, h = k.h, b = k.b, c0 = k.c0, n = k.n;
    const int64_t size = kv_part_floats(RB, a.d);
    // a unit's partial is the first of a CTA's two, but for the CTA in which it begins after another
    const auto part = [&](int j) { return a.part + ((int64_t)(c0 + j) * 2 + (j == 0 ? k.second : 0)) * size; };
    const bool vec = a.d % 4 == 0;
    const int cols = (a.d + 127) / 128, jobs = rows * cols;
    int team = 1;  // warps a job
    while (team < WARPS && team * 4 < n) team *= 2;
    const int teams = WARPS / team, mine = warp / team, me = warp - mine * team;
    const int rank = (i - c0) * SHARE + blockIdx.x % SHARE, ranks = (n - 1) * SHARE;
    const auto outputs = [&](int j, int r, int e) {
        const float* p = part(j) + (int64_t)r * a.d + e;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec) {
            if (e < a.d) x = *reinterpret_cast<const float4*>(p);
        } else {
            if (e < a.d) x.x = p[0];
            if (e + 1 < a.d) x.y = p[1];
            if (e + 2 < a.d) x.z = p[2];
            if (e + 3 < a.d) x.w = p[3];
        }
        return x;
    };
    const int stride = ranks * teams;
#pragma unroll 1
    for (int first = rank * teams; first < jobs; first += stride) {
        const int job = first + mine;
        const bool live = job < jobs;
        const int r = live ? job / cols : 0, e = live ? (job - r * cols) * 128 + lane * 4 : 0;
        float4 ahead[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x)
            if (me + x * team < n) ahead[x] = outputs(me + x * team, r, e);
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int j = lane; j < n; j += 32) m = fmaxf(m, part(j)[RB * a.d + r]);
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, x));
        const float base = m == -INFINITY ? 0.f : m;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        bool refused = false;
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += 32) {
            float f = 0.f;
            if (j0 + lane < n) {
                const float* p = part(j0 + lane) + (int64_t)RB * a.d + r;
                const float sum = p[RB];
                f = kv_ex2(p[0] - base);
                l += sum * f;
                refused = refused || sum == -1.f;
            }
            const int end = min(32, n - j0);
#pragma unroll 2
            for (int j = me, x = j0 == 0 ? 0 : AHEAD; j < end; j += team, ++x) {
                const float w = __shfl_sync(FULL_MASK, f, j);
                const float4 y = x == 0 ? ahead[0] : x == 1 ? ahead[1] : outputs(j0 + j, r, e);
                o.x = fmaf(y.x, w, o.x), o.y = fmaf(y.y, w, o.y), o.z = fmaf(y.z, w, o.z), o.w = fmaf(y.w, w, o.w);
            }
        }
        l = group_sum<32>(l);
        if (__any_sync(FULL_MASK, refused)) l = 0.f;
        if (team > 1) {
            sums[warp][lane] = o;
            __syncthreads();
            for (int x = 1; x < team && me == 0; ++x) {
                const float4 z = sums[warp + x][lane];
                o.x += z.x, o.y += z.y, o.z += z.z, o.w += z.w;
            }
            __syncthreads();
        }
        if (live && me == 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int node = (r0 + r) / a.G, hq = h * a.G + (r0 + r) - node * a.G;
            const int64_t row = ((int64_t)b * a.T + node) * a.Hq + hq;
            const float z[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (e + x < a.d) store_elem(a.out, row * a.d + e + x, a.dtype, l == 0.f ? 0.f : z[x] * inv);
            if (e == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
        }
    }
}

}  // namespace gdn
