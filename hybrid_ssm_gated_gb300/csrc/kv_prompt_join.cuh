// kv_prompt_join.cuh -- joins the partial results of prompt units that the ranges of
// several CTAs share: with m = max m_c, out = sum_c 2^{m_c - m} O_c / sum_c 2^{m_c - m} l_c.
//
// Bound by latency: a few tens of megabytes at most, read once, in two dependent loads (the
// border's record; maxima, sums and outputs of two parts at a time, over a running
// maximum). So a warp is 32 rows, a lane each, by eight outputs, with few registers, that
// many of them hide each other's waits: 7 us behind 700 tokens of d = 256, 11 behind 152
// CTAs with 256 rows of d = 128 each (40 MB). (Sixteen outputs behind maxima of all parts,
// 96 registers: 29 us there.)
// Maxima are scaled scores rounded to FP32, as the scores of any FP32 softmax: past 2^24
// two parts whose maxima differ are weighed by a difference of numbers in steps of two and
// more, while within a part a row's reference is taken off the unscaled scores first.
#pragma once

#include "kv_prompt.cuh"

namespace gdn {

namespace kpj {

constexpr int NT = 128, MINE = 8, COLS = MINE * (NT / 32);
// Blocks of a border.
__host__ __device__ inline int share(int places, int d) { return places / 32 * ((d + COLS - 1) / COLS); }

}  // namespace kpj

__global__ void __launch_bounds__(kpj::NT, 10) kp_join_kernel(const __grid_constant__ KvArgs a) {
    using namespace kpj;
    const int RB = a.part_rows, cols = (a.d + COLS - 1) / COLS, each = RB / 32 * cols;
    const int c = blockIdx.x / each, x = blockIdx.x - c * each, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = x / cols * 32 + lane, e0 = x % cols * COLS + warp * MINE;  // place in the unit, first output
    const int in_tile = r % a.tile_places, of_unit = r / a.tile_places * a.tile_rows + in_tile;
    kv_grid_wait();
    const KpBorder k = static_cast<const KpBorder*>(a.border)[c];
    if (k.n == 0 || in_tile >= a.tile_rows || of_unit >= k.rows || e0 >= a.d) return;
    const int64_t size = kp_part_floats(RB, a.d), stat = (int64_t)RB * a.d;
    const float* p = a.part + ((int64_t)c * 2 + 1) * size + r;  // (the first part is its CTA's second, the others their CTAs' first)
    const int mine = min(MINE, a.d - e0);
    float m = -INFINITY, l = 0.f, o[MINE] = {};
    bool refused = false;
#pragma unroll 2
    for (int j = 0; j < k.n; ++j, p += j == 1 ? size : 2 * size) {
        const float mj = p[stat], sum = p[stat + RB];
        float x[MINE];
        const float* q = p + (int64_t)e0 * RB;
#pragma unroll
        for (int e = 0; e < MINE; ++e) x[e] = e < mine ? q[e * RB] : 0.f;
        const float top = fmaxf(m, mj), base = top == -INFINITY ? 0.f : top, f = kv_ex2(m - base), g = kv_ex2(mj - base);
        l = fmaf(l, f, sum * g), m = top, refused = refused || sum == -1.f;
#pragma unroll
        for (int e = 0; e < MINE; ++e) o[e] = fmaf(o[e], f, x[e] * g);
    }
    if (refused) l = 0.f;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = k.r0 + of_unit, tok = row / a.G;
    const int64_t to = ((int64_t)k.first + tok) * a.Hq + k.h * a.G + (row - tok * a.G);
#pragma unroll
    for (int e = 0; e < MINE; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
    if (a.d % 8 == 0 && a.dtype != GDN_F32 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0) {
        uint16_t* out = static_cast<uint16_t*>(a.out) + to * a.d + e0;
#pragma unroll
        for (int e = 0; e < MINE; e += 8)
            if (e0 + e < a.d)
                *reinterpret_cast<uint4*>(out + e) =
                    a.dtype == GDN_BF16 ? Store<__nv_bfloat16>::pack(o + e) : Store<__half>::pack(o + e);
    } else {
#pragma unroll
        for (int e = 0; e < MINE; ++e)
            if (e0 + e < a.d) store_elem(a.out, to * a.d + e0 + e, a.dtype, o[e]);
    }
    if (e0 == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

}  // namespace gdn
