// kv_prompt_join.cuh -- joins the partial results of prompt units that the ranges of
// several CTAs share: with m = max m_c, out = sum_c 2^{m_c - m} O_c / sum_c 2^{m_c - m} l_c.
#pragma once

#include "kv_prompt.cuh"

namespace gdn {

namespace kpj {
constexpr int NT = 128, WARPS = NT / 32, SHARE = 16;  // blocks a border
}

// Blocks SHARE c .. SHARE c + SHARE - 1 join the unit of CTA c's record. A job is 32 rows (a lane each) by eight
// outputs.
__global__ void __launch_bounds__(kpj::NT) kp_join_kernel(const __grid_constant__ KvArgs a) {
    using namespace kpj;
    const int c = blockIdx.x / SHARE, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    kv_grid_wait();
    const KpBorder k = static_cast<const KpBorder*>(a.border)[c];
    if (k.n == 0) return;
    const int RB = a.part_rows, cols = (a.d + 7) / 8, jobs = RB / 32 * cols;
    const int64_t size = kp_part_floats(RB, a.d);
    const auto part = [&](int j) { return a.part + ((int64_t)(c + j) * 2 + (j == 0)) * size; };
    const bool vec = a.d % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
    for (int x = (blockIdx.x % SHARE) * WARPS + warp; x < jobs; x += SHARE * WARPS) {
        const int g = x / cols, e0 = (x - g * cols) * 8, r = g * 32 + lane;
        const int in_tile = r % a.tile_places, of_unit = r / a.tile_places * a.tile_rows + in_tile;
        if (in_tile >= a.tile_rows || of_unit >= k.rows) continue;
        float m = -INFINITY;
        bool refused = false;
        for (int j = 0; j < k.n; ++j) {
            const float* p = part(j) + (int64_t)RB * a.d + r;
            m = fmaxf(m, p[0]), refused = refused || p[RB] == -1.f;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float o[8] = {}, l = 0.f;
        for (int j = 0; j < k.n; ++j) {
            const float* p = part(j) + r;
            const float f = kv_ex2(p[(int64_t)RB * a.d] - base);
            l = fmaf(p[(int64_t)RB * a.d + RB], f, l);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e0 + e < a.d) o[e] = fmaf(p[(int64_t)(e0 + e) * RB], f, o[e]);
        }
        if (refused) l = 0.f;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int row = k.r0 + of_unit, tok = row / a.G;
        const int64_t to = ((int64_t)k.first + tok) * a.Hq + k.h * a.G + (row - tok * a.G);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
        if (vec && a.dtype != GDN_F32) {
            uint4 w;
            if (a.dtype == GDN_BF16) w = Store<__nv_bfloat16>::pack(o);
            else w = Store<__half>::pack(o);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to * a.d + e0) = w;
        } else {
            for (int e = 0; e < 8; ++e)
                if (e0 + e < a.d) store_elem(a.out, to * a.d + e0 + e, a.dtype, o[e]);
        }
        if (e0 == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
}

}  // namespace gdn
