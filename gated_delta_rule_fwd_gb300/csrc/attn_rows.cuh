// One attention row by a warp, straight from the definition: only the keys
// the row sees are read.  The tiled kernels multiply whole tiles, where a
// weight of zero times a NaN or an infinity in a masked row of v would reach
// rows that do not see it; a row whose result is not finite is therefore
// recomputed here (such rows are rare: finite inputs of ordinary size never
// take this path).
#pragma once

#include "attn_internal.cuh"

namespace lr {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// q: the row's d channels; k, v: row 0 of its key head, rows `kt` and `vt`
// elements apart.  Every lane of the warp calls this with the same arguments.
template <typename E, int D>
__device__ __forceinline__ void attn_row(const E *q, const E *k, const E *v, long long kt,
                                         long long vt, E *o, SeenKeys s, float scale) {
    constexpr int PL = D / 32;  // channels of a lane: lane + 32 i
    const int lane = threadIdx.x & 31;
    float qr[PL], acc[PL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        qr[i] = to_f<E>(q[lane + 32 * i]) * scale;
        acc[i] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j < s.hi; ++j) {
        if (j == s.s1 && j < s.lo) j = s.lo;
        if (j >= s.hi) break;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) x += qr[i] * to_f<E>(k[j * kt + lane + 32 * i]);
        x = warp_sum(x);
        if (x == -INFINITY) continue;  // weight zero
        const float mn = x > m || !(x == x) ? x : m;
        const float c = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn);
        m = mn;
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < PL; ++i) acc[i] = acc[i] * c + p * to_f<E>(v[j * vt + lane + 32 * i]);
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
        o[lane + 32 * i] = from_f<E>(m == -INFINITY ? 0.f : acc[i] / l);
}

}  // namespace lr
