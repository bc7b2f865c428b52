// Differential attention: what its kernels share.  A pair of heads has two
// softmax maps over the same keys' positions, each with queries and keys of its
// own, and one value row of 2 d channels, kept as two heads of d:
//
//     y = softmax(s q0 k0) v - lambda softmax(s q1 k1) v,
//     o = weight y / sqrt(mean(y^2) + eps)     where the norm is asked for.
#pragma once

#include "attn_internal.cuh"
#include "attn_rows.cuh"

namespace lr {

// What follows the difference, for the squares' sum of a whole row (2 d
// channels): a row of zeros stays one, with eps 0 too.
__device__ __forceinline__ float diff_rms(float squares, int d, float eps) {
    return squares > 0.f ? rsqrtf(squares * (0.5f / d) + eps) : (squares == 0.f ? 0.f : NAN);
}

// A row whose result is not finite, by one warp: both maps over all 2 d
// channels from the definition (attn_rows.cuh).  q0, q1: the maps' rows;
// keys(map, half, j, kj, vj): whether key j can be read, its row of k for the map
// and of v for the half; fin0, fin1: whether the maps' sums of weights are
// finite.  y[half][i]: the row's channel half d + lane + 32 i.
template <typename E, int D, typename Keys>
__device__ __forceinline__ void mend_diff(const E *q0, const E *q1, const Keys &keys, float lambda, bool norm,
                                          const float *weight, float eps, SeenKeys s, ScoreFactor f, bool fin0,
                                          bool fin1, float (&y)[2][D / 32]) {
    constexpr int PL = D / 32;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int half = 0; half < 2; ++half)
#pragma unroll 1
        for (int map = 0; map < 2; ++map) {
            float x[PL];
            unsigned odd[PL];
#pragma unroll
            for (int i = 0; i < PL; ++i) odd[i] = 1, x[i] = 0.f;
            mend_values<E, D>(
                map ? q1 : q0, [&](int j, const E *&kj, const E *&vj) { return keys(map, half, j, kj, vj); }, x, odd,
                s, f, map ? fin1 : fin0);
#pragma unroll
            for (int i = 0; i < PL; ++i) y[half][i] = map ? y[half][i] - lambda * x[i] : x[i];
        }
    if (!norm) return;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) sum += y[0][i] * y[0][i] + y[1][i] * y[1][i];
    const float r = diff_rms(warp_sum(sum), D, eps);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < PL; ++i)
            y[half][i] = y[half][i] * r * (weight ? weight[half * D + lane + 32 * i] : 1.f);
}

}  // namespace lr
