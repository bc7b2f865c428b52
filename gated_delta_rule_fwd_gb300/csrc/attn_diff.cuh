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

// What follows the difference, for the squares' sum of a whole row (2 d channels).  A mean
// that underflows counts as the smallest number there is: a row of zeros stays one, with
// eps 0 too, and a row that is not zero stays finite.
__device__ __forceinline__ float diff_rms(float squares, int d, float eps) {
    const float mean = squares * (0.5f / d) + eps;
    return mean > 0.f ? rsqrtf(mean) : (mean == 0.f ? 0x1.6a09e6p74f : NAN);  // 2^74.5
}

// N channels of a row in a row: one load.
template <int N>
__device__ __forceinline__ void load_run(const __nv_bfloat16 *p, float (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = __bfloat162float(*p);
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 2) w[0] = *reinterpret_cast<const uint32_t *>(p);
        else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 y = unpack2(w[i]);
            x[2 * i] = y.x, x[2 * i + 1] = y.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void load_run(const float *p, float (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = *p;
    } else if constexpr (N == 2) {
        const float2 u = *reinterpret_cast<const float2 *>(p);
        x[0] = u.x, x[1] = u.y;
    } else {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
}

// One map of a row that did not come out finite, by one warp, from what the row sees:
// 32 keys at a time from the newest on, a lane a key for their scores, then all lanes
// over the values, of which four keys are on their way at once.  A running mean, which no
// large value can drive out of range; infinities and NaN are noted channel by channel and
// stand for the channel in the end (attn_rows.cuh has the rules).  A score of NaN or +inf
// makes the row NaN: false.  y[half][i]: channel half d + lane d / 32 + i, of the halves
// (bits) that are asked for.
template <typename E, int D, typename Keys>
__device__ __forceinline__ bool mend_map(const E *q, int map, const Keys &keys, SeenKeys s, ScoreFactor f,
                                         unsigned halves, float (&y)[2][D / 32]) {
    constexpr int PL = D / 32, U = 4;
    constexpr float kMost = 3.402823466e38f;
    const int lane = threadIdx.x & 31;
    unsigned found[2][PL];  // seen in a channel: 1 +inf, 2 -inf, 4 NaN
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < PL; ++i) found[half][i] = 0, y[half][i] = 0.f;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int j0 = s.hi - 1; j0 >= 0; j0 -= 32) {
        if (j0 < s.lo && j0 >= s.s1) j0 = s.s1 - 1;
        const int j = j0 - lane;
        float x = -INFINITY;
        const E *kj, *vj;
        const bool on = j >= 0 && (j >= s.lo || j < s.s1) && keys(map, 0, j, kj, vj);
        if (on) {
            x = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 a = load4(q + c), b = load4(kj + c);
                x += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
            }
            x *= f.sign;
        }
        if (__any_sync(0xffffffffu, !(x < INFINITY))) return false;
        float top = x;
#pragma unroll
        for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        top = fmaxf(top, m);
        // a score of -inf weighs nothing
        const float old = m == -INFINITY ? 0.f : l * ex2((m - top) * f.c), p = x == -INFINITY ? 0.f : ex2((x - top) * f.c);
        m = top;
        l = old + warp_sum(p);
        const float keep = l > 0.f ? old / l : 0.f, take = l > 0.f ? p / l : 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < PL; ++i) y[half][i] *= keep;
        const unsigned some = __ballot_sync(0xffffffffu, on);
#pragma unroll 1
        for (int b = 0; b < 32; b += U) {
            float v[U][2][PL];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const bool read = (some >> (b + u) & 1u) && (halves >> half & 1u) && keys(map, half, j0 - b - u, kj, vj);
#pragma unroll
                    for (int i = 0; i < PL; ++i) v[u][half][i] = 0.f;
                    if (read) load_run<PL>(vj + lane * PL, v[u][half]);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = __shfl_sync(0xffffffffu, take, b + u);
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < PL; ++i) {
                        const float z = v[u][half][i];
                        if (!isfinite(z)) found[half][i] |= z > 0.f ? 1u : (z < 0.f ? 2u : 4u);
                        // a mean of the type's largest values, but for its rounding
                        y[half][i] = fminf(fmaxf(fmaf(w, z, y[half][i]), -kMost), kMost);
                    }
            }
        }
        bool open = false;  // a channel that more keys could still change
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < PL; ++i) open = open || ((halves >> half & 1u) && found[half][i] < 3u);
        if (!__any_sync(0xffffffffu, open)) break;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (found[half][i])
                y[half][i] = found[half][i] == 1u ? INFINITY : (found[half][i] == 2u ? -INFINITY : NAN);
    return true;
}

// A row whose difference is not finite, by one warp, from the definition.  q0, q1: the
// maps' rows; keys(map, half, j, kj, vj): whether key j can be read, its row of k for the
// map and of v for the half; halves: those of the value row (bits) that are wanted without
// the norm.  y[half][i]: the row's channel half d + lane d / 32 + i.
template <typename E, int D, typename Keys>
__device__ __forceinline__ void mend_diff(const E *q0, const E *q1, const Keys &keys, float lambda, bool norm,
                                          const float *weight, float eps, SeenKeys s, ScoreFactor f, unsigned halves,
                                          float (&y)[2][D / 32]) {
    constexpr int PL = D / 32;
    const int lane = threadIdx.x & 31;
    if (norm) halves = 3;
    bool fine = true;
#pragma unroll 1
    for (int map = 0; map < 2 && fine; ++map) {
        float x[2][PL];
        fine = mend_map<E, D>(map ? q1 : q0, map, keys, s, f, halves, x);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < PL; ++i) y[half][i] = map ? y[half][i] - lambda * x[half][i] : x[half][i];
    }
    float sum = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            if (!fine) y[half][i] = NAN;
            sum += y[half][i] * y[half][i];
        }
    if (!norm) return;
    const float r = diff_rms(warp_sum(sum), D, eps);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < PL; ++i)
            y[half][i] = y[half][i] * r * (weight ? weight[half * D + lane * PL + i] : 1.f);
}

}  // namespace lr
