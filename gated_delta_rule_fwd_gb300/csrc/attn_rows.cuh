// Rows whose result is not finite, put right by a warp.
//
// The tiled kernels multiply whole tiles, where a weight of zero times a NaN
// or an infinity in a masked row of v reaches rows that do not see it.  In all
// kernels a weight that underflows meets an infinity of v as 0 x inf, and the
// unnormalised sum of weights and values may overflow where their mean does
// not.  Such rows come out not finite, and only then is this called (finite
// inputs of ordinary size never are).  What is right for them:
//
//   - a sum of weights that is not finite: where a score that the row sees is
//     NaN or +inf every channel is NaN.  Operands at the type's ends make the
//     sum NaN as well (their split parts, or the maximum times the scale, leave
//     the range; window_tc.cu sets it to NaN where they made it vanish), so the
//     scores are formed once more to tell, 32 keys at a time; if none is NaN or
//     +inf the row is computed again, from differences of unscaled scores;
//   - a channel in which the row sees a NaN, or infinities of both signs, is
//     NaN; one in which it sees infinities of one sign is that infinity (every
//     weight is positive);
//   - any other channel takes its value from finite numbers alone: the row is
//     computed once more from the definition, reading only what it sees.
//
// The search goes back from the newest key and ends as soon as every channel
// is explained, so that a batch full of NaN costs little; the full row is
// computed for rows next to a masked one that is not finite.
#pragma once

#include "attn_internal.cuh"

namespace lr {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// q: the row's d channels; keys(j, kj, vj): whether key j can be read, and its
// rows of k and v.  odd: which of the lane's channels lane + 32 i want a value
// (all of them, on return, where the sum of weights is not finite); y: their
// values.  Every lane of the warp calls this with the same arguments.
template <typename E, int D, typename Keys>
__device__ __forceinline__ void mend_values(const E *q, const Keys &keys, float (&y)[D / 32],
                                            unsigned (&odd)[D / 32], SeenKeys s, ScoreFactor f,
                                            bool sum_finite) {
    constexpr int PL = D / 32;  // channels of a lane: lane + 32 i
    const int lane = threadIdx.x & 31;
    bool whole_row = false;
    if (!sum_finite) {
        bool bad = false;
#pragma unroll 1
        for (int j0 = s.hi - 1; j0 >= 0 && !bad; j0 -= 32) {
            if (j0 < s.lo && j0 >= s.s1) j0 = s.s1 - 1;
            const int j = j0 - lane;
            float x = 0.f;
            const E *kj, *vj;
            if (j >= 0 && (j >= s.lo || j < s.s1) && keys(j, kj, vj)) {
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    const float4 a = load4(q + c), b = load4(kj + c);
                    x += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
                }
            }
            bad = __any_sync(0xffffffffu, !(x * f.sign < INFINITY));
        }
        if (bad) {
#pragma unroll
            for (int i = 0; i < PL; ++i) y[i] = NAN, odd[i] = 1;
            return;
        }
        whole_row = true;
    }
    // seen in a channel: 1 +inf, 2 -inf, 4 NaN
    unsigned found[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        found[i] = 0;
        if (whole_row) odd[i] = 1;
    }
#pragma unroll 1
    for (int j = s.hi - 1; j >= 0; --j) {
        if (j < s.lo && j >= s.s1) {
            j = s.s1;
            continue;
        }
        const E *kj, *vj;
        if (!keys(j, kj, vj)) continue;
        bool open = false;  // a channel that more keys could still change
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const float x = to_f<E>(vj[lane + 32 * i]);
            if (!isfinite(x)) found[i] |= x > 0.f ? 1u : (x < 0.f ? 2u : 4u);
            open = open || (odd[i] && found[i] < 3u);
        }
        if (!__any_sync(0xffffffffu, open)) break;
    }
    bool unexplained = false;
#pragma unroll
    for (int i = 0; i < PL; ++i) unexplained = unexplained || (odd[i] && !found[i]);
    float acc[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) acc[i] = 0.f;
    const bool again = __any_sync(0xffffffffu, unexplained);
    if (again) {
        float qr[PL], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) qr[i] = to_f<E>(q[lane + 32 * i]) * f.sign;
#pragma unroll 1
        for (int j = 0; j < s.hi; ++j) {
            if (j == s.s1 && j < s.lo) j = s.lo;
            if (j >= s.hi) break;
            const E *kj, *vj;
            if (!keys(j, kj, vj)) continue;
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) x += qr[i] * to_f<E>(kj[lane + 32 * i]);
            x = warp_sum(x);
            if (x == -INFINITY) continue;  // weight zero
            // a running mean, which no large value can drive out of range
            const float mn = fmaxf(m, x), old = l * (m == -INFINITY ? 0.f : ex2((m - mn) * f.c)), p = ex2((x - mn) * f.c);
            m = mn;
            l = old + p;
            const float keep = old / l, take = p / l;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const float x = acc[i] * keep + take * to_f<E>(vj[lane + 32 * i]);
                // a mean of the type's largest values, but for its rounding
                acc[i] = fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const float inf = found[i] == 1u ? INFINITY : (found[i] == 2u ? -INFINITY : NAN);
        y[i] = found[i] ? inf : acc[i];
    }
}

// The same for a row o as the kernel left it.
template <typename E, int D, typename Keys>
__device__ __forceinline__ void mend_row_of(const E *q, const Keys &keys, E *o, SeenKeys s, ScoreFactor f,
                                            bool sum_finite) {
    const int lane = threadIdx.x & 31;
    float y[D / 32];
    unsigned odd[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) odd[i] = !isfinite(to_f<E>(o[lane + 32 * i]));
    mend_values<E, D>(q, keys, y, odd, s, f, sum_finite);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        if (odd[i]) o[lane + 32 * i] = from_f<E>(y[i]);
}

// The same with the key head's rows `kt` and `vt` elements apart.
template <typename E, int D>
__device__ __forceinline__ void mend_row(const E *q, const E *k, const E *v, long long kt, long long vt,
                                         E *o, SeenKeys s, ScoreFactor f, bool sum_finite) {
    mend_row_of<E, D>(
        q,
        [&](int j, const E *&kj, const E *&vj) {
            kj = k + j * kt, vj = v + j * vt;
            return true;
        },
        o, s, f, sum_finite);
}

}  // namespace lr
