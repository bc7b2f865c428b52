// Attention rows whose keys were shared out over the CTAs of a cluster.  Each
// CTA leaves, in its shared memory, the unnormalised fp32 outputs of its rows,
// [rows][D] with the 16-byte chunks of a row at chunk ^ row (rows are written
// by one thread or a few lanes each), and their (maximum, sum).
#pragma once

#include "attn_internal.cuh"
#include "attn_rows.cuh"
#include "tc_common.cuh"

namespace lr {

// Byte offset of a 16-byte chunk of a row.
template <int D> __device__ __forceinline__ uint32_t part_at(int row, int chunk) {
    return (uint32_t)(row * D * 4 + ((chunk ^ (row & (D / 4 - 1))) * 16));
}

template <int N> __device__ __forceinline__ void ld_cluster(float (&v)[N], uint32_t addr) {
    if constexpr (N == 4)
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(addr)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[0]) : "r"(addr) : "memory");
}

// One row by one warp: joins the parts of `splits` CTAs in their order, writes
// the row to `to`, gives the sum of its weights, and returns whether every
// channel is finite.  part, stats: shared-memory addresses of the outputs and
// of the (maximum, sum) pairs; c: the scores' factor to powers of two.
template <typename E, int D>
__device__ __forceinline__ bool join_row(uint32_t part, uint32_t stats, int row, int splits, float c, E *to,
                                         float &sum) {
    constexpr int N = D / 32;  // channels of a lane
    const int lane = threadIdx.x & 31;
    float ml[2] = {-INFINITY, 0.f};
    if (lane < splits) ld_cluster(ml, tc::map_to_rank(stats + 8 * row, lane));
    float mn = ml[0];
#pragma unroll
    for (int w = 16; w; w >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
    // a part without a key weighs nothing; a sum of NaN stays
    const float f = ml[0] == -INFINITY ? 0.f : ex2((ml[0] - mn) * c);
    sum = warp_sum(f * ml[1]);
    float o[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
    for (int i = 0; i < splits; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        // a part without a key may hold anything; one whose weight underflows
        // still shows an infinite value, as it does in a row that is not split
        if (__shfl_sync(0xffffffffu, ml[0], i) == -INFINITY) continue;
        ld_cluster(v, tc::map_to_rank(part + part_at<D>(row, lane * N / 4) + lane * N % 4 * 4, i));
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += fi * v[e];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key, or only scores of -inf
    bool finite = true;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float y = o[e] * inv;
        finite = finite && isfinite(y);
        to[lane * N + e] = from_f<E>(y);
    }
    finite = __all_sync(0xffffffffu, finite);
    __syncwarp();
    return finite;
}

}  // namespace lr
