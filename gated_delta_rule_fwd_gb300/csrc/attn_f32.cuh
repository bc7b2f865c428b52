// What the fp32 attention kernels on warp-level tensor-core products share: the
// split of fp32 values into tf32 parts (window_f32.cu says why) and one tile of
// 32 keys for 16 query rows of a warp.
#pragma once

#include "attn_internal.cuh"
#include "tc_common.cuh"

namespace lr {

constexpr int kF32Keys = 32;  // keys of a tile
// floats of a key's and a value's row in shared memory: see the fragment loads
template <int D> struct F32Rows {
    static constexpr int KS = D + 16, VS = D + 4;
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// x = hi + lo, hi with 11 significant bits (nearest); lo is cut to as many by the
// product.  Infinities and the type's largest values give a NaN: rows that meet
// one are put right afterwards.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
// D (16x8, fp32) += A (16x8, tf32) B (8x8, tf32), fragments as in the PTX
// m16n8k8 layout (g = lane / 4, t = lane % 4): a = {A[g][t], A[g+8][t],
// A[g][t+4], A[g+8][t+4]}, b = {B[t][g], B[t+4][g]}, d = {D[g][2t], D[g][2t+1],
// D[g+8][2t], D[g+8][2t+1]}.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One tile: scores of the warp's rows g and g + 8 (g = lane / 4), their running
// maximum m and sum l (the lane's own columns of it), and the outputs acc.
//   qr      channels 16 i + 4 t .. + 3 of the two rows (t = lane % 4), signed
//   ks, vs  the tile's keys and values, F32Rows floats apart
//   c       the scores' factor to powers of two
//   seen(i, r)  whether row g + 8 r sees key i of the tile; not asked where `whole`
// DV: channels of a value row.
template <int D, int DV = D, typename Seen>
__device__ __forceinline__ void f32_tile(const float4 (&qr)[D / 16][2], const float *ks, const float *vs,
                                         float (&acc)[DV / 8][4], float (&m)[2], float (&l)[2], float c, bool whole,
                                         const Seen &seen) {
    constexpr int BK = kF32Keys;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[BK / 8][4], low[BK / 8][4];  // low: the parts with a lo factor
#pragma unroll
    for (int j = 0; j < BK / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = low[j][e] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t ah[2][4], al[2][4];
        split(qr[i][0].x, ah[0][0], al[0][0]), split(qr[i][1].x, ah[0][1], al[0][1]);
        split(qr[i][0].y, ah[0][2], al[0][2]), split(qr[i][1].y, ah[0][3], al[0][3]);
        split(qr[i][0].z, ah[1][0], al[1][0]), split(qr[i][1].z, ah[1][1], al[1][1]);
        split(qr[i][0].w, ah[1][2], al[1][2]), split(qr[i][1].w, ah[1][3], al[1][3]);
        uint32_t bh_[BK / 8][4], bl[BK / 8][4];
#pragma unroll
        for (int j = 0; j < BK / 8; ++j) {
            const float4 x = *reinterpret_cast<const float4 *>(ks + (8 * j + g) * F32Rows<D>::KS + 16 * i + 4 * t);
            split(x.x, bh_[j][0], bl[j][0]), split(x.y, bh_[j][1], bl[j][1]);
            split(x.z, bh_[j][2], bl[j][2]), split(x.w, bh_[j][3], bl[j][3]);
        }
        float part[BK / 8][4];
#pragma unroll
        for (int j = 0; j < BK / 8; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) part[j][e] = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                mma_tf32(part[j], ah[u], bh_[j][2 * u], bh_[j][2 * u + 1]);
                mma_tf32(low[j], al[u], bh_[j][2 * u], bh_[j][2 * u + 1]);
                mma_tf32(low[j], ah[u], bl[j][2 * u], bl[j][2 * u + 1]);
            }
        }
#pragma unroll
        for (int j = 0; j < BK / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] += part[j][e];
    }
#pragma unroll
    for (int j = 0; j < BK / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] += low[j][e];
    if (!whole) {
#pragma unroll
        for (int j = 0; j < BK / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!seen(8 * j + 2 * t + (e & 1), e >> 1)) s[j][e] = -INFINITY;
    }
    float f[2];  // of what the sums hold, as the maximum grows
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < BK / 8; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * r], s[j][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
        f[r] = m[r] == -INFINITY ? 0.f : ex2((m[r] - base) * c);
        m[r] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < BK / 8; ++j) {
            s[j][2 * r] = ex2((s[j][2 * r] - base) * c);
            s[j][2 * r + 1] = ex2((s[j][2 * r + 1] - base) * c);
            sum += s[j][2 * r] + s[j][2 * r + 1];
        }
        l[r] = l[r] * f[r] + sum;  // this lane's columns; joined at the end
    }
    // weights of keys 8 j + 2 t and + 1 stand for k = t and t + 4
    uint32_t ah[BK / 8][4], al[BK / 8][4];
#pragma unroll
    for (int j = 0; j < BK / 8; ++j) {
        split(s[j][0], ah[j][0], al[j][0]), split(s[j][2], ah[j][1], al[j][1]);
        split(s[j][1], ah[j][2], al[j][2]), split(s[j][3], ah[j][3], al[j][3]);
    }
#pragma unroll
    for (int i = 0; i < DV / 32; ++i) {
        float high[4][4], small[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) high[u][e] = small[u][e] = 0.f;
#pragma unroll
        for (int j = 0; j < BK / 8; ++j) {
            const float4 x = *reinterpret_cast<const float4 *>(vs + (8 * j + 2 * t) * F32Rows<DV>::VS + 32 * i + 4 * g);
            const float4 y = *reinterpret_cast<const float4 *>(vs + (8 * j + 2 * t + 1) * F32Rows<DV>::VS + 32 * i + 4 * g);
            const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t b0h, b0l, b1h, b1l;
                split(xv[u], b0h, b0l), split(yv[u], b1h, b1l);
                mma_tf32(high[u], ah[j], b0h, b1h);
                mma_tf32(small[u], al[j], b0h, b1h);
                mma_tf32(small[u], ah[j], b0l, b1l);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[4 * i + u][e] = fmaf(acc[4 * i + u][e], f[e >> 1], high[u][e] + small[u][e]);
    }
}

}  // namespace lr
