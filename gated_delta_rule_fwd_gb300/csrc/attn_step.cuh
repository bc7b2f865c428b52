// What the paged step's kernels share: loads past L1, warp-level products,
// reads of another CTA's shared memory, launches cut into clusters.
#pragma once

#include "attn_internal.cuh"
#include "tc_common.cuh"

namespace lr {

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)),
                 b = __ldg(reinterpret_cast<const float4 *>(p + 4));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

constexpr int kTile = 16;            // keys of a product
constexpr int kMostTiles = 256;      // of a chunk

// D (16x8, fp32) += A (16x16, bf16) B (16x8, bf16), fragments as in the PTX
// m16n8k16 layout (g = lane / 4, t = lane % 4): a = {A[g][2t..], A[g+8][2t..],
// A[g][2t+8..], A[g+8][2t+8..]}, b = {B[2t..][g], B[2t+8..][g]}, d = {D[g][2t],
// D[g][2t+1], D[g+8][2t], D[g+8][2t+1]}.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, two per lane, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Cache rows are read once: past L1.
__device__ __forceinline__ uint4 load_once16(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 load_once8(const void *p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// In a kernel that another one follows early: the follower's CTAs may take the SMs
// that this kernel leaves free.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// In the follower: the kernel before it has ended and what it wrote is there.  Every
// CTA waits, also one that reads nothing of it, so that the follower never ends first.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches a step kernel; cluster: CTAs of a cluster, 1 for none; smem: dynamic bytes;
// early: it may start before the kernel ahead of it has ended (and waits itself).
template <typename... A, typename... B>
inline cudaError_t launch_cut(void (*fn)(A...), unsigned grid, int threads, int cluster, size_t smem,
                              bool early, cudaStream_t stream, const B &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    cfg.attrs = at;
    if (cluster > 1) {
        cudaLaunchAttribute &t = at[cfg.numAttrs++];
        t.id = cudaLaunchAttributeClusterDimension;
        t.val.clusterDim.x = (unsigned)cluster;
        t.val.clusterDim.y = t.val.clusterDim.z = 1;
    }
    if (early) {
        cudaLaunchAttribute &t = at[cfg.numAttrs++];
        t.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        t.val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace lr
