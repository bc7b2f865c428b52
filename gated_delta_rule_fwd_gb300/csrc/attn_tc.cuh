// What the tensor-core attention kernels share: waits, tensor memory written
// from registers, loads of strided rows, and the softmax of a score tile.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "attn_internal.cuh"
#include "tc_common.cuh"

namespace lr {
namespace tc {

// mbar_wait in few instructions: the loop stays a loop.  The kernel has some
// thirty waits, and code that does not fit the instruction cache costs it more
// than anything else it does between two pieces of work.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %3;\n"
        "again_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra done_%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra again_%=;\n"
        "done_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kSpinLimit)
        : "memory");
    return done != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns, written from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}
// The same, 32 columns.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
        "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]),
        "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]),
        "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Tiled TMA load of a 4-D box (x innermost), completion counted on `bar`.
__device__ __forceinline__ void tma_load_4d(void *dst, const void *map, int x, int y, int z, int w,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
// The same of a 5-D box.
__device__ __forceinline__ void tma_load_5d(void *dst, const void *map, int x, int y, int z, int w, int v,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// The tensor pipe for one warp's products at a time: two warps that issue
// together would both finish late, and their softmaxes then run together too,
// with the pipe idle.  A hint for the order, not a lock: two warps may see the
// flag free at once, and after the limit a warp goes on; no result depends on it.
__device__ __forceinline__ void take_pipe(uint32_t *flag) {
    const uint32_t at = smem_u32(flag);
#pragma unroll 1
    for (int i = 0; i < 4096; ++i) {
        uint32_t old;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(old) : "r"(at) : "memory");
        if (!old) break;
    }
    asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(at) : "memory");
}
__device__ __forceinline__ void free_pipe(uint32_t *flag) {
    asm volatile("st.volatile.shared.u32 [%0], 0;" ::"r"(smem_u32(flag)) : "memory");
}
// Register shares of the warpgroups (all four warps execute these).
template <int N> __device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// the lowest n bits (n clipped to 0..32)
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// The bf16 pair nearest to x, and (in `rest`) to what that rounding left.
__device__ __forceinline__ uint32_t pack2_rest(float2 x, uint32_t &rest) {
    const uint32_t r = pack2(x.x, x.y);
    const float2 y = unpack2(r);
    rest = pack2(x.x - y.x, x.y - y.y);
    return r;
}

// One 128-key tile of a row of scores, a row per thread: raises the row's
// maximum m in use where a score passes it by 2^8 (rescaling the sum l and the
// output's DV columns at `to`), replaces the 128 scores at `ts` by bf16 weights
// over their first 64 columns, handing them over in halves (ready0, ready1, one
// arrival a warp), and adds the weights to l.  REST: the other 64 columns take what the
// weights' rounding left, as bf16 weights of their own, handed over with their halves.  A
// weight is 2^(c s - b) with b = c m rounded, so all of a row refer to the same b.
// keep(i): which of the columns 32 i .. 32 i + 31 the row sees; not asked where `whole`.
//
// A tile at the edge of what the rows see gets -inf over the scores that a row
// does not see, in tensor memory, so that one code serves all tiles.
template <int DV, bool REST, typename Keep>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, float c, bool whole, const Keep &keep,
                                             float &m, float &l, uint64_t *ready0, uint64_t *ready1) {
    const float2 c2 = make_float2(c, c);
    const bool lead = (threadIdx.x & 31) == 0;
    if (!whole) {
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
            const uint32_t k = keep(ch);
            if (__all_sync(0xffffffffu, k == 0xffffffffu)) continue;
            float s[32];
            tmem_ld32(ts + 32 * ch, s);
            tmem_ld_wait(s);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!((k >> i) & 1u)) s[i] = -INFINITY;
            tmem_st32(ts + 32 * ch, s);
        }
        tmem_st_wait();
    }
    float s[4][32];
    tmem_ld32(ts, s[0]);
    tmem_ld32(ts + 32, s[1]);
    tmem_ld32(ts + 64, s[2]);
    tmem_ld32(ts + 96, s[3]);
    tmem_ld_wait(s[0], s[1], s[2], s[3]);
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
        for (int i = 0; i < 32; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[ch][i], s[ch][i + 1]);
    const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    const bool grow = mn > m && (m == -INFINITY || (mn - m) * c > 8.f);
    // a row that has seen nothing yet has l = 0 and zeros in the output (or it is unset)
    if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
        // no fma here: both products as the exponent's base has them
        const float f = grow && m != -INFINITY ? ex2(__fsub_rn(__fmul_rn(m, c), __fmul_rn(mn, c))) : 1.f;
        l *= f;
#pragma unroll 1
        for (int ch = 0; ch < DV / 16; ++ch) {
            float v[16];
            tmem_ld16(to + 16 * ch, v);
            tmem_ld_wait(v);
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i] * f);
            tmem_st16(to + 16 * ch, r);
        }
    }
    if (grow) m = mn;
    const float base = m == -INFINITY ? 0.f : -__fmul_rn(m, c);
    const float2 b2 = make_float2(base, base);
    float2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
        uint32_t r[16], rest[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float2 e = fma2(make_float2(s[ch][2 * i], s[ch][2 * i + 1]), c2, b2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[i & 3] = add2(sum[i & 3], e);
            r[i] = REST ? pack2_rest(e, rest[i]) : pack2(e.x, e.y);
        }
        tmem_st16(ts + 16 * ch, r);
        if (REST) tmem_st16(ts + 64 + 16 * ch, rest);
        if (ch & 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lead) mbar_arrive(ch == 1 ? ready0 : ready1);
        }
    }
    const float2 two = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
    l += two.x + two.y;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A strided [B, H, T, d] tensor, boxes of 128 rows x 64 columns, 128-byte
// swizzle, zero fill outside (also the columns of a box wider than d).
inline cudaError_t rows_map(CUtensorMap *m, const void *base, const lr_strides &s, int B, int H, int T, int d) {
    auto enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
    // a dimension of size 1 has stride 0 here: any valid one will do
    auto bytes = [d](long long st) { return (cuuint64_t)(st ? st * 2 : d * 2); };
    const cuuint64_t strides[3] = {bytes(s.t), bytes(s.h), bytes(s.b)};
    const cuuint32_t box[4] = {64, 128, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows of 64-column blocks: element (x, row, block, head, batch) of a strided [B, H,
// T, d] tensor is channel 64 block + x.  A box holds `heads` heads, one behind the
// other, each with all its blocks (or one) of `rows` rows, 128-byte swizzle, zero fill
// of what lies outside (also the columns of a block wider than d), so one copy brings
// a whole tile: a copy costs its issuing thread some 120 cycles whatever its size.
inline cudaError_t blocks_map(CUtensorMap *m, const void *base, const lr_strides &s, int B, int H, int T, int d,
                              int rows, int heads, bool one_block = false) {
    auto enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const int blocks = d > 64 ? 2 : 1;
    const cuuint64_t dims[5] = {(cuuint64_t)(d / blocks), (cuuint64_t)T, (cuuint64_t)blocks, (cuuint64_t)H, (cuuint64_t)B};
    // a dimension of size 1 has stride 0 here: any valid one will do
    auto bytes = [d](long long st) { return (cuuint64_t)(st ? st * 2 : d * 2); };
    const cuuint64_t strides[4] = {bytes(s.t), 128, bytes(s.h), bytes(s.b)};
    const cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)(one_block ? 1 : blocks), (cuuint32_t)heads, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// The same of a pool [pages, H, page, d]: (x, row of the page, block, head, page).
inline cudaError_t pool_map(CUtensorMap *m, const void *pool, int d, int page, int H, int pages, int rows, int heads,
                            bool one_block = false) {
    return blocks_map(m, pool, {(long long)H * page * d, (long long)page * d, d}, pages, H, page, d, rows, heads,
                      one_block);
}

}  // namespace tc
}  // namespace lr
