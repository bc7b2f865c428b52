// lr_step_paged_prefix in fp32: the part of a step's attention that lies in the
// prefix shared by the batch.
//
// The query rows of all sequences that read one key head (N times Hq / Hk) are
// worked on as one matrix, 64 rows to a CTA, on the split tf32 products of
// window_f32.cu.  The prefix is cut into runs of 32-key tiles; every CTA leaves
// (maximum, sum, unnormalised output) of its run for its rows, and the step over
// each sequence's own keys joins them (step_paged.cu).
//
// Measured: 33 sequences behind 1501 tokens, window 1024, 20.5 us with their own tokens
// (25.4 when the parts were joined at the end of the own ones); the bound is the issue of
// split products, as in window_f32.cu.
#include <limits.h>

#include "attn_f32.cuh"
#include "attn_internal.cuh"
#include "attn_step.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

__device__ unsigned g_prefix_f32_error = 0;

constexpr int BQ = 64, BK = kF32Keys, NT = 128;

template <int D>
struct Smem {
    float k[2][BK * F32Rows<D>::KS];
    float v[2][BK * F32Rows<D>::VS];
    int page[2][BK / 16];  // of each 16 keys, -1: outside the pool or behind the prefix
};

template <int D>
__global__ void __launch_bounds__(NT) prefix_f32_kernel(StepArgs a, PrefixPlan plan, float c, float sign) {
    using R = F32Rows<D>;
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    let_next_start();
    const int G = a.Hq / a.Hk, rows = a.N * G;
    int id = blockIdx.x;
    const int run = id % plan.parts;
    id /= plan.parts;
    const int hk = id % a.Hk, row0 = id / a.Hk * BQ;
    const int begin = run * plan.chunk, end = min(plan.tiles, begin + plan.chunk);
    auto key0 = [&](int it) { return BK * (it < plan.sink_tiles ? it : it - plan.sink_tiles + plan.first); };

    // the rows' queries and the first key of each one's window; a row that is
    // not computed sees nothing
    const int r0 = row0 + 16 * warp + g;
    int lo[2], head[2];
    float4 qr[D / 16][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = min(r0 + 8 * r, rows - 1), n = row / G, len = a.lens[n];
        const bool on = r0 + 8 * r < rows && len >= 0 && len <= a.max_len;
        lo[r] = on ? window_start(a.plen + len - 1, a.window) : INT_MAX;
        head[r] = on ? n * a.Hq + hk * G + row - n * G : -1;
        const float *q = static_cast<const float *>(a.q) + ((size_t)n * a.Hq + hk * G + row - n * G) * D + 4 * t;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(q + 16 * i);
            qr[i][r] = make_float4(x.x * sign, x.y * sign, x.z * sign, x.w * sign);
        }
    }
    const int lo_most = __reduce_max_sync(0xffffffffu, max(lo[0] == INT_MAX ? 0 : lo[0], lo[1] == INT_MAX ? 0 : lo[1]));
    const int all_sinks = min(a.all_sinks, a.plen);

    auto load = [&](int it) {
        const int k0 = key0(it), half = (it - begin) & 1;
        float *kd = sm.k[half], *vd = sm.v[half];
#pragma unroll
        for (int i = 0; i < BK * D / 4 / NT; ++i) {
            const int e = i * NT + tid, r = e / (D / 4), ch = (e - r * (D / 4)) * 4, key = k0 + r;
            int page = -1;
            if (key < a.plen) {
                page = a.ptable[key >> a.page_log2];
                if (page < 0 || page >= a.num_pages) {
                    if (ch == 0) atomicOr(&g_prefix_f32_error, kAttnIndex);
                    page = -1;
                }
            }
            if ((r & 15) == 0 && ch == 0) sm.page[half][r >> 4] = page;
            const bool on = page >= 0;
            const long long row =
                on ? (((long long)page * a.Hk + hk) << a.page_log2) + (key & ((1 << a.page_log2) - 1)) : 0;
            copy16(kd + r * R::KS + ch, static_cast<const float *>(a.k) + row * D + ch, on);
            copy16(vd + r * R::VS + ch, static_cast<const float *>(a.v) + row * D + ch, on);
        }
    };
    float acc[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    if (begin < end) load(begin);
    copies_commit();
    for (int it = begin; it < end; ++it) {
        if (it + 1 < end) load(it + 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        const int k0 = key0(it), half = (it - begin) & 1;
        const int *page = sm.page[half];
        const bool whole = k0 + BK <= a.plen && (k0 >= lo_most || k0 + BK <= all_sinks) && page[0] >= 0 && page[1] >= 0;
        f32_tile<D>(qr, sm.k[half], sm.v[half], acc, m, l, c, whole, [&](int i, int r) {
            const int key = k0 + i;
            return key < a.plen && (key >= lo[r] || key < all_sinks) && page[i >> 4] >= 0;
        });
        __syncthreads();  // the buffer is free for the tile after next
    }
    copies_wait<0>();
    // columns 32 i + 8 t .. + 7 of rows g and g + 8
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float sum = l[r];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (head[r] < 0) continue;
        const size_t at = (size_t)head[r] * plan.parts + run;
        if (t == 0) a.pml[at] = make_float2(m[r], sum);
        float *to = a.po + at * D + 8 * t;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            *reinterpret_cast<float4 *>(to + 32 * i) = make_float4(acc[4 * i][2 * r], acc[4 * i + 1][2 * r],
                                                                   acc[4 * i + 2][2 * r], acc[4 * i + 3][2 * r]);
            *reinterpret_cast<float4 *>(to + 32 * i + 4) =
                make_float4(acc[4 * i][2 * r + 1], acc[4 * i + 1][2 * r + 1], acc[4 * i + 2][2 * r + 1],
                            acc[4 * i + 3][2 * r + 1]);
        }
    }
}

template <int D>
cudaError_t launch(const StepArgs &a, const PrefixPlan &plan, int slot, cudaStream_t stream) {
    auto *fn = prefix_f32_kernel<D>;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fn), sizeof(Smem<D>), slot);
    if (e != cudaSuccess) return e;
    const long long blocks = ((long long)a.N * (a.Hq / a.Hk) + BQ - 1) / BQ;
    const ScoreFactor f = score_factor(a.scale);
    fn<<<(unsigned)(blocks * a.Hk * plan.parts), NT, sizeof(Smem<D>), stream>>>(a, plan, f.c, f.sign);
    return cudaGetLastError();
}

}  // namespace

// ensure_smem_attr slots 227..229 belong to this file.
cudaError_t launch_prefix_f32(const StepArgs &a, const PrefixPlan &plan, int d, cudaStream_t stream) {
    if (d == 32) return launch<32>(a, plan, 227, stream);
    if (d == 64) return launch<64>(a, plan, 228, stream);
    return launch<128>(a, plan, 229, stream);
}

int attn_errors_prefix_f32() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_prefix_f32_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_prefix_f32_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
