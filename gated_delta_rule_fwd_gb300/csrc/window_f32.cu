// lr_fwd_window in fp32 on warp-level tensor-core products, one pass over the
// keys with the running maximum and sum of the softmax.
//
// Every operand is split into two tf32 parts, x = hi + lo (hi rounded to 11
// significant bits), and a product is taken as hi hi + hi lo + lo hi with fp32
// accumulation: what is left out is 2^-22 of it, so the result is that of fp32
// arithmetic.  Three tf32 products are 100 TFLOP/s on this GPU, the CUDA cores'
// fp32 peak is 74 and in a tiled kernel they are held up by shared memory.
// The products' accumulators are cut, not rounded, so long sums in them drift
// (2e-6 of the output when the whole sum stayed there, 4e-7 now): only a few
// products are summed there and then added in ordinary fp32.
//
// A CTA holds 64 query rows of one head, 16 per warp, in registers; tiles of
// 32 keys and values come by asynchronous copies into two buffers.  At d = 128,
// where registers leave eight warps to an SM, two groups of four warps hold the
// same rows and take every other tile; their parts are joined at the end (8
// heads x 2048 rows, causal: 228 -> 177 us; at d = 64 one group is 6 % faster).
//
// Where the row blocks would leave SMs idle, up to eight CTAs of a cluster share
// one, each a run of its key tiles, and join their parts through distributed
// shared memory (cluster_size; 16 rows of 8 heads on 8192 keys: 680 -> 93 us).
//
// Measured: 4 x 8 heads x 2048 with window 512, d = 64: 160 us, 47 TFLOP/s of
// visible work; the tensor pipe is busy 37 % of the time of an SM that has work.
// What bounds it is the issue of about 1000 instructions per warp and tile, a
// third of them the splitting, by few warps (registers).  At d = 128 all 255
// registers are taken and about 300 bytes a thread spilled: queries and outputs of 16
// rows are 128 of them, and one group of warps with fewer rows was slower.
// The order of channels inside a product, and of keys inside the second one,
// is free: it is chosen so that every lane reads 16 contiguous bytes of a row
// without bank conflicts, and the weights stay in the registers that the
// scores' product left them in.
#include <algorithm>

#include "attn_f32.cuh"
#include "attn_internal.cuh"
#include "attn_join.cuh"
#include "attn_rows.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

__device__ unsigned g_window_error = 0;

constexpr int BQ = 64, BK = kF32Keys, GT = 128;  // GT: threads of a group

template <int D, int G, int DV>
struct Smem {
    static constexpr int KS = F32Rows<D>::KS, VS = F32Rows<DV>::VS;
    struct Group {
        float k[2][BK * KS];
        float v[2][BK * VS];
    } group[G];
    static_assert(G == 1 || sizeof(Group) >= GT * (DV / 2 + 4) * sizeof(float), "room for a group's part");
    static_assert(sizeof(Group) >= BQ * (DV + 2) * sizeof(float), "room for a CTA's part");
};
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(GT) : "memory");
}

// DV: channels of a value row, 2 D where a pair's two value heads are taken together.
template <int D, int G, bool SPLIT, int DV>
__global__ void __launch_bounds__(G * GT) window_f32_kernel(WindowArgs a, float c, float sign, int splits) {
    extern __shared__ __align__(16) uint8_t raw[];
    using S = Smem<D, G, DV>;
    S &sm = *reinterpret_cast<S *>(raw);
    const int group = G == 1 ? 0 : threadIdx.x / GT, tid = threadIdx.x % GT, warp = tid >> 5, lane = tid & 31,
              g = lane >> 2, t = lane & 3;
    typename S::Group &buf = sm.group[group];

    const int tiles = (a.Tq + BQ - 1) / BQ;
    // the last rows see the most keys: of all heads they start first
    const unsigned block = SPLIT ? blockIdx.x / splits : blockIdx.x, rank = SPLIT ? blockIdx.x - block * splits : 0;
    const unsigned heads = (unsigned)(a.B * a.Hq), turn = block / heads, bh = block - turn * heads;
    const int tile = tiles - 1 - (int)turn;
    const int b = bh / a.Hq, h = bh - b * a.Hq;
    int hq = h, hk = h / (a.Hq / a.Hk), hv = hk;
    if (DV > D) hv = 2 * hk, hk = 2 * hk + (h & 1);
    else if (a.pairs) hq = h >> 1, hv = 2 * hk + (h & 1), hk = 2 * hk + (hq & 1);
    bool bad = false;
    const int ql = clamp_len(a.q_len, b, a.Tq, &bad), kl = clamp_len(a.k_len, b, a.Tk, &bad);
    if (bad && threadIdx.x == 0) atomicOr(&g_window_error, kAttnIndex);
    const int i0 = tile * BQ;
    if (i0 >= ql) return;
    const int rows = min(BQ, ql - i0), p0 = kl - ql + i0;
    const float *q = static_cast<const float *>(a.q) + b * a.qs.b + hq * a.qs.h + (long long)i0 * a.qs.t;
    const float *k = static_cast<const float *>(a.k) + b * a.ks.b + hk * a.ks.h;
    const float *v = static_cast<const float *>(a.v) + b * a.vs.b + hv * a.vs.h;
    float *o = static_cast<float *>(a.o) + b * a.os.b + h * a.os.h + (long long)i0 * a.os.t;

    // key tiles: the sinks' before the window of every row, then the window's
    const SeenKeys first = seen_keys(p0, kl, a.window, a.sinks);
    const SeenKeys last = seen_keys(p0 + rows - 1, kl, a.window, a.sinks);
    const int sink_keys = min(last.s1, first.lo), sink_tiles = (sink_keys + BK - 1) / BK;
    const int all = sink_tiles + (last.hi > first.lo ? (last.hi - first.lo + BK - 1) / BK : 0);
    const int begin = SPLIT ? (int)((long long)all * rank / splits) : 0,
              n = SPLIT ? (int)((long long)all * (rank + 1) / splits) : all;
    auto key0 = [&](int it) { return it < sink_tiles ? it * BK : first.lo + (it - sink_tiles) * BK; };
    auto limit = [&](int it) { return it < sink_tiles ? sink_keys : last.hi; };
    // keys and values past the tile's limit are zeros
    auto load = [&](int it) {
        const int k0 = key0(it), end = limit(it);
        const int half = ((it - begin) / G) & 1;
        float *kd = buf.k[half], *vd = buf.v[half];
#pragma unroll
        for (int i = 0; i < BK * D / 4 / GT; ++i) {
            const int e = i * GT + tid, r = e / (D / 4), ch = (e - r * (D / 4)) * 4;
            const bool on = k0 + r < end;
            const long long row = on ? k0 + r : 0;
            copy16(kd + r * S::KS + ch, k + row * a.ks.t + ch, on);
#pragma unroll
            for (int u = 0; u < DV / D; ++u) copy16(vd + r * S::VS + u * D + ch, v + u * a.vs.h + row * a.vs.t + ch, on);
        }
    };
    if (begin + group < n) load(begin + group);
    copies_commit();

    // queries: channels 16 i + 4 t .. + 3 of rows g and g + 8, which are two
    // products' A fragments: (0, 1) and (2, 3) stand for k = t and t + 4
    const int r0 = 16 * warp + g, pw = p0 + 16 * warp;
    float4 qr[D / 16][2];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r0 + 8 * r < rows) x = *reinterpret_cast<const float4 *>(q + (r0 + 8 * r) * a.qs.t + 16 * i + 4 * t);
            qr[i][r] = make_float4(x.x * sign, x.y * sign, x.z * sign, x.w * sign);
        }
    float acc[DV / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DV / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

    for (int it = begin + group; it < n; it += G) {
        if (it + G < n) load(it + G);
        copies_commit();
        copies_wait<1>();
        group_sync(group);
        const int k0 = key0(it), end = limit(it);
        // the warp's rows: positions pw .. pw + 15
        const bool some = k0 <= pw + 15 && ((long long)k0 + BK - 1 > (long long)pw - a.window || k0 < a.sinks);
        if (some) {
            const int half = ((it - begin) / G) & 1;
            const bool whole = k0 + BK <= end && k0 + BK - 1 <= pw && (long long)k0 > (long long)pw + 15 - a.window;
            f32_tile<D, DV>(qr, buf.k[half], buf.v[half], acc, m, l, c, whole, [&](int i, int r) {
                const int key = k0 + i, p = pw + g + 8 * r;
                return key <= p && key < end && (p - key < a.window || key < a.sinks);
            });
        }
        group_sync(group);  // the buffer is free for the tile after next
    }
    copies_wait<0>();
    if constexpr (G == 2) {
        // the second group hands its part over, each lane to its twin
        __syncthreads();
        float *part = reinterpret_cast<float *>(&sm.group[1]);
        if (group == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) part[(2 * r) * GT + tid] = m[r], part[(2 * r + 1) * GT + tid] = l[r];
#pragma unroll
            for (int j = 0; j < DV / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[(4 + 4 * j + e) * GT + tid] = acc[j][e];
        }
        __syncthreads();
        if (!SPLIT && group == 1) return;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float m1 = part[(2 * r) * GT + tid], l1 = part[(2 * r + 1) * GT + tid];
            const float mn = fmaxf(m[r], m1);
            const float f0 = m[r] == -INFINITY ? 0.f : ex2((m[r] - mn) * c), f1 = m1 == -INFINITY ? 0.f : ex2((m1 - mn) * c);
            l[r] = l[r] * f0 + l1 * f1;
            m[r] = mn;
#pragma unroll
            for (int j = 0; j < DV / 8; ++j)
#pragma unroll
                for (int e = 2 * r; e < 2 * r + 2; ++e)
                    acc[j][e] = acc[j][e] * f0 + part[(4 + 4 * j + e) * GT + tid] * f1;
        }
    }
    auto mend = [&](int row, bool sum_finite) {
#pragma unroll 1
        for (int u = 0; u < DV / D; ++u)
            mend_row<float, D>(q + row * a.qs.t, k, v + u * a.vs.h, a.ks.t, a.vs.t, o + row * a.os.t + u * D,
                               seen_keys(p0 + row, kl, a.window, a.sinks), {sign, c}, sum_finite);
    };
    if constexpr (SPLIT) {
        // the part over the first buffers, which no one reads any more
        __syncthreads();
        uint8_t *part = reinterpret_cast<uint8_t *>(&sm.group[0]);
        float2 *stats = reinterpret_cast<float2 *>(part + BQ * DV * 4);
        if (group == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int row = r0 + 8 * r;
                if (t == 0) stats[row] = make_float2(m[r], sum);
#pragma unroll
                for (int i = 0; i < DV / 32; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4 *>(part + part_at<DV>(row, 8 * i + 2 * t + e)) =
                            make_float4(acc[4 * i][2 * r + e], acc[4 * i + 1][2 * r + e],
                                        acc[4 * i + 2][2 * r + e], acc[4 * i + 3][2 * r + e]);
            }
        }
        tc::cluster_sync_all();
        for (int row = (int)rank * (G * 4) + (int)(threadIdx.x >> 5); row < rows; row += splits * (G * 4)) {
            float sum;
            if (join_row<float, DV>(tc::smem_u32(part), tc::smem_u32(stats), row, splits, c, o + row * a.os.t, sum))
                continue;
            mend(row, isfinite(sum));
        }
        tc::cluster_sync_all();  // no CTA leaves while another reads its part
    } else {
        // columns 32 i + 8 t .. + 7 of rows g and g + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float sum = l[r];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key, or only scores of -inf
            const int row = r0 + 8 * r;
            float odd = 0.f;  // NaN once a value is not finite
#pragma unroll
            for (int i = 0; i < DV / 32; ++i) {
                float y[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    y[u] = acc[4 * i + u][2 * r] * inv;
                    y[4 + u] = acc[4 * i + u][2 * r + 1] * inv;
                    odd = fmaf(y[u], 0.f, fmaf(y[4 + u], 0.f, odd));
                }
                if (row < rows) {
                    float *to = o + row * a.os.t + 32 * i + 8 * t;
                    *reinterpret_cast<float4 *>(to) = make_float4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<float4 *>(to + 4) = make_float4(y[4], y[5], y[6], y[7]);
                }
            }
            unsigned again = __ballot_sync(0xffffffffu, row < rows && !(odd == 0.f));
            __syncwarp();
            for (int x = 0; x < 8; ++x) {
                if (!((again >> (4 * x)) & 0xfu)) continue;
                const int rr = 16 * warp + x + 8 * r;
                mend(rr, isfinite(__shfl_sync(0xffffffffu, sum, 4 * x)));
            }
        }
    }
}

// Key tiles that row block i of a sequence without padding needs.
int key_tiles(const WindowArgs &a, int i) {
    const long long p0 = (long long)a.Tk - a.Tq + (long long)i * BQ, p1 = std::min<long long>(p0 + BQ, a.Tk);
    const long long lo = std::max(0ll, p0 - a.window + 1), sinks = std::min<long long>(lo, a.sinks);
    return p1 <= 0 ? 0 : (int)((p1 - lo + BK - 1) / BK + (sinks + BK - 1) / BK);
}

// CTAs that share a row block: what takes the least time, in key tiles of a
// CTA.  The longest block counts, and the rounds of CTAs, each with the mean of
// the blocks' tiles and what a CTA costs besides: `start` is the time of its
// launch and first loads, `join` of joining the parts.  A tile takes 2.7 us at
// d = 128, 1.3 below.
// Measured, one CTA a block and as chosen: 80 blocks of 34 tiles, d = 128: 96
// and 82 us (by 3; by 2, which needs two rounds as well, 108); 1024 rows of 8
// heads, causal: 91 and 57 (by 2; by 3 75); d = 64, 2048 rows of 8 heads: 119
// and 93 (by 2; by 3 97); 512 rows of 32: 34 (alone; by 2 38); 215 rows of 6,
// d = 128: 24 and 13 (by 5); 173 rows of 32, window 64, d = 64: 9.5 (alone; by
// 3 14).  With both value heads of a pair a tile takes 2 us (starts of 3 to 8 tiles
// chose alike but for 173 rows of 16 maps, window 64: 16.6 us alone, 19.5 split).
int cluster_size(const WindowArgs &a, long long ctas, int per_sm, int start, int join) {
    if (ctas > 8 * kClusterRoom[per_sm - 1][1]) return 1;  // the last round hardly counts
    const int blocks = (a.Tq + BQ - 1) / BQ;
    const int longest = key_tiles(a, blocks - 1), mean = key_tiles(a, (blocks - 1) / 2);
    int best = 1;
    float least = 0.f;
    for (int s = 1; s <= kMostCluster && (s == 1 || longest >= s); ++s) {
        const long long room = kClusterRoom[per_sm - 1][s], rounds = (ctas * s + room - 1) / room;
        const float cost = std::max((float)longest / s + start, rounds * ((float)mean / s + start)) + (s > 1 ? join : 0);
        if (s == 1 || cost < least) best = s, least = cost;
    }
    return best;
}

template <int D, int DV = D>
cudaError_t launch(const WindowArgs &a, int slot, cudaStream_t stream) {
    constexpr int G = D == 128 ? 2 : 1, bytes = sizeof(Smem<D, G, DV>);
    const long long ctas = (long long)a.B * a.Hq * ((a.Tq + BQ - 1) / BQ);
    const int splits = D == 128 ? cluster_size(a, ctas, 1, 3, 1) : cluster_size(a, ctas, 2, DV > D ? 5 : 7, DV > D ? 4 : 5);
    auto *fn = splits > 1 ? window_f32_kernel<D, G, true, DV> : window_f32_kernel<D, G, false, DV>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fn), bytes, slot + (splits > 1 ? 12 : 0));
    if (e != cudaSuccess) return e;
    const ScoreFactor f = score_factor(a.scale);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * splits));
    cfg.blockDim = dim3(G * GT);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, a, f.c, f.sign, splits);
}

// ensure_smem_attr slots 208..210, 220..222, 236, 237, 248 and 249
constexpr int kSlot = 208, kPairSlot = 236;

template <typename E>
__global__ void window_zero_kernel(WindowArgs a, int units, long long n) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int u = (int)(i % units);
        long long r = i / units;
        const int t = (int)(r % a.Tq);
        r /= a.Tq;
        const int h = (int)(r % a.Hq), b = (int)(r / a.Hq);
        bool bad = false;
        const int ql = clamp_len(a.q_len, b, a.Tq, &bad);
        clamp_len(a.k_len, b, a.Tk, &bad);
        if (bad) atomicOr(&g_window_error, kAttnIndex);
        if (t < ql)
            *reinterpret_cast<uint4 *>(static_cast<E *>(a.o) + b * a.os.b + h * a.os.h + t * a.os.t +
                                       u * (16 / (int)sizeof(E))) = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace

cudaError_t launch_window_f32(const WindowArgs &a, int d, cudaStream_t stream) {
    if (d == 32) return a.pairs ? launch<32, 64>(a, kPairSlot, stream) : launch<32>(a, kSlot, stream);
    if (d == 64) return a.pairs ? launch<64, 128>(a, kPairSlot + 1, stream) : launch<64>(a, kSlot + 1, stream);
    return launch<128>(a, kSlot + 2, stream);
}

cudaError_t launch_window_zero(const WindowArgs &a, int d, lr_dtype dt, cudaStream_t stream) {
    const int units = d * (dt == LR_DT_F32 ? 4 : 2) / 16;  // 16-byte units of a row
    const long long n = (long long)a.B * a.Hq * a.Tq * units;
    const unsigned grid = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
    if (dt == LR_DT_F32) window_zero_kernel<float><<<grid, 256, 0, stream>>>(a, units, n);
    else window_zero_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, units, n);
    return cudaGetLastError();
}

int attn_errors_window_f32() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_window_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_window_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
