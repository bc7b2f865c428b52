// lr_step_paged: attention of one new token per sequence over a paged cache.
//
// The keys that a sequence sees (its sinks, then its window) form one list,
// cut into chunks.  One CTA takes one chunk of one sequence and key head for
// the query heads that share it, so a chunk's keys and values are read once
// for them.  With one chunk per sequence the CTA writes the output.  A few
// chunks of a small call are the CTAs of a thread-block cluster, which join
// their parts through distributed shared memory in the same launch.  Otherwise
// each CTA writes (maximum, sum, unnormalised output) to the workspace and a
// second kernel joins the chunks in order.  The bound is the read of the cache.
//
// bf16 (step_mma_kernel): warp-level products.  A warp takes 16 keys at a
// time, S^T = K Q^T (16 keys x 8 heads) and O^T += V^T P^T, with keys and
// values loaded from global memory straight into the fragments: the order of
// the channels inside a product is free, so each lane loads 16 contiguous
// bytes of a row; value pairs along the keys are made with byte permutes.  No
// shared memory and no barrier stand between a load and its product, and the
// next keys are on their way while the values of the last ones are used.
//
// Measured: 128 sequences of 500 to 8192 tokens, 32 heads on 8, 351 us (95 % of
// the copy bandwidth); two caches of 131K 82 us (96 %).
//
// fp32 (step_simt_kernel): CUDA cores.  Every group of d / 8 lanes takes keys
// of its own, with a running maximum and sum of its own (33 sequences with
// window 1024, 139 MB: 24.2 us).  With up to two heads on a key head it reads
// the cache at the copy rate; more heads cost instructions, and more than four
// are parts that read the cache again (32 sequences of 4096, 4 key heads, d =
// 128, 537 MB: 81 us with 1 head on each, 84 with 2, 147 with 4, 205 with 8, 324
// with 16).  bf16 takes up to 16 heads in one read (268 MB: 60 us with 1, 63 with
// 8, 68 with 16, 124 with 32).
//
// Rows that come out not finite are explained or computed again from the keys
// they see (attn_rows.cuh), as in the window form; one vote of the CTA that
// writes a row finds them.
#include "attn_internal.cuh"
#include "attn_rows.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

__device__ unsigned g_step_error = 0;

constexpr int NT = 128;

// fp32 partial results in the workspace: [N * Hq][splits][d], then
// (maximum, sum) [N * Hq][splits].
struct Parts {
    float *o;
    float2 *ml;
    int splits, chunk;
    bool cluster;  // the chunks of a row are the CTAs of a cluster
};

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}

// Rows of a sequence that is not computed.
template <typename E, int D>
__device__ __forceinline__ void zero_rows(const StepArgs &a, int n, int h0, int heads) {
    E *o = static_cast<E *>(a.o) + ((size_t)n * a.Hq + h0) * D;
    for (int i = threadIdx.x; i < heads * D; i += NT) o[i] = from_f<E>(0.f);
}

// Output row `head` of sequence n by one warp, put right where it is not
// finite.  sum(): of its weights.  Keys of pages outside the pool are left out.
template <typename E, int D, typename Sum>
__device__ __forceinline__ void mend_step_row(const StepArgs &a, int n, int head, ScoreFactor f, Sum sum) {
    const int lane = threadIdx.x & 31, hk = head / (a.Hq / a.Hk), len = a.lens[n];
    const size_t at = ((size_t)n * a.Hq + head) * D;
    E *o = static_cast<E *>(a.o) + at;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) odd = odd || !isfinite(to_f<E>(o[lane + 32 * i]));
    if (!__any_sync(0xffffffffu, odd)) return;
    const int *table = a.table + (size_t)n * a.max_pages;
    mend_row_of<E, D>(
        static_cast<const E *>(a.q) + at,
        [&](int j, const E *&kj, const E *&vj) {
            const int page = table[j >> a.page_log2];
            if (page < 0 || page >= a.num_pages) return false;
            const long long row = (((long long)page * a.Hk + hk) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
            kj = static_cast<const E *>(a.k) + row * D, vj = static_cast<const E *>(a.v) + row * D;
            return true;
        },
        o, seen_keys(len - 1, len, a.window, a.sinks), f, isfinite(sum()));
}

// The end of a CTA: joins its warps' parts and hands the result on.  so: the
// warps' unnormalised outputs, P floats a head; sml: their (maximum, sum); f:
// the scores' factor; n, h0: sequence and first head.  A part without a key has
// a maximum of -inf and weighs nothing; one whose scores were all NaN too, but
// its sum of NaN stays.
template <typename E, int D, int HEADS, int P>
__device__ __forceinline__ void finish(float (&so)[NT / 32][HEADS][P], float (&sml)[NT / 32][HEADS][2],
                                       int heads, int n, int h0, int split, ScoreFactor f, const StepArgs &a,
                                       const Parts &parts) {
    const int tid = threadIdx.x;
    const size_t row0 = (size_t)n * a.Hq + h0;
    const float c = f.c;
    E *out = static_cast<E *>(a.o);
    bool odd = false;  // a value that is not finite
    __syncthreads();
    for (int i = tid; i < heads * D; i += NT) {
        const int h = i / D, ch = i - h * D;
        float mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) mn = fmaxf(mn, sml[w][h][0]);
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const float mw = sml[w][h][0], fw = mw == -INFINITY ? 0.f : ex2((mw - mn) * c);
            sum += fw * sml[w][h][1];
            x += fw * so[w][h][ch];
        }
        const size_t r = row0 + h;
        if (parts.splits == 1) {
            const float y = sum == 0.f ? 0.f : x / sum;
            out[r * D + ch] = from_f<E>(y);
            odd = odd || !isfinite(y);
        } else if (parts.cluster) {
            so[0][h][ch] = x;  // read and written by this thread alone
        } else {
            parts.o[(r * parts.splits + split) * D + ch] = x;
            if (ch == 0) parts.ml[r * parts.splits + split] = make_float2(mn, sum);
        }
    }
    // the warps' parts of a head as one
    auto whole = [&](int h, float &mn) {
        float sum = 0.f;
        mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) mn = fmaxf(mn, sml[w][h][0]);
#pragma unroll
        for (int w = 0; w < NT / 32; ++w)
            sum += sml[w][h][1] * (sml[w][h][0] == -INFINITY ? 0.f : ex2((sml[w][h][0] - mn) * c));
        return sum;
    };
    if (!parts.cluster) {
        if (parts.splits == 1 && __syncthreads_or(odd))
            for (int h = tid >> 5; h < heads; h += NT / 32)
                mend_step_row<E, D>(a, n, h0 + h, f, [&] {
                    float mn;
                    return whole(h, mn);
                });
        return;
    }
    __syncthreads();
    if (tid < heads) {
        float mn;
        const float sum = whole(tid, mn);
        sml[0][tid][0] = mn, sml[0][tid][1] = sum;
    }
    tc::cluster_sync_all();
    const uint32_t o_at = tc::smem_u32(&so[0][0][0]), ml_at = tc::smem_u32(&sml[0][0][0]);
    for (int i = split * NT + tid; i < heads * D; i += parts.splits * NT) {
        const int h = i / D, ch = i - h * D;
        float m[kMostCluster], mn = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r) {
            m[r] = r < parts.splits ? ld_cluster(tc::map_to_rank(ml_at + 8 * h, r)) : -INFINITY;
            mn = fmaxf(mn, m[r]);
        }
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r)
            if (r < parts.splits) {
                const float fr = m[r] == -INFINITY ? 0.f : ex2((m[r] - mn) * c);
                sum += fr * ld_cluster(tc::map_to_rank(ml_at + 8 * h + 4, r));
                x += fr * ld_cluster(tc::map_to_rank(o_at + 4 * (h * P + ch), r));
            }
        const float y = sum == 0.f ? 0.f : x / sum;
        out[(row0 + h) * D + ch] = from_f<E>(y);
        odd = odd || !isfinite(y);
        if (ch == 0) sml[1][h][1] = sum;  // only the first pair is read by other CTAs
    }
    const int again = __syncthreads_or(odd);
    tc::cluster_sync_all();  // no CTA leaves while another reads its part
    if (again)
        for (int h = tid >> 5; h < heads; h += NT / 32)
            if (h * D / NT % parts.splits == split)  // a row that was written here
                mend_step_row<E, D>(a, n, h0 + h, f, [&] { return sml[1][h][1]; });
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)),
                 b = __ldg(reinterpret_cast<const float4 *>(p + 4));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <int D, int GC>
__global__ void __launch_bounds__(NT) step_simt_kernel(StepArgs a, Parts parts, ScoreFactor f) {
    constexpr int LANES = D / 8;            // lanes of a key
    constexpr int GROUPS = NT / LANES;      // keys in flight
    constexpr int U = 4;                    // keys of a group per pass
    __shared__ float so[GROUPS / (32 / LANES)][GC][D];
    __shared__ float sml[GROUPS / (32 / LANES)][GC][2];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int G = a.Hq / a.Hk, gq = (G + GC - 1) / GC;
    int id = blockIdx.x;
    const int split = id % parts.splits;
    id /= parts.splits;
    const int gi = id % gq;
    id /= gq;
    const int hk = id % a.Hk, n = id / a.Hk;
    const int len = a.lens[n];
    const int h0 = hk * G + gi * GC, heads = min(GC, G - gi * GC);
    if (len < 0 || len > a.max_len) {
        if (len > 0 && tid == 0 && split == 0 && gi == 0 && hk == 0) atomicOr(&g_step_error, kAttnIndex);
        if (a.fill && split == 0) zero_rows<float, D>(a, n, h0, heads);
        return;
    }
    const SeenKeys s = seen_keys(len - 1, len, a.window, a.sinks);
    const int seen = s.s1 + s.hi - s.lo;
    const int c0 = split * parts.chunk;
    if (c0 >= seen && split > 0 && !parts.cluster) return;  // the join knows how many chunks there are
    const int c1 = min(seen, c0 + parts.chunk);
    const int lane = tid % LANES, group = tid / LANES, ch = lane * 8;

    const float *qn = static_cast<const float *>(a.q) + (size_t)n * a.Hq * D;
    float q[GC][8], acc[GC][8], m[GC], l[GC];
#pragma unroll
    for (int g = 0; g < GC; ++g) {
        load8(qn + (size_t)(h0 + min(g, heads - 1)) * D + ch, q[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[g][i] *= f.sign, acc[g][i] = 0.f;
        m[g] = -INFINITY, l[g] = 0.f;
    }
    const int *table = a.table + (size_t)n * a.max_pages;
    const int in_page = (1 << a.page_log2) - 1;
    const int lanes0 = (tid & 31) / LANES * LANES;
    const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << lanes0;
    bool bad = false;
    for (int base = c0 + group; base < c1; base += GROUPS * U) {
        long long row[U];
        float x[U][8], y[U][8], sc[U][GC];  // keys, values: all on their way at once
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * GROUPS;
            row[u] = -1;
            if (i < c1) {
                const int key = i < s.s1 ? i : i - s.s1 + s.lo;
                const int page = table[key >> a.page_log2];
                if (page >= 0 && page < a.num_pages)
                    row[u] = ((((long long)page * a.Hk + hk) << a.page_log2) + (key & in_page)) * D + ch;
                else
                    bad = true;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = y[u][i] = 0.f;
            if (row[u] >= 0) {
                load8(static_cast<const float *>(a.k) + row[u], x[u]);
                load8(static_cast<const float *>(a.v) + row[u], y[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) t += q[g][i] * x[u][i];
#pragma unroll
                for (int w = 1; w < LANES; w <<= 1) t += __shfl_xor_sync(mask, t, w);
                sc[u][g] = row[u] >= 0 ? t : -INFINITY;
            }
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            float mn = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) mn = fmaxf(mn, sc[u][g]);
            const float b = mn == -INFINITY ? 0.f : mn;
            const float c = ex2((m[g] - b) * f.c);
            m[g] = mn;
            l[g] *= c;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[g][i] *= c;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p = ex2((sc[u][g] - b) * f.c);
                l[g] += p;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[g][i] += p * y[u][i];
            }
        }
    }
    if (bad) atomicOr(&g_step_error, kAttnIndex);
    __syncwarp();
    // the groups of a warp, then the warps
#pragma unroll
    for (int g = 0; g < GC; ++g) {
        float mn = m[g];
#pragma unroll
        for (int w = LANES; w < 32; w <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
        const float c = m[g] == -INFINITY ? 0.f : ex2((m[g] - mn) * f.c);
        l[g] *= c;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[g][i] *= c;
#pragma unroll
        for (int w = LANES; w < 32; w <<= 1) {
            l[g] += __shfl_xor_sync(0xffffffffu, l[g], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[g][i] += __shfl_xor_sync(0xffffffffu, acc[g][i], w);
        }
        if ((tid & 31) < LANES) {
#pragma unroll
            for (int i = 0; i < 8; ++i) so[warp][g][ch + i] = acc[g][i];
            if (lane == 0) sml[warp][g][0] = mn, sml[warp][g][1] = l[g];
        }
    }
    finish<float, D, GC, D>(so, sml, heads, n, h0, split, f, a, parts);
}

// ------------------------------------------------------------------- bf16

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

// NH: 8-head column blocks of the products.
template <int D, int NH>
__global__ void __launch_bounds__(NT)
    step_mma_kernel(StepArgs a, Parts parts, ScoreFactor f) {
    const float c = f.c;
    const __nv_bfloat162 sign = __float2bfloat162_rn(f.sign);
    auto with_sign = [&](uint32_t x) {  // exact: 1, -1 or 0 times a pair
        const __nv_bfloat162 y = __hmul2(reinterpret_cast<const __nv_bfloat162 &>(x), sign);
        return reinterpret_cast<const uint32_t &>(y);
    };
    constexpr int KC = D / 32;   // 32-channel pieces of a key: 16 bytes per lane and row
    constexpr int VW = D / 16;   // words of a value row per lane = 16-channel blocks of O^T
    constexpr int HEADS = 8 * NH;
    __shared__ float so[NT / 32][HEADS][D + 8];
    __shared__ float sml[NT / 32][HEADS][2];
    __shared__ long long rows[kMostTiles];  // first cache row of each tile, -1: a bad page
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = a.Hq / a.Hk, gq = (G + HEADS - 1) / HEADS;
    int id = blockIdx.x;
    const int split = id % parts.splits;
    id /= parts.splits;
    const int gi = id % gq;
    id /= gq;
    const int hk = id % a.Hk, n = id / a.Hk;
    const int len = a.lens[n];
    const int h0 = hk * G + gi * HEADS, heads = min(HEADS, G - gi * HEADS);
    if (len < 0 || len > a.max_len) {
        if (len > 0 && tid == 0 && split == 0 && gi == 0 && hk == 0) atomicOr(&g_step_error, kAttnIndex);
        if (a.fill && split == 0) zero_rows<__nv_bfloat16, D>(a, n, h0, heads);
        return;
    }
    const SeenKeys s = seen_keys(len - 1, len, a.window, a.sinks);
    const int sink_tiles = (s.s1 + kTile - 1) / kTile;
    const int k_first = max(s.lo / kTile, sink_tiles);  // a tile that holds both is a sink tile
    const int tiles = sink_tiles + max(0, (s.hi + kTile - 1) / kTile - k_first);
    const int per = parts.chunk / kTile, t0 = split * per, t1 = min(tiles, t0 + per);
    if (t0 >= tiles && split > 0 && !parts.cluster) return;  // the join knows how many chunks there are

    auto key_of = [&](int i) { return kTile * (i < sink_tiles ? i : i - sink_tiles + k_first); };
    for (int i = tid; i < t1 - t0; i += NT) {
        const int key = key_of(t0 + i);
        const int page = a.table[(size_t)n * a.max_pages + (key >> a.page_log2)];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok) atomicOr(&g_step_error, kAttnIndex);
        rows[i] = ok ? (((long long)page * a.Hk + hk) << a.page_log2) + (key & ((1 << a.page_log2) - 1)) : -1;
    }

    // queries: head g of each block, the channels that the lane's keys hold
    uint32_t q[NH][2 * KC][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const bool live = 8 * nh + g < heads;
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.q) +
                                 ((size_t)n * a.Hq + h0 + (live ? 8 * nh + g : 0)) * D + 8 * t;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *reinterpret_cast<const uint4 *>(p + 32 * i);
            q[nh][2 * i][0] = with_sign(x.x), q[nh][2 * i][1] = with_sign(x.y);
            q[nh][2 * i + 1][0] = with_sign(x.z), q[nh][2 * i + 1][1] = with_sign(x.w);
        }
    }
    __syncthreads();

    float acc[VW][NH][4], m[NH][2], l[NH][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        m[nh][0] = m[nh][1] = -INFINITY;
        l[nh][0] = l[nh][1] = 0.f;
#pragma unroll
        for (int j = 0; j < VW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][nh][i] = 0.f;
    }
    uint4 kr[2][KC];        // keys g and g + 8
    uint32_t vr[4][VW];     // values of keys 2t, 2t+1, 2t+8, 2t+9
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.k),
                        *vp = static_cast<const __nv_bfloat16 *>(a.v);
    // Rows that the sequence does not see are not read: zeros.
    auto sees = [&](int key) { return key < s.hi && (key >= s.lo || key < s.s1); };
    auto load_k = [&](int i) {
        const long long row = rows[i - t0];
        const int key = key_of(i);
        const bool all = row >= 0 && sees(key) && sees(key + kTile - 1) && (key >= s.lo || key + kTile <= s.s1);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool on = all || (row >= 0 && sees(key + g + 8 * r));
            const __nv_bfloat16 *p = kp + (row + g + 8 * r) * D + 8 * t;
#pragma unroll
            for (int i2 = 0; i2 < KC; ++i2) {
                kr[r][i2] = make_uint4(0, 0, 0, 0);
                if (on) kr[r][i2] = load_once16(p + 32 * i2);
            }
        }
    };
    auto load_v = [&](int i) {
        const long long row = rows[i - t0];
        const int key = key_of(i);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int kk = 2 * t + (r & 1) + 8 * (r >> 1);
            const bool on = row >= 0 && sees(key + kk);
            const __nv_bfloat16 *p = vp + (row + kk) * D;
#pragma unroll
            for (int w = 0; w < VW; ++w) vr[r][w] = 0u;
            if (on) {
                if (D == 32) {
                    const uint2 x = load_once8(p + 4 * g);
                    vr[r][0] = x.x, vr[r][1] = x.y;
                } else {
#pragma unroll
                    for (int w = 0; w < VW / 4; ++w) {
                        const uint4 x = load_once16(p + 64 * w + 8 * g);
                        vr[r][4 * w] = x.x, vr[r][4 * w + 1] = x.y, vr[r][4 * w + 2] = x.z,
                                   vr[r][4 * w + 3] = x.w;
                    }
                }
            }
        }
    };

    const int first = t0 + warp;
    if (first < t1) {
        load_k(first);
        load_v(first);
    }
    for (int i = first; i < t1; i += NT / 32) {
        float sc[NH][4];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nh][e] = 0.f;
#pragma unroll
            for (int i2 = 0; i2 < KC; ++i2) {
                mma16816(sc[nh], kr[0][i2].x, kr[1][i2].x, kr[0][i2].y, kr[1][i2].y, q[nh][2 * i2][0],
                         q[nh][2 * i2][1]);
                mma16816(sc[nh], kr[0][i2].z, kr[1][i2].z, kr[0][i2].w, kr[1][i2].w,
                         q[nh][2 * i2 + 1][0], q[nh][2 * i2 + 1][1]);
            }
        }
        const bool page_ok = rows[i - t0] >= 0;
        const int key = key_of(i);
        const bool see0 = page_ok && sees(key + g), see1 = page_ok && sees(key + g + 8);
        const int next = i + NT / 32;
        if (next < t1) load_k(next);
        bool grow = false;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = (e < 2 ? see0 : see1) ? sc[nh][e] : -INFINITY, y = m[nh][e & 1];
                sc[nh][e] = x;
                grow = grow || (x > y && !((x - y) * c <= 8.f));
            }
        // the maximum in use is raised only when a score passes it by 2^8
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(sc[nh][e], sc[nh][e + 2]);
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                    const float mn = fmaxf(m[nh][e], mx);
                    const float less = m[nh][e] == -INFINITY ? 0.f : ex2((m[nh][e] - mn) * c);
                    m[nh][e] = mn;
                    // nothing seen yet: sums and output are zero (or NaN, which stays)
                    l[nh][e] *= less;
#pragma unroll
                    for (int j = 0; j < VW; ++j) acc[j][nh][e] *= less, acc[j][nh][e + 2] *= less;
                }
        }
        uint32_t p[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const float b0 = m[nh][0] == -INFINITY ? 0.f : m[nh][0], b1 = m[nh][1] == -INFINITY ? 0.f : m[nh][1];
            // differences first: a product of one large score would overflow
            const float e0 = ex2((sc[nh][0] - b0) * c), e1 = ex2((sc[nh][1] - b1) * c),
                        e2 = ex2((sc[nh][2] - b0) * c), e3 = ex2((sc[nh][3] - b1) * c);
            l[nh][0] += e0 + e2;
            l[nh][1] += e1 + e3;
            p[nh][0] = transpose8x8(pack2(e0, e1));
            p[nh][1] = transpose8x8(pack2(e2, e3));
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            const uint32_t a0 = __byte_perm(vr[0][j], vr[1][j], 0x5410), a1 = __byte_perm(vr[0][j], vr[1][j], 0x7632),
                           a2 = __byte_perm(vr[2][j], vr[3][j], 0x5410), a3 = __byte_perm(vr[2][j], vr[3][j], 0x7632);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma16816(acc[j][nh], a0, a1, a2, a3, p[nh][0], p[nh][1]);
        }
        if (next < t1) load_v(next);
    }
    // this warp's part: word j of a lane holds channels col_j and col_j + 1
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[nh][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int h = 8 * nh + 2 * t + e;
            if (g == 0) sml[warp][h][0] = m[nh][e], sml[warp][h][1] = sum;
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const int col = D == 32 ? 4 * g + 2 * j : 64 * (j >> 2) + 8 * g + 2 * (j & 3);
                *reinterpret_cast<float2 *>(&so[warp][h][col]) = make_float2(acc[j][nh][e], acc[j][nh][e + 2]);
            }
        }
    finish<__nv_bfloat16, D, HEADS, D + 8>(so, sml, heads, n, h0, split, f, a, parts);
}

// One CTA of D threads per output row: the chunks' parts in order.
template <typename E, int D>
__global__ void __launch_bounds__(D) step_join_kernel(StepArgs a, Parts parts, ScoreFactor factor) {
    const float c = factor.c;
    const int r = blockIdx.x, n = r / a.Hq, ch = threadIdx.x;
    const int len = a.lens[n];
    if (len < 0 || len > a.max_len) return;
    const SeenKeys s = seen_keys(len - 1, len, a.window, a.sinks);
    int seen = s.s1 + s.hi - s.lo;
    if (sizeof(E) == 2) {  // whole tiles of 16 keys (step_mma_kernel)
        const int sink_tiles = (s.s1 + kTile - 1) / kTile, k_first = max(s.lo / kTile, sink_tiles);
        seen = kTile * (sink_tiles + max(0, (s.hi + kTile - 1) / kTile - k_first));
    }
    const int used = max(1, (seen + parts.chunk - 1) / parts.chunk);
    const float2 *ml = parts.ml + (size_t)r * parts.splits;
    const float *po = parts.o + (size_t)r * parts.splits * D + ch;
    float m = -INFINITY, l = 0.f, x = 0.f;
    for (int i0 = 0; i0 < used; i0 += 8) {
        float2 t[8];
        float y[8], mn = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] = i0 + i < used ? ml[i0 + i] : make_float2(-INFINITY, 0.f);
            y[i] = i0 + i < used ? po[(size_t)(i0 + i) * D] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mn = fmaxf(mn, t[i].x);
        const float f = m == -INFINITY ? 0.f : ex2((m - mn) * c);
        l *= f;
        x *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // a part without a key weighs nothing; one whose scores were all
            // NaN has no maximum either, but a sum of NaN
            const float w = t[i].x == -INFINITY ? 0.f : ex2((t[i].x - mn) * c);
            l += t[i].y * w;
            x += y[i] * w;
        }
        m = mn;
    }
    const float out = l == 0.f ? 0.f : x / l;
    static_cast<E *>(a.o)[(size_t)r * D + ch] = from_f<E>(out);
    if (__syncthreads_or(!isfinite(out)) && ch < 32)
        mend_step_row<E, D>(a, n, r - n * a.Hq, factor, [&] { return l; });
}

Parts parts_of(const StepArgs &a, int d, const StepPlan &p, void *ws) {
    Parts r{};
    r.splits = p.splits, r.chunk = p.chunk, r.cluster = p.cluster;
    if (p.splits > 1 && !p.cluster) {
        r.o = static_cast<float *>(ws);
        r.ml = reinterpret_cast<float2 *>(r.o + (size_t)a.N * a.Hq * p.splits * d);
    }
    return r;
}

// Query heads that a CTA takes, of G that share a key head.
int heads_of_cta(int G, lr_dtype dt) {
    if (dt == LR_DT_BF16) return G <= 8 ? 8 : 16;
    return G == 1 ? 1 : G == 2 ? 2 : 4;
}

// Launches a step kernel, its chunks as clusters where the plan says so.
cudaError_t launch_parts(void (*fn)(StepArgs, Parts, ScoreFactor), unsigned grid, cudaStream_t stream,
                         const StepArgs &a, const Parts &parts, ScoreFactor f) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(NT);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    if (parts.cluster) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)parts.splits;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, fn, a, parts, f);
}

template <int D>
cudaError_t launch_f32(const StepArgs &a, const Parts &parts, cudaStream_t stream) {
    const int G = a.Hq / a.Hk;
    const int gc = heads_of_cta(G, LR_DT_F32);
    const unsigned grid = (unsigned)(a.N * a.Hk * ((G + gc - 1) / gc) * parts.splits);
    const ScoreFactor f = score_factor(a.scale);
    if (gc == 1) return launch_parts(&step_simt_kernel<D, 1>, grid, stream, a, parts, f);
    if (gc == 2) return launch_parts(&step_simt_kernel<D, 2>, grid, stream, a, parts, f);
    return launch_parts(&step_simt_kernel<D, 4>, grid, stream, a, parts, f);
}

template <int D>
cudaError_t launch_bf16(const StepArgs &a, const Parts &parts, cudaStream_t stream) {
    const int G = a.Hq / a.Hk, heads = heads_of_cta(G, LR_DT_BF16);
    const unsigned grid = (unsigned)(a.N * a.Hk * ((G + heads - 1) / heads) * parts.splits);
    const ScoreFactor f = score_factor(a.scale);
    if (heads == 8) return launch_parts(&step_mma_kernel<D, 1>, grid, stream, a, parts, f);
    return launch_parts(&step_mma_kernel<D, 2>, grid, stream, a, parts, f);
}

template <int D>
cudaError_t launch(const StepArgs &a, void *ws, lr_dtype dt, cudaStream_t stream) {
    const StepPlan p = step_plan(a.N, a.Hq, a.Hk, D, a.max_len, a.window, a.sinks, dt);
    const Parts parts = parts_of(a, D, p, ws);
    const cudaError_t e = dt == LR_DT_F32 ? launch_f32<D>(a, parts, stream) : launch_bf16<D>(a, parts, stream);
    if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
    const unsigned rows = (unsigned)(a.N * a.Hq);
    const ScoreFactor f = score_factor(a.scale);
    if (dt == LR_DT_F32) step_join_kernel<float, D><<<rows, D, 0, stream>>>(a, parts, f);
    else step_join_kernel<__nv_bfloat16, D><<<rows, D, 0, stream>>>(a, parts, f);
    return cudaGetLastError();
}

}  // namespace

StepPlan step_plan(int N, int Hq, int Hk, int d, int max_len, int window, int sinks, lr_dtype dt) {
    const long long w = (long long)window + sinks;
    // whole tiles in bf16: the sinks' and the window's first and last may be cut
    const long long most = w < max_len ? w + (dt == LR_DT_BF16 ? 2 * kTile + (sinks > 0 ? kTile : 0) : 0) : max_len;
    const int seen = (int)(most < max_len ? most : max_len);
    // CTAs that run at once: an SM holds the registers of three of the bf16
    // kernel at d = 128 (two with more than 8 heads; more at smaller widths,
    // where one wave matters less), of three in fp32 with four heads, else of
    // four or five (33 sequences with window 1024: 26 us with 4, 39 with 3, 33
    // with 6).
    const int G = Hq / Hk, heads = heads_of_cta(G, dt);
    const int per_sm = dt == LR_DT_BF16 ? (heads == 8 ? 3 : 2) : (heads == 4 ? 3 : 4);
    const int *room = kClusterRoom[(dt == LR_DT_BF16 && d < 128 ? 4 : per_sm) - 1];
    const long long rows = (long long)N * Hk * ((G + heads - 1) / heads), wave = 152 * per_sm;
    auto cut = [](long long keys, long long parts) {  // chunks of whole 64s, 64 at least
        const long long c = ((keys + parts - 1) / parts + 63) / 64 * 64;
        return c < 64 ? 64 : c;
    };
    StepPlan p;
    // Chunks of 64 to 1024 keys that one wave holds (a wave and a third took
    // 113 us on two 131K caches, one 87); for few rows up to 4096 keys, with
    // more rows pieces of 1024, which even out sequences of different lengths
    // (128 of 500 to 8192 keys: 355 us with 1024, 378 with 4096, 411 with 256).
    long long parts = rows < wave ? wave / rows : 1;
    // a cluster too many would be a second wave (8 sequences of 8192, 8 key
    // heads: 47 us by 6, 71 by 7)
    if (parts <= kMostCluster)
        while (parts > 1 && rows * parts > room[parts]) --parts;
    long long chunk = cut(seen, parts);
    if (chunk > (4 * rows <= wave ? kTile * kMostTiles : 1024)) chunk = 1024;
    p.chunk = (int)chunk;
    p.splits = (int)((seen + chunk - 1) / chunk);
    // Eight chunks or fewer that find room: a cluster joins them.  It does so too
    // where 512 keys for a CTA still leave eight chunks: one launch less is
    // worth more than the rest of the wave.
    const long long eighth = cut(seen, kMostCluster);
    p.cluster = false;
    const int most_parts = p.splits < kMostCluster ? p.splits : kMostCluster;
    if (p.splits > 1 && rows * most_parts <= room[most_parts] &&
        (p.splits <= kMostCluster || eighth <= 512)) {
        if (p.splits > kMostCluster) {
            p.chunk = (int)eighth;
            p.splits = (int)((seen + eighth - 1) / eighth);
        }
        p.cluster = p.splits > 1;
    }
    return p;
}

size_t step_workspace_bytes(int N, int Hq, int d, const StepPlan &p) {
    if (p.splits <= 1 || p.cluster) return 0;
    return (size_t)N * Hq * p.splits * ((size_t)d * 4 + 8);
}

cudaError_t launch_step_paged(const StepArgs &a, int d, lr_dtype dt, void *ws, cudaStream_t stream) {
    if (d == 32) return launch<32>(a, ws, dt, stream);
    if (d == 64) return launch<64>(a, ws, dt, stream);
    return launch<128>(a, ws, dt, stream);
}

int attn_errors_step() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_step_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_step_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
