// lr_step_paged_diff: differential attention of one new token per sequence over a
// paged cache (attn_diff.cuh has the formula; key and value heads in pairs).
//
// The cut is that of step_paged.cu: a CTA takes a chunk of the keys of one
// sequence and pair of key heads, for up to 8 pairs of query heads that share
// them (2 in fp32); chunks are joined by a cluster or a second kernel, in their
// order.  The bound is the read of the cache.
//
// bf16 (step_diff_mma_kernel): one warp fills a ring of 16-key tiles by TMA, both
// maps' keys and the value rows, so the reads in flight do not depend on registers;
// four others each work on one map and every other tile, S^T = K Q^T and O^T += V^T
// P^T with warp-level products, the values shared by the two maps' warps.  What the
// rounding of a weight to bf16 left is multiplied as well: the difference of the
// maps takes away what they have in common, but not their roundings.
// Measured: 64 sequences of 500 to 8192 tokens, 16 pairs on 4, d = 128: 184 us, 92 % of the
// copy rate (fragments loaded to registers as in step_paged.cu: 262, 216 registers); one
// sequence of 1200, d = 64: 12.3 us, length, page and rows one after the other.
//
// fp32 (step_diff_simt_kernel): CUDA cores; d / 8 lanes hold a key of both maps
// and its value row.
#include "attn_diff.cuh"
#include "attn_internal.cuh"
#include "attn_rows.cuh"
#include "attn_step.cuh"
#include "attn_tc.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

__device__ unsigned g_step_diff_error = 0;

constexpr int NT = 128;

// a: H = Hq pairs of query heads on Hk pairs of key heads.
struct DiffStep {
    StepArgs a;
    const float *lambda, *weight;
    float eps;
    int norm;
};

// fp32 partial results in the workspace: [N H][2 maps][splits][2 d], then
// (maximum, sum) [N H][2][splits].
struct Parts {
    float *o;
    float2 *ml;
    int splits, chunk;
    bool cluster;  // the chunks of a row are the CTAs of a cluster
};

__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 r;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(addr) : "memory");
    return r;
}

// Rows of a sequence that is not computed.
template <typename E, int D>
__device__ __forceinline__ void zero_rows(const StepArgs &a, int n, int h0, int heads) {
    E *o = static_cast<E *>(a.o) + ((size_t)n * a.Hq + h0) * 2 * D;
    for (int i = threadIdx.x; i < heads * 2 * D; i += blockDim.x) o[i] = from_f<E>(0.f);
}

// The row of pair h of sequence n by one warp, from `count` parts of each map:
// ml(i, map) is part i's (maximum, sum), value(i, map, ch) its unnormalised
// output.  A part without a key has a maximum of -inf and weighs nothing; one
// whose scores were all NaN too, but its sum of NaN stays.
template <typename E, int D, typename ML, typename Value>
__device__ __forceinline__ void finish_pair(const DiffStep &s, int n, int h, int count, ScoreFactor f, const ML &ml,
                                            const Value &value) {
    constexpr int N = D / 16;  // channels of a lane: lane + 32 i of 2 D
    const StepArgs &a = s.a;
    const int lane = threadIdx.x & 31;
    const float lambda = s.lambda[h];
    float y[N];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
        float top = -INFINITY, sum = 0.f, x[N];
#pragma unroll
        for (int c = 0; c < N; ++c) x[c] = 0.f;
        // a lane a part, then all lanes part by part: the loads of a batch do not
        // wait for each other
        for (int i0 = 0; i0 < count; i0 += 32) {
            const float2 t = i0 + lane < count ? ml(i0 + lane, map) : make_float2(-INFINITY, 0.f);
            float mn = t.x;
#pragma unroll
            for (int w = 16; w; w >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
            mn = fmaxf(mn, top);
            const float less = top == -INFINITY ? 0.f : ex2((top - mn) * f.c);
            const float w = t.x == -INFINITY ? 0.f : ex2((t.x - mn) * f.c);
            sum = sum * less + warp_sum(w * t.y);
#pragma unroll
            for (int c = 0; c < N; ++c) x[c] *= less;
            const int many = min(32, count - i0);
#pragma unroll 4
            for (int j = 0; j < many; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
                for (int c = 0; c < N; ++c) x[c] += wj * value(i0 + j, map, lane + 32 * c);
            }
            top = mn;
        }
        // no key, or only scores of -inf: zeros
        const float inv = sum == 0.f ? 0.f : (map ? -lambda : 1.f) / sum;
        // each product rounded, so that equal maps cancel exactly
#pragma unroll
        for (int c = 0; c < N; ++c) y[c] = map ? __fadd_rn(y[c], __fmul_rn(x[c], inv)) : __fmul_rn(x[c], inv);
    }
    float squares = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) squares = fmaf(y[c], y[c], squares);
    squares = warp_sum(squares);
    bool odd = false;
    const float r = s.norm ? diff_rms(squares, D, s.eps) : 1.f;
    E *o = static_cast<E *>(a.o) + ((size_t)n * a.Hq + h) * 2 * D;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        odd = odd || !isfinite(y[c]);
        o[lane + 32 * c] = from_f<E>(y[c] * r * (s.norm && s.weight ? s.weight[lane + 32 * c] : 1.f));
    }
    if (!__any_sync(0xffffffffu, odd)) return;
    // not finite: from the definition; keys of pages outside the pool are left out
    const int g = h / (a.Hq / a.Hk), len = a.lens[n];
    const int *table = a.table + (size_t)n * a.max_pages;
    const E *q = static_cast<const E *>(a.q) + ((size_t)n * a.Hq + h) * 2 * D;
    float z[2][D / 32];
    mend_diff<E, D>(
        q, q + D,
        [&](int map, int half, int j, const E *&kj, const E *&vj) {
            const int page = table[j >> a.page_log2];
            if (page < 0 || page >= a.num_pages) return false;
            const long long head = (long long)page * 2 * a.Hk + 2 * g, at = j & ((1 << a.page_log2) - 1);
            kj = static_cast<const E *>(a.k) + (((head + map) << a.page_log2) + at) * D;
            vj = static_cast<const E *>(a.v) + (((head + half) << a.page_log2) + at) * D;
            return true;
        },
        lambda, s.norm, s.weight, s.eps, seen_keys(len - 1, len, a.window, a.sinks), f, 3, z);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[half * D + lane * (D / 32) + i] = from_f<E>(z[half][i]);
}

// The end of a CTA: its warps' parts of each map, streams of them, are joined
// and handed on.  so[stream][map][head]: unnormalised outputs, P floats a row;
// sml: their (maximum, sum).
template <typename E, int D, int STREAMS, int HEADS, int P, int THREADS>
__device__ __forceinline__ void finish(float (&so)[STREAMS][2][HEADS][P], float2 (&sml)[STREAMS][2][HEADS], int heads,
                                       int n, int h0, int split, ScoreFactor f, const DiffStep &s,
                                       const Parts &parts) {
    const int tid = threadIdx.x, warp = tid >> 5;
    if (parts.cluster) tc::cluster_sync_all();
    else __syncthreads();
    if (parts.splits == 1) {
        for (int h = warp; h < heads; h += THREADS / 32)
            finish_pair<E, D>(
                s, n, h0 + h, STREAMS, f, [&](int i, int map) { return sml[i][map][h]; },
                [&](int i, int map, int ch) { return so[i][map][h][ch]; });
    } else if (parts.cluster) {
        const uint32_t o_at = tc::smem_u32(&so[0][0][0][0]), ml_at = tc::smem_u32(&sml[0][0][0]);
        for (int h = split * (THREADS / 32) + warp; h < heads; h += parts.splits * (THREADS / 32))
            finish_pair<E, D>(
                s, n, h0 + h, parts.splits * STREAMS, f,
                [&](int i, int map) {
                    return ld_cluster2(tc::map_to_rank(ml_at + 8 * ((i % STREAMS * 2 + map) * HEADS + h), i / STREAMS));
                },
                [&](int i, int map, int ch) {
                    return ld_cluster(
                        tc::map_to_rank(o_at + 4 * (((i % STREAMS * 2 + map) * HEADS + h) * P + ch), i / STREAMS));
                });
        tc::cluster_sync_all();  // no CTA leaves while another reads its part
    } else {
        for (int i = tid; i < 2 * heads * 2 * D; i += THREADS) {
            const int row = i / (2 * D), ch = i - row * 2 * D, map = row & 1, h = row >> 1;
            float mn = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < STREAMS; ++w) mn = fmaxf(mn, sml[w][map][h].x);
#pragma unroll
            for (int w = 0; w < STREAMS; ++w) {
                const float2 t = sml[w][map][h];
                const float fw = t.x == -INFINITY ? 0.f : ex2((t.x - mn) * f.c);
                sum += fw * t.y;
                x += fw * so[w][map][h][ch];
            }
            const size_t r = (((size_t)n * s.a.Hq + h0 + h) * 2 + map) * parts.splits + split;
            parts.o[r * 2 * D + ch] = x;
            if (ch == 0) parts.ml[r] = make_float2(mn, sum);
        }
    }
}

// The keys of a sequence as tiles of 16: its sinks', then its window's.
struct Tiles {
    SeenKeys s;
    int sink_tiles, first, count;  // first: window tile in units of 16 keys

    __device__ __forceinline__ explicit Tiles(const SeenKeys &seen) : s(seen) {
        sink_tiles = (s.s1 + kTile - 1) / kTile;
        first = max(s.lo / kTile, sink_tiles);  // a tile that holds both is a sink tile
        count = sink_tiles + max(0, (s.hi + kTile - 1) / kTile - first);
    }
    __device__ __forceinline__ int key(int i) const { return kTile * (i < sink_tiles ? i : i - sink_tiles + first); }
    __device__ __forceinline__ bool sees(int key) const { return key < s.hi && (key >= s.lo || key < s.s1); }
};

// Shared memory of the bf16 kernel: a ring of tiles, each 16 rows of both maps'
// keys and of both halves of the values in 64-column blocks as TMA leaves them
// (128-byte swizzle); the warps' parts lie over it when the tiles are used up.
template <int D>
struct Ring {
    static constexpr int KB = D > 64 ? 2 : 1;    // 64-column blocks of a row
    static constexpr int PIECE = KB * kTile * 128;
    static constexpr int TILE = 4 * PIECE;
    static constexpr int NS = D > 64 ? 6 : 8;    // tiles in flight
    static constexpr int HEADS = 8, STREAMS = 2, P = 2 * D + 8;
    struct Parts {
        float so[STREAMS][2][HEADS][P];
        float2 sml[STREAMS][2][HEADS];
    };
    static_assert(sizeof(Parts) <= NS * TILE, "the parts over the ring");
    static constexpr int BYTES = NS * TILE + 1024;  // the ring starts on a 1024-byte boundary
};
constexpr int kMmaThreads = 160;  // four warps of products, one of loads

template <int D>
__global__ void __launch_bounds__(kMmaThreads)
    step_diff_mma_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, DiffStep s,
                         Parts parts, ScoreFactor f) {
    using R = Ring<D>;
    const StepArgs &a = s.a;
    const float c = f.c;
    const __nv_bfloat162 sign = __float2bfloat162_rn(f.sign);
    auto with_sign = [&](uint32_t x) {  // exact: 1, -1 or 0 times a pair
        const __nv_bfloat162 y = __hmul2(reinterpret_cast<const __nv_bfloat162 &>(x), sign);
        return reinterpret_cast<const uint32_t &>(y);
    };
    constexpr int KC = D / 32;   // 32-channel pieces of a key: 16 bytes per lane and row
    constexpr int VW = D / 16;   // words of a value half-row per lane = 16-channel blocks of O^T
    constexpr int HEADS = R::HEADS, STREAMS = R::STREAMS;
    extern __shared__ uint8_t raw[];
    __shared__ int pages[kMostTiles];  // of each tile, -1: outside the pool
    __shared__ uint64_t full[R::NS], empty[R::NS];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int map = warp & 1, stream = warp >> 1;
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
        if (len > 0 && tid == 0 && split == 0 && gi == 0 && hk == 0) atomicOr(&g_step_diff_error, kAttnIndex);
        if (a.fill && split == 0) zero_rows<__nv_bfloat16, D>(a, n, h0, heads);
        return;
    }
    const Tiles tiles(seen_keys(len - 1, len, a.window, a.sinks));
    const int per = parts.chunk / kTile, t0 = split * per, t1 = min(tiles.count, t0 + per);
    if (t0 >= tiles.count && split > 0 && !parts.cluster) return;  // the join knows how many chunks there are

    if (tid == 0) {
        for (int i = 0; i < R::NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 2);  // the warps of both maps
        }
        tc::fence_mbar_init();
    }
    for (int i = tid; i < t1 - t0; i += kMmaThreads) {
        const int page = a.table[(size_t)n * a.max_pages + (tiles.key(t0 + i) >> a.page_log2)];
        const bool in = page >= 0 && page < a.num_pages;
        if (!in) atomicOr(&g_step_diff_error, kAttnIndex);
        pages[i] = in ? page : -1;
    }
    // queries of the warp's map: head g, the channels that the lane's keys hold
    uint32_t q[2 * KC][2];
    {
        const bool live = g < heads;
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(a.q) +
                                 (((size_t)n * a.Hq + h0 + (live ? g : 0)) * 2 + map) * D + 8 * t;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *reinterpret_cast<const uint4 *>(p + 32 * i);
            q[2 * i][0] = with_sign(x.x), q[2 * i][1] = with_sign(x.y);
            q[2 * i + 1][0] = with_sign(x.z), q[2 * i + 1][1] = with_sign(x.w);
        }
    }
    __syncthreads();

    bool ok = true;
    float acc[2 * VW][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2 * VW; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    if (warp == 4) {
        // loads: both maps' keys, both halves of the values
        int i = t0;
        for (; i < t1; ++i) {
            const int k = i - t0, slot = k % R::NS, page = pages[k];
            if (k >= R::NS) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[slot], (k / R::NS - 1) & 1));
            if (!ok) break;
            if (lane == 0) {
                if (page >= 0) {
                    const int row = tiles.key(i) & ((1 << a.page_log2) - 1);
                    uint8_t *to = ring + slot * R::TILE;
                    tc::mbar_expect_tx(&full[slot], R::TILE);
                    tc::tma_load_5d(to, &tmk, 0, row, 0, 2 * hk, page, &full[slot]);
                    tc::tma_load_5d(to + 2 * R::PIECE, &tmv, 0, row, 0, 2 * hk, page, &full[slot]);
                } else {
                    tc::mbar_arrive(&full[slot]);  // nothing is read of it
                }
            }
            __syncwarp();
        }
        // never leave with copies into shared memory in flight
        for (int k = max(0, i - t0 - R::NS); k < i - t0; ++k)
            if (!tc::mbar_wait(&full[k % R::NS], (k / R::NS) & 1)) ok = false;
    } else {
        for (int i = t0 + stream; i < t1; i += STREAMS) {
            const int k = i - t0, slot = k % R::NS, key = tiles.key(i);
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[slot], (k / R::NS) & 1));
            if (!ok) break;
            const uint8_t *tile = ring + slot * R::TILE, *kt = tile + map * R::PIECE;
            const bool page_ok = pages[k] >= 0;
            // rows that the sequence does not see: scores of -inf, values of zero
            const bool all = page_ok && tiles.sees(key) && tiles.sees(key + kTile - 1) &&
                             (key >= tiles.s.lo || key + kTile <= tiles.s.s1);
            float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                // chunk of 8 channels (j & 1) 4 + t of block j / 2, rows g and g + 8
                const uint8_t *p = kt + (j >> 1) * (kTile * 128) + g * 128 + ((((j & 1) * 4 + t) ^ g) << 4);
                const uint4 x = *reinterpret_cast<const uint4 *>(p), y = *reinterpret_cast<const uint4 *>(p + 1024);
                mma16816(sc, x.x, y.x, x.y, y.y, q[2 * j][0], q[2 * j][1]);
                mma16816(sd, x.z, y.z, x.w, y.w, q[2 * j + 1][0], q[2 * j + 1][1]);
            }
            const bool see0 = all || (page_ok && tiles.sees(key + g)), see1 = all || (page_ok && tiles.sees(key + g + 8));
            bool grow = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = (e < 2 ? see0 : see1) ? sc[e] + sd[e] : -INFINITY, y = m[e & 1];
                sc[e] = x;
                grow = grow || (x > y && !((x - y) * c <= 8.f));
            }
            // the maximum in use is raised only when a score passes it by 2^8
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(sc[e], sc[e + 2]);
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                    const float mn = fmaxf(m[e], mx);
                    const float less = m[e] == -INFINITY ? 0.f : ex2((m[e] - mn) * c);
                    m[e] = mn;
                    // nothing seen yet: sums and output are zero (or NaN, which stays)
                    l[e] *= less;
#pragma unroll
                    for (int j = 0; j < 2 * VW; ++j) acc[j][e] *= less, acc[j][e + 2] *= less;
                }
            }
            const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
            // differences first: a product of one large score would overflow
            const float2 e0 = make_float2(ex2((sc[0] - b0) * c), ex2((sc[1] - b1) * c)),
                         e1 = make_float2(ex2((sc[2] - b0) * c), ex2((sc[3] - b1) * c));
            l[0] += e0.x + e1.x;
            l[1] += e0.y + e1.y;
            // the weights, and as weights of their own what their rounding left
            uint32_t r0, r1;
            const uint32_t p0 = transpose8x8(tc::pack2_rest(e0, r0)), p1 = transpose8x8(tc::pack2_rest(e1, r1));
            r0 = transpose8x8(r0), r1 = transpose8x8(r1);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t vr[4][VW];  // values of keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 2 * t + (r & 1) + 8 * (r >> 1);
                    const uint8_t *p = tile + (2 + half) * R::PIECE + row * 128;
                    if (D == 32) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(p + (((g >> 1) ^ (row & 7)) << 4) + (g & 1) * 8);
                        vr[r][0] = x.x, vr[r][1] = x.y;
                    } else {
#pragma unroll
                        for (int w = 0; w < VW / 4; ++w) {
                            const uint4 x =
                                *reinterpret_cast<const uint4 *>(p + w * (kTile * 128) + ((g ^ (row & 7)) << 4));
                            vr[r][4 * w] = x.x, vr[r][4 * w + 1] = x.y, vr[r][4 * w + 2] = x.z, vr[r][4 * w + 3] = x.w;
                        }
                    }
                    if (!all && !(page_ok && tiles.sees(key + row))) {
#pragma unroll
                        for (int w = 0; w < VW; ++w) vr[r][w] = 0u;
                    }
                }
                if (half == 1) {  // the tile has been read
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&empty[slot]);
                }
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const uint32_t a0 = __byte_perm(vr[0][j], vr[1][j], 0x5410), a1 = __byte_perm(vr[0][j], vr[1][j], 0x7632),
                                   a2 = __byte_perm(vr[2][j], vr[3][j], 0x5410), a3 = __byte_perm(vr[2][j], vr[3][j], 0x7632);
                    mma16816(acc[half * VW + j], a0, a1, a2, a3, p0, p1);
                    mma16816(acc[half * VW + j], a0, a1, a2, a3, r0, r1);
                }
            }
        }
    }
    if (!ok) atomicOr(&g_step_diff_error, kAttnTimeout);
    __syncthreads();  // the ring is free
    typename R::Parts &own = *reinterpret_cast<typename R::Parts *>(ring);
    if (warp < 4) {
        // this warp's part: word j of a half's lane holds channels col_j and col_j + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int h = 2 * t + e;
            if (g == 0) own.sml[stream][map][h] = make_float2(m[e], sum);
#pragma unroll
            for (int j = 0; j < 2 * VW; ++j) {
                const int w = j % VW, col = D == 32 ? 4 * g + 2 * w : 64 * (w >> 2) + 8 * g + 2 * (w & 3);
                *reinterpret_cast<float2 *>(&own.so[stream][map][h][j / VW * D + col]) =
                    make_float2(acc[j][e], acc[j][e + 2]);
            }
        }
    }
    finish<__nv_bfloat16, D, STREAMS, HEADS, R::P, kMmaThreads>(own.so, own.sml, heads, n, h0, split, f, s, parts);
}

// ------------------------------------------------------------------- fp32

template <int D, int GC>
__global__ void __launch_bounds__(NT) step_diff_simt_kernel(DiffStep s, Parts parts, ScoreFactor f) {
    const StepArgs &a = s.a;
    constexpr int LANES = D / 8;            // lanes of a key
    constexpr int GROUPS = NT / LANES;      // keys in flight
    constexpr int U = 2;                    // keys of a group per pass
    constexpr int STREAMS = NT / 32;
    __shared__ float so[STREAMS][2][GC][2 * D];
    __shared__ float2 sml[STREAMS][2][GC];
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
        if (len > 0 && tid == 0 && split == 0 && gi == 0 && hk == 0) atomicOr(&g_step_diff_error, kAttnIndex);
        if (a.fill && split == 0) zero_rows<float, D>(a, n, h0, heads);
        return;
    }
    const SeenKeys sk = seen_keys(len - 1, len, a.window, a.sinks);
    const int seen = sk.s1 + sk.hi - sk.lo;
    const int c0 = split * parts.chunk;
    if (c0 >= seen && split > 0 && !parts.cluster) return;  // the join knows how many chunks there are
    const int c1 = min(seen, c0 + parts.chunk);
    const int lane = tid % LANES, group = tid / LANES, ch = lane * 8;

    const float *qn = static_cast<const float *>(a.q) + (size_t)n * a.Hq * 2 * D;
    float q[2][GC][8], acc[2][GC][16], m[2][GC], l[2][GC];
#pragma unroll
    for (int map = 0; map < 2; ++map)
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            load8(qn + (size_t)((h0 + min(g, heads - 1)) * 2 + map) * D + ch, q[map][g]);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[map][g][i] *= f.sign;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[map][g][i] = 0.f;
            m[map][g] = -INFINITY, l[map][g] = 0.f;
        }
    const int *table = a.table + (size_t)n * a.max_pages;
    const int in_page = (1 << a.page_log2) - 1;
    const long long next_head = (long long)D << a.page_log2;
    const int lanes0 = (tid & 31) / LANES * LANES;
    const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << lanes0;
    bool bad = false;
    for (int base = c0 + group; base < c1; base += GROUPS * U) {
        long long row[U];
        float x[U][2][8], y[U][16], sc[U][2][GC];  // keys of both maps, values: all on their way at once
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * GROUPS;
            row[u] = -1;
            if (i < c1) {
                const int key = i < sk.s1 ? i : i - sk.s1 + sk.lo;
                const int page = table[key >> a.page_log2];
                if (page >= 0 && page < a.num_pages)
                    row[u] = ((((long long)page * 2 * a.Hk + 2 * hk) << a.page_log2) + (key & in_page)) * D + ch;
                else
                    bad = true;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][half][i] = v8[i] = 0.f;
                if (row[u] >= 0) {
                    load8(static_cast<const float *>(a.k) + row[u] + half * next_head, x[u][half]);
                    load8(static_cast<const float *>(a.v) + row[u] + half * next_head, v8);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) y[u][half * 8 + i] = v8[i];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int map = 0; map < 2; ++map)
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    float t = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) t += q[map][g][i] * x[u][map][i];
#pragma unroll
                    for (int w = 1; w < LANES; w <<= 1) t += __shfl_xor_sync(mask, t, w);
                    sc[u][map][g] = row[u] >= 0 ? t : -INFINITY;
                }
#pragma unroll
        for (int map = 0; map < 2; ++map)
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                float mn = m[map][g];
#pragma unroll
                for (int u = 0; u < U; ++u) mn = fmaxf(mn, sc[u][map][g]);
                const float b = mn == -INFINITY ? 0.f : mn;
                const float less = ex2((m[map][g] - b) * f.c);
                m[map][g] = mn;
                l[map][g] *= less;
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[map][g][i] *= less;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float p = ex2((sc[u][map][g] - b) * f.c);
                    l[map][g] += p;
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[map][g][i] += p * y[u][i];
                }
            }
    }
    if (bad) atomicOr(&g_step_diff_error, kAttnIndex);
    __syncwarp();
    // the groups of a warp, then the warps
#pragma unroll
    for (int map = 0; map < 2; ++map)
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            float mn = m[map][g];
#pragma unroll
            for (int w = LANES; w < 32; w <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
            const float less = m[map][g] == -INFINITY ? 0.f : ex2((m[map][g] - mn) * f.c);
            l[map][g] *= less;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[map][g][i] *= less;
#pragma unroll
            for (int w = LANES; w < 32; w <<= 1) {
                l[map][g] += __shfl_xor_sync(0xffffffffu, l[map][g], w);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[map][g][i] += __shfl_xor_sync(0xffffffffu, acc[map][g][i], w);
            }
            if ((tid & 31) < LANES) {
#pragma unroll
                for (int i = 0; i < 16; ++i) so[warp][map][g][(i >> 3) * D + ch + (i & 7)] = acc[map][g][i];
                if (lane == 0) sml[warp][map][g] = make_float2(mn, l[map][g]);
            }
        }
    finish<float, D, STREAMS, GC, 2 * D, NT>(so, sml, heads, n, h0, split, f, s, parts);
}

// A warp per pair of a sequence: the chunks' parts in order.
template <typename E, int D>
__global__ void __launch_bounds__(32) step_diff_join_kernel(DiffStep s, Parts parts, ScoreFactor f) {
    const StepArgs &a = s.a;
    const int r = blockIdx.x, n = r / a.Hq, len = a.lens[n];
    if (len < 0 || len > a.max_len) return;
    const SeenKeys sk = seen_keys(len - 1, len, a.window, a.sinks);
    // whole tiles of 16 keys in bf16
    const int seen = sizeof(E) == 2 ? kTile * Tiles(sk).count : sk.s1 + sk.hi - sk.lo;
    const int used = max(1, (seen + parts.chunk - 1) / parts.chunk);
    const float2 *ml = parts.ml + (size_t)r * 2 * parts.splits;
    const float *o = parts.o + (size_t)r * 2 * parts.splits * 2 * D;
    finish_pair<E, D>(
        s, n, r - n * a.Hq, used, f, [&](int i, int map) { return ml[map * parts.splits + i]; },
        [&](int i, int map, int ch) { return o[((size_t)map * parts.splits + i) * 2 * D + ch]; });
}

// Pairs of query heads that a CTA takes, of G that share keys.
int pairs_of_cta(int G, lr_dtype dt) { return dt == LR_DT_BF16 ? 8 : (G == 1 ? 1 : 2); }

template <int D>
cudaError_t launch(const DiffStep &s, void *ws, lr_dtype dt, cudaStream_t stream) {
    const StepArgs &a = s.a;
    const StepPlan p = diff_step_plan(a.N, a.Hq, a.Hk, D, a.max_len, a.window, a.sinks, dt);
    Parts parts{};
    parts.splits = p.splits, parts.chunk = p.chunk, parts.cluster = p.cluster;
    if (p.splits > 1 && !p.cluster) {
        parts.o = static_cast<float *>(ws);
        parts.ml = reinterpret_cast<float2 *>(parts.o + (size_t)a.N * a.Hq * 2 * p.splits * 2 * D);
    }
    const int G = a.Hq / a.Hk, gc = pairs_of_cta(G, dt);
    const unsigned grid = (unsigned)(a.N * a.Hk * ((G + gc - 1) / gc) * p.splits);
    const int cluster = p.cluster ? p.splits : 1;
    const ScoreFactor f = score_factor(a.scale);
    cudaError_t e;
    if (dt == LR_DT_BF16) {
        CUtensorMap mk, mv;
        e = tc::pool_map(&mk, a.k, D, 1 << a.page_log2, 2 * a.Hk, a.num_pages, kTile, 2);
        if (e == cudaSuccess) e = tc::pool_map(&mv, a.v, D, 1 << a.page_log2, 2 * a.Hk, a.num_pages, kTile, 2);
        auto *fn = &step_diff_mma_kernel<D>;
        if (e == cudaSuccess)
            e = ensure_smem_attr(reinterpret_cast<const void *>(fn), Ring<D>::BYTES, 233 + D / 64);
        if (e == cudaSuccess)
            e = launch_cut(fn, grid, kMmaThreads, cluster, Ring<D>::BYTES, false, stream, mk, mv, s, parts, f);
    } else if (gc == 1) {
        e = launch_cut(&step_diff_simt_kernel<D, 1>, grid, NT, cluster, 0, false, stream, s, parts, f);
    } else {
        e = launch_cut(&step_diff_simt_kernel<D, 2>, grid, NT, cluster, 0, false, stream, s, parts, f);
    }
    if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
    const unsigned rows = (unsigned)(a.N * a.Hq);
    if (dt == LR_DT_F32) step_diff_join_kernel<float, D><<<rows, 32, 0, stream>>>(s, parts, f);
    else step_diff_join_kernel<__nv_bfloat16, D><<<rows, 32, 0, stream>>>(s, parts, f);
    return cudaGetLastError();
}

// ensure_smem_attr slots 233..235 belong to this file.

}  // namespace

StepPlan diff_step_plan(int N, int H, int Hk, int d, int max_len, int window, int sinks, lr_dtype dt) {
    const long long w = (long long)window + sinks;
    // whole tiles in bf16: the sinks' and the window's first and last may be cut
    const long long most = w < max_len ? w + (dt == LR_DT_BF16 ? 2 * kTile + (sinks > 0 ? kTile : 0) : 0) : max_len;
    const int seen = (int)(most < max_len ? most : max_len);
    const int G = H / Hk, pairs = pairs_of_cta(G, dt);
    // CTAs on an SM: the rings fill its shared memory; registers in fp32
    const int per_sm = dt == LR_DT_BF16 && d == 128 ? 2 : 3;
    return plan_chunks(seen, (long long)N * Hk * ((G + pairs - 1) / pairs), per_sm, kClusterRoom[per_sm - 1]);
}

size_t diff_step_workspace_bytes(int N, int H, int d, const StepPlan &p) {
    if (p.splits <= 1 || p.cluster) return 0;
    return (size_t)N * H * 2 * p.splits * ((size_t)d * 8 + 8);
}

cudaError_t launch_step_diff(const StepArgs &a, const float *lambda, const float *weight, float eps, bool norm, int d,
                             lr_dtype dt, void *ws, cudaStream_t stream) {
    const DiffStep s{a, lambda, weight, eps, norm};
    if (d == 32) return launch<32>(s, ws, dt, stream);
    if (d == 64) return launch<64>(s, ws, dt, stream);
    return launch<128>(s, ws, dt, stream);
}

int attn_errors_step_diff() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_step_diff_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_step_diff_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
