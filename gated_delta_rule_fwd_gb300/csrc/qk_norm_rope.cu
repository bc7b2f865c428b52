// lr_qk_norm_rope and lr_qk_norm_rope_axes: RMS norm of each query and key head,
// the position rotation and the write of keys and values into a paged cache, in
// one pass.
//
// A row (one head of one token) is held by d / 8 lanes of a warp, eight
// channels each, so that its sum of squares and the partner channels of the
// split-half rotation come from shuffles.  The angles of a token are the same
// for all its heads: a lane forms the cosines and sines of its channels once
// and then walks the heads of its token, several rows in flight; no lane waits
// for another outside the shuffles.  With few tokens the lanes of a CTA are
// shared out over the heads instead.
//
// Angle: th = p f.  With s = frac(f / 2 pi) as a 64-bit fixed-point fraction
// of a turn, p s mod 2^64 is the exact fraction of the product, so the only
// errors are those of s (2^-64 of a turn) and of the final fp32 conversion
// (2^-25 of a half turn), whatever the position and the frequency.  s takes the
// product f / 2 pi with what its rounding and that of 1 / 2 pi leave out (fp64
// alone would be off by 2^-53 of the turns of a position, which shows at the
// far end of an int from about one turn on).  It is formed once per CTA on the
// fp64 pipe, which does two operations a cycle.
#include "attn_internal.cuh"

namespace lr {
namespace {

__device__ unsigned g_rope_error = 0;

constexpr int NT = 256;
// Rows in flight per lane, and CTAs per SM: both hold the reads in flight that
// bound the kernel (with the issue of about 110 instructions a pair of rows).
// On 2 x 16384 tokens of 16 + 4 heads (bf16, 336 MB): 62 us, 5.4 TB/s, with 4
// rows and 3 CTAs; before the last cuts in instructions 72, and 79 with 2 rows
// and 4 CTAs, 85 with 4 rows and 2.  Fetching each next row as its place is
// free, across queries, keys and tokens, costs more instructions than it hides
// (65 to 67).  fp32 rows take twice the registers: two CTAs.  The bf16 form with
// split halves spills 12 bytes a thread at its 80 registers.
// With positions of three axes and the append: 76 us, 85 % of the copy rate.
constexpr int U = 4;
template <typename E> constexpr int kCtas = sizeof(E) == 2 ? 3 : 2;

struct RopeArgs {
    const void *q, *k, *v;
    void *qo, *ko, *ck, *cv;
    const int *positions, *table;
    const int *turns, *axis;  // several axes: positions [axes][B][T] and the axis of each
    int axes;                 // channel pair; `positions` then are places in the cache
    lr_strides qs, ks, vs;
    QkMaps maps;
    int T, Hq, Hk, num_pages, page_log2, max_pages;
    int tokens;  // of a group: a power of two
    int total;   // B * T
};

// Eight consecutive channels of a row as they are moved (16 or 32 bytes a
// lane) and as fp32 pairs.
template <typename E> struct Row8;
template <> struct Row8<float> {
    float2 x[4];
    __device__ __forceinline__ float2 pair(int i) const { return x[i]; }
    __device__ __forceinline__ void set(int i, float2 v) { x[i] = v; }
    // the same channels of another lane
    __device__ __forceinline__ float2 pair_of(int i, int lane) const {
        return make_float2(__shfl_sync(0xffffffffu, x[i].x, lane), __shfl_sync(0xffffffffu, x[i].y, lane));
    }
};
template <> struct Row8<__nv_bfloat16> {
    uint32_t x[4];
    __device__ __forceinline__ float2 pair(int i) const { return unpack2(x[i]); }
    __device__ __forceinline__ void set(int i, float2 v) { x[i] = pack2(v.x, v.y); }
    __device__ __forceinline__ float2 pair_of(int i, int lane) const {
        return unpack2(__shfl_sync(0xffffffffu, x[i], lane));
    }
};
__device__ __forceinline__ Row8<float> fetch(const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    return {{{a.x, a.y}, {a.z, a.w}, {b.x, b.y}, {b.z, b.w}}};
}
__device__ __forceinline__ Row8<__nv_bfloat16> fetch(const __nv_bfloat16 *p) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    return {{a.x, a.y, a.z, a.w}};
}
__device__ __forceinline__ void put(float *p, const Row8<float> &r) {
    *reinterpret_cast<float4 *>(p) = make_float4(r.x[0].x, r.x[0].y, r.x[1].x, r.x[1].y);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(r.x[2].x, r.x[2].y, r.x[3].x, r.x[3].y);
}
__device__ __forceinline__ void put(__nv_bfloat16 *p, const Row8<__nv_bfloat16> &r) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(r.x[0], r.x[1], r.x[2], r.x[3]);
}

enum Rotation { kNone, kHalves, kPairs };  // channels (i, i + rot/2) or (2i, 2i+1)

// AXES: the angles come from positions of several axes.
template <typename E, int D, Rotation ROT, bool AXES>
__global__ void __launch_bounds__(NT, kCtas<E>) qk_norm_rope_kernel(RopeArgs a) {
    constexpr int LANES = D / 8;      // lanes of a row
    constexpr int ROWS = NT / LANES;  // rows at once: tokens x head parts
    __shared__ unsigned long long step[D / 2];
    __shared__ const int *along[AXES ? D / 2 : 1];  // positions of the pair's axis
    const int tid = threadIdx.x, half = a.maps.rot >> 1;
    const bool norm = a.maps.flags & LR_QK_NORM, partial = a.maps.rot < D;
    // the lane's place: channels c0.., token `mine` of the group, every parts-th head
    const int c0 = tid % LANES * 8, row = tid / LANES;
    const int mine = row & (a.tokens - 1), part = row / a.tokens, parts = ROWS / a.tokens;
    const bool turns_here = ROT != kNone && c0 < a.maps.rot, low = c0 < half;
    // split halves: the partner channel c +- half sits half / 8 lanes away
    const int hop = ROT == kHalves && turns_here ? (low ? half : -half) : 0;
    const int from = (tid & 31) + hop / 8;
    if (ROT != kNone) {
        if (tid < half) {
            // 1 / (2 pi) as a sum of two; below, 2^64 units of a turn
            constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
            const double f = a.maps.inv_freq[tid], turns = f * kHigh;
            const double rest = fma(f, kLow, fma(f, kHigh, -turns));
            step[tid] = __double2ull_rz((turns - floor(turns)) * 0x1p64) +
                        (unsigned long long)__double2ll_rn(rest * 0x1p64);
            if (AXES) {
                int axis = a.axis[tid];
                if (axis < 0 || axis >= a.axes) {
                    atomicOr(&g_rope_error, kAttnIndex);
                    axis = 0;
                }
                along[tid] = a.turns + (size_t)axis * a.total;
            }
        }
        __syncthreads();
    }

    const int groups = (a.total + a.tokens - 1) / a.tokens;
    for (int group = blockIdx.x; group < groups; group += gridDim.x) {
        const int n0 = group * a.tokens + mine, n = n0 < a.total ? n0 : a.total - 1;
        const int b = n / a.T, t = n - b * a.T;
        const int p = a.positions ? a.positions[n] : t;
        const bool on = n0 < a.total && p >= 0;
        // U rows of heads h, h + parts, ... (the last head where there are none:
        // every address is a row of the tensor, and nothing of it is kept)
        auto fetch_rows = [&](Row8<E>(&r)[U], const E *src, long long stride, int count, int h) {
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = fetch(src + min(h + u * parts, count - 1) * stride);
        };
        // the first rows are on their way while the angles are formed
        const E *q_from = static_cast<const E *>(a.q) + b * a.qs.b + t * a.qs.t + c0;
        Row8<E> r[U];
        fetch_rows(r, q_from, a.qs.h, a.Hq, part);
        if (!on && n0 < a.total && (a.maps.flags & (LR_QK_ZERO_Q | LR_QK_ZERO_K))) {
            const Row8<E> zero{};
            if (a.maps.flags & LR_QK_ZERO_Q)
                for (int h = part; h < a.Hq; h += parts)
                    put(static_cast<E *>(a.qo) + (((size_t)b * a.Hq + h) * a.T + t) * D + c0, zero);
            if (a.ko && (a.maps.flags & LR_QK_ZERO_K))
                for (int h = part; h < a.Hk; h += parts)
                    put(static_cast<E *>(a.ko) + (((size_t)b * a.Hk + h) * a.T + t) * D + c0, zero);
        }
        if (!__any_sync(0xffffffffu, on)) continue;  // padding
        long long place = -1;  // first cache row of the token (head 0)
        if (a.ck && on) {
            const int pg = p >> a.page_log2;
            const int page = pg < a.max_pages ? a.table[(size_t)b * a.max_pages + pg] : -1;
            if (page >= 0 && page < a.num_pages)
                place = (((long long)page * a.Hk) << a.page_log2) + (p & ((1 << a.page_log2) - 1));
            else
                atomicOr(&g_rope_error, kAttnIndex);
        }
        float co[8], si[8];  // of the lane's channels, the partner's sign in si
#pragma unroll
        for (int i = 0; i < 8; ++i) co[i] = 1.f, si[i] = 0.f;
        if (turns_here) {
            // halves: both lanes of a pair need the same eight angles, each forms four
            constexpr int N = 4;
            float c4[N], s4[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = ROT == kPairs ? (c0 >> 1) + i : (low ? c0 + i : c0 - half + 4 + i);
                const int at = AXES ? along[c][n] : p;
                const unsigned long long phase = step[c] * (unsigned long long)(long long)at;
                // signed half turns in [-1, 1)
                const float x = (float)(int)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
                sincospif(x, &s4[i], &c4[i]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (ROT == kPairs) {
                    co[2 * i] = co[2 * i + 1] = c4[i];
                    si[2 * i] = -s4[i], si[2 * i + 1] = s4[i];
                } else {
                    co[i] = co[4 + i] = c4[i];  // one half is replaced by the other lane's below
                    si[i] = si[4 + i] = s4[i];
                }
            }
        }
        if (ROT == kHalves) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = __shfl_sync(0xffffffffu, co[i], from), s = __shfl_sync(0xffffffffu, si[i], from);
                if (turns_here) {
                    if (low) co[4 + i] = c, si[4 + i] = s;
                    else co[i] = c, si[i] = s;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (low) si[i] = -si[i];
        }
        // All heads of queries or keys, the first rows already in r; `keep`
        // stores a finished row.  A pair of channels becomes
        // (x wc + partner ws) / rms, the weight in the rotation's factors.
        auto heads = [&](const E *src, long long stride, int count, const float *weight, auto keep) {
            float2 wc[4], ws[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = c0 + i;
                const float w = weight ? weight[c] : 1.f;
                const float pw = weight ? weight[ROT == kPairs ? c ^ 1 : c + hop] : 1.f;
                float &fc = i & 1 ? wc[i / 2].y : wc[i / 2].x, &fs = i & 1 ? ws[i / 2].y : ws[i / 2].x;
                fc = w * co[i], fs = pw * si[i];
            }
#pragma unroll 1
            for (int h0 = part; h0 - part < count; h0 += parts * U) {
                if (h0 != part) fetch_rows(r, src, stride, count, h0);
                // bf16: the sums of the U rows together, with half the shuffles; lane
                // 4 j + u of a row ends up with row u's, takes its root and hands it to
                // the others (2 x 16384 tokens of 16 + 4 heads: 64.1 -> 62.1 us; fp32,
                // which is bound by its bytes, 107 -> 113).
                constexpr bool TOGETHER = sizeof(E) == 2;
                static_assert(U == 4, "four rows' sums");
                float inv = 1.f;
                if (TOGETHER && norm) {
                    float sum[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float2 ss = mul2(r[u].pair(0), r[u].pair(0));
#pragma unroll
                        for (int i = 1; i < 4; ++i) ss = fma2(r[u].pair(i), r[u].pair(i), ss);
                        sum[u] = ss.x + ss.y;
                    }
                    const bool one = tid & 1, two = tid & 2;
                    const float a0 = (one ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, one ? sum[0] : sum[1], 1);
                    const float a1 = (one ? sum[3] : sum[2]) + __shfl_xor_sync(0xffffffffu, one ? sum[2] : sum[3], 1);
                    float all = (two ? a1 : a0) + __shfl_xor_sync(0xffffffffu, two ? a0 : a1, 2);
#pragma unroll
                    for (int m = 4; m < LANES; m <<= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
                    inv = rsqrtf(all * (1.f / D) + a.maps.eps);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 - part + u * parts >= count) break;  // for all lanes
                    float2 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = r[u].pair(i);
                    float of_u = TOGETHER ? __shfl_sync(0xffffffffu, inv, (tid & 28) | u) : 1.f;
                    if (!TOGETHER && norm) {
                        float2 ss = mul2(x[0], x[0]);
#pragma unroll
                        for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
                        float sum = ss.x + ss.y;
#pragma unroll
                        for (int m = 1; m < LANES; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                        of_u = rsqrtf(sum * (1.f / D) + a.maps.eps);
                    }
                    const float2 inv2 = make_float2(of_u, of_u);
                    Row8<E> y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 z = mul2(x[i], wc[i]);
                        if (ROT != kNone) {
                            float2 w = ROT == kPairs ? make_float2(x[i].y, x[i].x) : r[u].pair_of(i, from);
                            // where nothing turns the partner is not looked at (it may be infinite)
                            if (partial && !turns_here) w = make_float2(0.f, 0.f);
                            z = fma2(w, ws[i], z);
                        }
                        y.set(i, mul2(z, inv2));
                    }
                    if (on && h0 + u * parts < count) keep(h0 + u * parts, y);
                }
            }
        };
        E *q_to = static_cast<E *>(a.qo) + ((size_t)b * a.Hq * a.T + t) * D + c0;
        heads(q_from, a.qs.h, a.Hq, a.maps.qw,
              [&](int h, const Row8<E> &y) { put(q_to + (size_t)h * a.T * D, y); });
        const E *k_from = static_cast<const E *>(a.k) + b * a.ks.b + t * a.ks.t + c0;
        fetch_rows(r, k_from, a.ks.h, a.Hk, part);
        E *k_to = a.ko ? static_cast<E *>(a.ko) + ((size_t)b * a.Hk * a.T + t) * D + c0 : nullptr;
        E *kept = place >= 0 ? static_cast<E *>(a.ck) + place * D + c0 : nullptr;
        heads(k_from, a.ks.h, a.Hk, a.maps.kw, [&](int h, const Row8<E> &y) {
            if (k_to) put(k_to + (size_t)h * a.T * D, y);
            if (kept) put(kept + ((size_t)h << a.page_log2) * D, y);
        });
        if (a.ck) {
            const E *v_from = static_cast<const E *>(a.v) + b * a.vs.b + t * a.vs.t + c0;
            E *to = static_cast<E *>(a.cv) + place * D + c0;
#pragma unroll 1
            for (int h0 = part; h0 < a.Hk; h0 += parts * U) {
                fetch_rows(r, v_from, a.vs.h, a.Hk, h0);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (place >= 0 && h0 + u * parts < a.Hk)
                        put(to + ((size_t)(h0 + u * parts) << a.page_log2) * D, r[u]);
            }
        }
    }
}

template <typename E, int D>
cudaError_t launch(RopeArgs &a, cudaStream_t stream) {
    // as many tokens at once as leave two CTAs for every SM
    constexpr int ROWS = NT / (D / 8);
    a.tokens = 1;
    while (a.tokens < ROWS && (a.total + a.tokens - 1) / a.tokens > 304) a.tokens *= 2;
    const int groups = (a.total + a.tokens - 1) / a.tokens;
    const int most = 152 * kCtas<E>;
    const int grid = groups < most ? groups : most;
    const bool pairs = a.maps.flags & LR_QK_INTERLEAVED;
    if (a.maps.rot == 0) qk_norm_rope_kernel<E, D, kNone, false><<<grid, NT, 0, stream>>>(a);
    else if (a.axes && pairs) qk_norm_rope_kernel<E, D, kPairs, true><<<grid, NT, 0, stream>>>(a);
    else if (a.axes) qk_norm_rope_kernel<E, D, kHalves, true><<<grid, NT, 0, stream>>>(a);
    else if (pairs) qk_norm_rope_kernel<E, D, kPairs, false><<<grid, NT, 0, stream>>>(a);
    else qk_norm_rope_kernel<E, D, kHalves, false><<<grid, NT, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_d(RopeArgs &a, int d, cudaStream_t stream) {
    if (d == 32) return launch<E, 32>(a, stream);
    if (d == 64) return launch<E, 64>(a, stream);
    return launch<E, 128>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const void *q, lr_strides qs, const void *k, lr_strides ks,
                                const int *positions, const QkAxes &axes, const QkMaps &maps,
                                void *q_out, void *k_out, const void *v, lr_strides vs,
                                const lr_paged *cache, int B, int T, int Hq, int Hk, int d,
                                lr_dtype dt, cudaStream_t stream) {
    RopeArgs a{};
    a.turns = axes.positions, a.axis = axes.axis, a.axes = axes.count;
    a.q = q, a.k = k, a.v = v, a.qo = q_out, a.ko = k_out;
    a.positions = positions;
    a.qs = qs, a.ks = ks, a.vs = vs;
    a.maps = maps;
    a.T = T, a.Hq = Hq, a.Hk = Hk;
    if (cache) {
        a.ck = cache->k, a.cv = cache->v, a.table = cache->table;
        a.num_pages = cache->num_pages, a.max_pages = cache->max_pages;
        while ((1 << a.page_log2) < cache->page) ++a.page_log2;
    }
    a.total = B * T;
    return dt == LR_DT_F32 ? launch_d<float>(a, d, stream) : launch_d<__nv_bfloat16>(a, d, stream);
}

int attn_errors_rope() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_rope_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
