// lr_qk_norm_rope: RMS norm of each query and key head, the position rotation
// and the write of keys and values into a paged cache, in one pass.
//
// A row (one head of one token) is held by d / 8 lanes of a warp, eight
// channels each, so that its sum of squares and the partner channels of the
// split-half rotation come from shuffles.  The angles of a token are the same
// for all its heads: a CTA takes a few tokens, forms their cosines and sines
// once in shared memory and then streams the rows of all their heads.
//
// Angle: th = p f.  With s = frac(f / 2 pi) as a 64-bit fixed-point fraction
// of a turn, p s mod 2^64 is the exact fraction of the product, so the only
// errors are those of s (2^-53 relative) and of the final fp32 conversion
// (2^-25 of a half turn), whatever the position.
#include "attn_internal.cuh"

namespace lr {
namespace {

__device__ unsigned g_rope_error = 0;

constexpr int NT = 256;
constexpr int kMostTokens = 16;  // tokens of one CTA

struct RopeArgs {
    const void *q, *k, *v;
    void *qo, *ko, *ck, *cv;
    const int *positions, *table;
    lr_strides qs, ks, vs;
    QkMaps maps;
    int T, Hq, Hk, num_pages, page_log2, max_pages;
    int tokens;  // per CTA
    int rows;    // rows of a token: Hq + Hk (+ Hk values with a cache)
    int total;   // B * T
};

// Eight consecutive channels as fp32.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

template <typename E, int D>
__global__ void __launch_bounds__(NT) qk_norm_rope_kernel(RopeArgs a) {
    constexpr int LANES = D / 8;       // lanes of a row
    constexpr int ROWS = NT / LANES;   // rows in flight
    __shared__ float2 cs[kMostTokens][D / 2];
    __shared__ int pos[kMostTokens];
    __shared__ long long slot[kMostTokens];  // first cache row of the token (head 0), -1: none
    const int tid = threadIdx.x;
    const int n0 = blockIdx.x * a.tokens;
    const int nt = min(a.tokens, a.total - n0);
    const int half = a.maps.rot >> 1;

    for (int i = tid; i < nt; i += NT) {
        const int n = n0 + i, b = n / a.T;
        const int p = a.positions ? a.positions[n] : n - b * a.T;
        pos[i] = p;
        long long s = -1;
        if (a.ck && p >= 0) {
            const int pg = p >> a.page_log2;
            const int page = pg < a.max_pages ? a.table[(size_t)b * a.max_pages + pg] : -1;
            if (page >= 0 && page < a.num_pages)
                s = (((long long)page * a.Hk) << a.page_log2) + (p & ((1 << a.page_log2) - 1));
            else
                atomicOr(&g_rope_error, kAttnIndex);
        }
        slot[i] = s;
    }
    __syncthreads();
    if (half) {
        for (int i = tid; i < nt * half; i += NT) {
            const int t = i / half, c = i - t * half;
            double turns = a.maps.inv_freq[c] * 0.15915494309189533577;  // 1 / (2 pi)
            turns -= floor(turns);
            const unsigned long long step = __double2ull_rz(turns * 18446744073709551616.0);
            const unsigned long long phase = step * (unsigned long long)(long long)pos[t];
            // signed half turns in [-1, 1)
            const float x = (float)(int)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
            float sn, cn;
            sincospif(x, &sn, &cn);
            cs[t][c] = make_float2(cn, sn);
        }
    }
    __syncthreads();

    const int lane = tid % LANES, c0 = lane * 8;
    const int r0 = blockIdx.y * ROWS + tid / LANES;
    // every lane of a warp takes part in the shuffles: rows past the end compute nothing kept
    const int all = nt * a.rows;
    const int step = gridDim.y * ROWS;
    for (int base = 0; base < all; base += step) {
        const int r = base + r0;
        const bool live = r < all;
        const int head = live ? r / nt : 0, t = live ? r - head * nt : 0;
        const int n = n0 + t, b = n / a.T, tt = n - b * a.T;
        const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hk;
        const int h = is_q ? head : (is_v ? head - a.Hq - a.Hk : head - a.Hq);
        const bool on = live && pos[t] >= 0;
        const lr_strides &st = is_q ? a.qs : (is_v ? a.vs : a.ks);
        const E *src = static_cast<const E *>(is_q ? a.q : (is_v ? a.v : a.k)) + b * st.b +
                       h * st.h + tt * st.t + c0;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on) load8(src, x);
        if (a.maps.flags & LR_QK_NORM) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
            for (int m = 1; m < LANES; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            if (!is_v) {
                const float inv = 1.f / sqrtf(ss * (1.f / D) + a.maps.eps);
                const float *w = is_q ? a.maps.qw : a.maps.kw;
                float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
                if (w) load8(w + c0, wv);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= inv * wv[i];
            }
        }
        if (half) {
            if (a.maps.flags & LR_QK_INTERLEAVED) {
                if (!is_v && c0 < a.maps.rot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = cs[t][(c0 >> 1) + i];
                        const float u = x[2 * i], w = x[2 * i + 1];
                        x[2 * i] = u * f.x - w * f.y;
                        x[2 * i + 1] = w * f.x + u * f.y;
                    }
                }
            } else {
                // the partner channel c +- half sits half / 8 lanes away
                const int hl = half >> 3;
                const bool lo = c0 < half;
                const int from = (tid & 31) + (c0 < a.maps.rot ? (lo ? hl : -hl) : 0);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = __shfl_sync(0xffffffffu, x[i], from);
                    if (!is_v && c0 < a.maps.rot) {
                        const float2 f = cs[t][lo ? c0 + i : c0 - half + i];
                        x[i] = lo ? x[i] * f.x - y * f.y : x[i] * f.x + y * f.y;
                    }
                }
            }
        }
        if (!on) continue;
        if (is_q) {
            store8(static_cast<E *>(a.qo) + (((size_t)b * a.Hq + h) * a.T + tt) * D + c0, x);
        } else {
            if (!is_v && a.ko)
                store8(static_cast<E *>(a.ko) + (((size_t)b * a.Hk + h) * a.T + tt) * D + c0, x);
            if (a.ck && slot[t] >= 0)
                store8(static_cast<E *>(is_v ? a.cv : a.ck) +
                           ((size_t)slot[t] + ((size_t)h << a.page_log2)) * D + c0, x);
        }
    }
}

template <typename E>
cudaError_t launch(const RopeArgs &a, int d, cudaStream_t stream) {
    const int gx = (a.total + a.tokens - 1) / a.tokens;
    const int in_flight = NT / (d / 8);
    // few tokens: their rows are spread over more CTAs
    int gy = 1;
    while (gx * gy < 304 && gy * in_flight < a.tokens * a.rows) gy *= 2;
    const dim3 grid(gx, gy);
    if (d == 32) qk_norm_rope_kernel<E, 32><<<grid, NT, 0, stream>>>(a);
    else if (d == 64) qk_norm_rope_kernel<E, 64><<<grid, NT, 0, stream>>>(a);
    else qk_norm_rope_kernel<E, 128><<<grid, NT, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const void *q, lr_strides qs, const void *k, lr_strides ks,
                                const int *positions, const QkMaps &maps, void *q_out, void *k_out,
                                const void *v, lr_strides vs, const lr_paged *cache, int B, int T,
                                int Hq, int Hk, int d, lr_dtype dt, cudaStream_t stream) {
    RopeArgs a{};
    a.q = q, a.k = k, a.v = v, a.qo = q_out, a.ko = k_out;
    a.positions = positions;
    a.qs = qs, a.ks = ks, a.vs = vs;
    a.maps = maps;
    a.T = T, a.Hq = Hq, a.Hk = Hk;
    a.rows = Hq + Hk;
    if (cache) {
        a.ck = cache->k, a.cv = cache->v, a.table = cache->table;
        a.num_pages = cache->num_pages, a.max_pages = cache->max_pages;
        while ((1 << a.page_log2) < cache->page) ++a.page_log2;
        a.rows += Hk;
    }
    a.total = B * T;
    a.tokens = kMostTokens;
    while (a.tokens > 1 && (a.total + a.tokens - 1) / a.tokens < 608) a.tokens /= 2;
    return dt == LR_DT_F32 ? launch<float>(a, d, stream) : launch<__nv_bfloat16>(a, d, stream);
}

int attn_errors_rope() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_rope_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
