// lr_fwd_window in fp32 on CUDA cores: one pass over the keys of a 64-row tile with
// the running maximum and sum of the softmax.
//
// A CTA of 256 threads holds 64 query rows of one head.  For each tile of 64
// keys it forms the 64 x 64 scores (a 4 x 4 block per thread), updates the
// rows' maximum and sum, and accumulates the 64 x d output in registers (4
// rows x d / 16 columns per thread).  Tiles that no row of the CTA sees are
// skipped: it walks the sink keys' tiles, then those of the window.
#include "attn_internal.cuh"
#include "attn_rows.cuh"

namespace lr {
namespace {

__device__ unsigned g_window_error = 0;

constexpr int BQ = 64, BK = 64, NT = 256;
constexpr int RS = BQ + 4;  // fp32 row of the transposed tiles: channel c of row r at [c * RS + r]

template <int D>
struct Smem {
    float qt[D * RS];   // scaled queries, transposed
    float kt[D * RS];   // keys, transposed
    float v[BK * D];    // values
    float pt[BK * RS];  // weights, transposed: [key][row]
};

// Rows [r0, r0 + 64) of a strided tensor, transposed into t; rows outside
// [0, n) are zeros.
template <typename E, int D>
__device__ __forceinline__ void load_t(float *t, const E *src, long long st, int r0, int n,
                                       float f) {
    for (int i = threadIdx.x; i < BK * (D / 4); i += NT) {
        const int r = i & (BK - 1), c = (i / BK) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < n) x = load4(src + (long long)(r0 + r) * st + c);
        t[(c + 0) * RS + r] = x.x * f;
        t[(c + 1) * RS + r] = x.y * f;
        t[(c + 2) * RS + r] = x.z * f;
        t[(c + 3) * RS + r] = x.w * f;
    }
}

template <typename E, int D>
__global__ void __launch_bounds__(NT) window_simt_kernel(WindowArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    constexpr int CV = D / 16;  // output columns of a thread: tx + 16 j
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

    const int tiles = (a.Tq + BQ - 1) / BQ;
    // the last rows see the most keys: they start first
    const int bh = blockIdx.x / tiles, tile = tiles - 1 - (blockIdx.x - bh * tiles);
    const int b = bh / a.Hq, h = bh - b * a.Hq, hk = h / (a.Hq / a.Hk);
    bool bad = false;
    const int ql = clamp_len(a.q_len, b, a.Tq, &bad), kl = clamp_len(a.k_len, b, a.Tk, &bad);
    if (bad && tid == 0) atomicOr(&g_window_error, kAttnIndex);
    const int i0 = tile * BQ;
    if (i0 >= ql) return;
    const int p0 = kl - ql + i0;
    const E *q = static_cast<const E *>(a.q) + b * a.qs.b + h * a.qs.h;
    const E *k = static_cast<const E *>(a.k) + b * a.ks.b + hk * a.ks.h;
    const E *v = static_cast<const E *>(a.v) + b * a.vs.b + hk * a.vs.h;
    E *o = static_cast<E *>(a.o) + b * a.os.b + h * a.os.h;
    const int rows = min(BQ, ql - i0);

    load_t<E, D>(sm.qt, q, a.qs.t, i0, ql, a.scale);
    float acc[4][CV], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < CV; ++j) acc[i][j] = 0.f;
    }

    // the keys that the tile's first and last rows see bound those of all
    const SeenKeys first = seen_keys(p0, kl, a.window, a.sinks);
    const SeenKeys last = seen_keys(p0 + rows - 1, kl, a.window, a.sinks);
    const int sink_tiles = (min(last.s1, first.lo) + BK - 1) / BK;
    const int k_first = max(first.lo / BK, sink_tiles);
    const int k_tiles = last.hi > k_first * BK ? (last.hi - k_first * BK + BK - 1) / BK : 0;
    for (int it = 0; it < sink_tiles + k_tiles; ++it) {
        const int j0 = (it < sink_tiles ? it : it - sink_tiles + k_first) * BK;
        __syncthreads();
        load_t<E, D>(sm.kt, k, a.ks.t, j0, kl, 1.f);
        for (int i = tid; i < BK * (D / 4); i += NT) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + r < kl) x = load4(v + (long long)(j0 + r) * a.vs.t + c);
            *reinterpret_cast<float4 *>(&sm.v[r * D + c]) = x;
        }
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 8
        for (int c = 0; c < D; ++c) {
            const float4 x = *reinterpret_cast<const float4 *>(&sm.qt[c * RS + 4 * ty]);
            const float4 y = *reinterpret_cast<const float4 *>(&sm.kt[c * RS + 4 * tx]);
            const float xr[4] = {x.x, x.y, x.z, x.w}, yr[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] += xr[i] * yr[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * ty + i;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + 4 * tx + j;
                const bool seen = key <= p && key < kl && (p - key < a.window || key < a.sinks);
                if (!seen) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
            const float c = __expf(m[i] - base);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = __expf(s[i][j] - base);
                sum += e;
                sm.pt[(4 * tx + j) * RS + 4 * ty + i] = e;
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * c + sum;
#pragma unroll
            for (int j = 0; j < CV; ++j) acc[i][j] *= c;
        }
        __syncthreads();
#pragma unroll 4
        for (int r = 0; r < BK; ++r) {
            const float4 x = *reinterpret_cast<const float4 *>(&sm.pt[r * RS + 4 * ty]);
            const float xr[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < CV; ++j) {
                const float y = sm.v[r * D + tx + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] += xr[i] * y;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no key, or only scores of -inf
        bool finite = true;
#pragma unroll
        for (int j = 0; j < CV; ++j) {
            acc[i][j] *= inv;
            finite = finite && isfinite(acc[i][j]);
        }
        // rows of both half warps, decided by all lanes
        const unsigned oddity = __ballot_sync(0xffffffffu, r < rows && !finite);
        if (r < rows) {
#pragma unroll
            for (int j = 0; j < CV; ++j)
                o[(long long)(i0 + r) * a.os.t + tx + 16 * j] = from_f<E>(acc[i][j]);
        }
        if (oddity) {
            __syncwarp();
            const int w0 = 8 * (tid >> 5);  // first row of this warp
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                if (!(oddity & (0xffffu << (16 * g)))) continue;
                const int rr = w0 + 4 * g + i;
                attn_row<E, D>(q + (long long)(i0 + rr) * a.qs.t, k, v, a.ks.t, a.vs.t,
                               o + (long long)(i0 + rr) * a.os.t,
                               seen_keys(p0 + rr, kl, a.window, a.sinks), a.scale);
            }
        }
    }
}

template <typename E, int D>
cudaError_t launch(const WindowArgs &a, int slot, cudaStream_t stream) {
    auto *fn = window_simt_kernel<E, D>;
    const cudaError_t e =
        ensure_smem_attr(reinterpret_cast<const void *>(fn), sizeof(Smem<D>), slot);
    if (e != cudaSuccess) return e;
    const int tiles = (a.Tq + BQ - 1) / BQ;
    fn<<<(unsigned)(a.B * a.Hq * tiles), NT, sizeof(Smem<D>), stream>>>(a);
    return cudaGetLastError();
}

constexpr int kSlot = 208;  // ensure_smem_attr slots 208..210

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

cudaError_t launch_window_simt(const WindowArgs &a, int d, cudaStream_t stream) {
    if (d == 32) return launch<float, 32>(a, kSlot, stream);
    if (d == 64) return launch<float, 64>(a, kSlot + 1, stream);
    return launch<float, 128>(a, kSlot + 2, stream);
}

cudaError_t launch_window_zero(const WindowArgs &a, int d, lr_dtype dt, cudaStream_t stream) {
    const int units = d * (dt == LR_DT_F32 ? 4 : 2) / 16;  // 16-byte units of a row
    const long long n = (long long)a.B * a.Hq * a.Tq * units;
    const unsigned grid = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
    if (dt == LR_DT_F32) window_zero_kernel<float><<<grid, 256, 0, stream>>>(a, units, n);
    else window_zero_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, units, n);
    return cudaGetLastError();
}

int attn_errors_window_simt() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_window_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_window_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
