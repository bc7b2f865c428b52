// lr_step_paged: attention of one new token per sequence over a paged cache.
//
// The keys that a sequence sees (its sinks, then its window) form one list,
// cut into chunks.  One CTA takes one chunk of one sequence and key head for
// up to GC of the query heads that share it, so a chunk's keys and values are
// read once for them.  Inside the CTA every group of d / 8 lanes takes keys
// of its own, with a running maximum and sum of its own; the groups are
// joined through shuffles and shared memory at the end.  With one chunk per
// sequence the CTA writes the output; otherwise it writes (maximum, sum,
// unnormalised output) to the workspace and a second kernel joins the chunks
// in order.
#include "attn_internal.cuh"

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
};

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)),
                 b = __ldg(reinterpret_cast<const float4 *>(p + 4));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// exp(m - base) with an empty part's maximum of -inf
__device__ __forceinline__ float part_weight(float m, float base) {
    return m == -INFINITY ? 0.f : __expf(m - base);
}

template <typename E, int D, int GC>
__global__ void __launch_bounds__(NT) step_simt_kernel(StepArgs a, Parts parts) {
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
    if (len < 0) return;
    if (len > a.max_len) {
        if (tid == 0 && split == 0 && gi == 0 && hk == 0) atomicOr(&g_step_error, kAttnIndex);
        return;
    }
    const SeenKeys s = seen_keys(len - 1, len, a.window, a.sinks);
    const int seen = s.s1 + s.hi - s.lo;
    const int c0 = split * parts.chunk;
    if (c0 >= seen && split > 0) return;  // the join knows how many chunks there are
    const int c1 = min(seen, c0 + parts.chunk);
    const int h0 = hk * G + gi * GC, heads = min(GC, G - gi * GC);
    const int lane = tid % LANES, group = tid / LANES, ch = lane * 8;

    const E *qn = static_cast<const E *>(a.q) + (size_t)n * a.Hq * D;
    float q[GC][8], acc[GC][8], m[GC], l[GC];
#pragma unroll
    for (int g = 0; g < GC; ++g) {
        load8(qn + (size_t)(h0 + min(g, heads - 1)) * D + ch, q[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[g][i] *= a.scale, acc[g][i] = 0.f;
        m[g] = -INFINITY, l[g] = 0.f;
    }
    const int *table = a.table + (size_t)n * a.max_pages;
    const int in_page = (1 << a.page_log2) - 1;
    const int lanes0 = (tid & 31) / LANES * LANES;
    const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1) << lanes0;
    bool bad = false;
    for (int base = c0 + group; base < c1; base += GROUPS * U) {
        long long row[U];
        float x[U][8], sc[U][GC];
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
            for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
            if (row[u] >= 0) load8(static_cast<const E *>(a.k) + row[u], x[u]);
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
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
            if (row[u] >= 0) load8(static_cast<const E *>(a.v) + row[u], x[u]);
        }
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            float mn = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) mn = fmaxf(mn, sc[u][g]);
            const float b = mn == -INFINITY ? 0.f : mn;
            const float c = __expf(m[g] - b);
            m[g] = mn;
            l[g] *= c;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[g][i] *= c;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p = __expf(sc[u][g] - b);
                l[g] += p;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[g][i] += p * x[u][i];
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
        const float c = part_weight(m[g], mn);
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
    __syncthreads();
    for (int i = tid; i < heads * D; i += NT) {
        const int g = i / D, c = i - g * D;
        float mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) mn = fmaxf(mn, sml[w][g][0]);
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const float f = part_weight(sml[w][g][0], mn);
            sum += f * sml[w][g][1];
            x += f * so[w][g][c];
        }
        const size_t r = (size_t)n * a.Hq + h0 + g;
        if (parts.splits == 1) {
            static_cast<E *>(a.o)[r * D + c] = from_f<E>(sum == 0.f ? 0.f : x / sum);
        } else {
            parts.o[(r * parts.splits + split) * D + c] = x;
            if (c == 0) parts.ml[r * parts.splits + split] = make_float2(mn, sum);
        }
    }
}

// One CTA of D threads per output row: the chunks' parts in order.
template <typename E, int D>
__global__ void __launch_bounds__(D) step_join_kernel(StepArgs a, Parts parts) {
    const int r = blockIdx.x, n = r / a.Hq, c = threadIdx.x;
    const int len = a.lens[n];
    if (len < 0 || len > a.max_len) return;
    const SeenKeys s = seen_keys(len - 1, len, a.window, a.sinks);
    const int seen = s.s1 + s.hi - s.lo;
    const int used = max(1, (seen + parts.chunk - 1) / parts.chunk);
    const float2 *ml = parts.ml + (size_t)r * parts.splits;
    const float *po = parts.o + (size_t)r * parts.splits * D + c;
    float m = -INFINITY, l = 0.f, x = 0.f;
    for (int i = 0; i < used; ++i) {
        const float2 t = ml[i];
        const float y = po[(size_t)i * D];
        const float mn = fmaxf(m, t.x);
        const float f = part_weight(m, mn), g = part_weight(t.x, mn);
        l = l * f + t.y * g;
        x = x * f + y * g;
        m = mn;
    }
    static_cast<E *>(a.o)[(size_t)r * D + c] = from_f<E>(l == 0.f ? 0.f : x / l);
}

Parts parts_of(const StepArgs &a, int d, const StepPlan &p, void *ws) {
    Parts r{};
    r.splits = p.splits, r.chunk = p.chunk;
    if (p.splits > 1) {
        r.o = static_cast<float *>(ws);
        r.ml = reinterpret_cast<float2 *>(r.o + (size_t)a.N * a.Hq * p.splits * d);
    }
    return r;
}

template <typename E, int D>
cudaError_t launch(const StepArgs &a, void *ws, lr_dtype dt, cudaStream_t stream) {
    const StepPlan p = step_plan(a.N, a.Hq, a.Hk, a.max_len, a.window, a.sinks, dt);
    const Parts parts = parts_of(a, D, p, ws);
    const int G = a.Hq / a.Hk;
    const int gc = G == 1 ? 1 : G == 2 ? 2 : 4;
    const unsigned grid = (unsigned)(a.N * a.Hk * ((G + gc - 1) / gc) * p.splits);
    if (gc == 1) step_simt_kernel<E, D, 1><<<grid, NT, 0, stream>>>(a, parts);
    else if (gc == 2) step_simt_kernel<E, D, 2><<<grid, NT, 0, stream>>>(a, parts);
    else step_simt_kernel<E, D, 4><<<grid, NT, 0, stream>>>(a, parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    step_join_kernel<E, D><<<(unsigned)(a.N * a.Hq), D, 0, stream>>>(a, parts);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_d(const StepArgs &a, int d, void *ws, lr_dtype dt, cudaStream_t stream) {
    if (d == 32) return launch<E, 32>(a, ws, dt, stream);
    if (d == 64) return launch<E, 64>(a, ws, dt, stream);
    return launch<E, 128>(a, ws, dt, stream);
}

}  // namespace

StepPlan step_plan(int N, int Hq, int Hk, int max_len, int window, int sinks, lr_dtype dt) {
    (void)dt;
    (void)Hq;
    const long long w = (long long)window + sinks;
    const int seen = w < max_len ? (int)w : max_len;
    // about four CTAs per SM in all, chunks of 128 to 2048 keys
    const long long rows = (long long)N * Hk;
    const long long want = (608 + rows - 1) / rows;
    long long chunk = (seen + want - 1) / want;
    chunk = (chunk + 63) / 64 * 64;
    if (chunk < 128) chunk = 128;
    if (chunk > 2048) chunk = 2048;
    StepPlan p;
    p.chunk = (int)chunk;
    p.splits = (seen + p.chunk - 1) / p.chunk;
    return p;
}

size_t step_workspace_bytes(int N, int Hq, int d, const StepPlan &p) {
    if (p.splits <= 1) return 0;
    return (size_t)N * Hq * p.splits * ((size_t)d * 4 + 8);
}

cudaError_t launch_step_paged(const StepArgs &a, int d, lr_dtype dt, void *ws, cudaStream_t stream) {
    return dt == LR_DT_F32 ? launch_d<float>(a, d, ws, dt, stream)
                           : launch_d<__nv_bfloat16>(a, d, ws, dt, stream);
}

int attn_errors_step() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_step_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_step_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
