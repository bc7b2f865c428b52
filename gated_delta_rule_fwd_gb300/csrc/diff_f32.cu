// lr_fwd_diff in fp32: the two maps of a pair by the fp32 window kernel
// (window_f32.cu), into the workspace in one launch, then one pass that takes the
// difference and its norm (attn_diff.cuh).  At d = 128 the two halves of the value row
// are apart and the scores are formed twice, once for each (8 units of products where 6
// would do): a row's 2 d channels of output leave no registers for both.
//
// Measured: 2 x 350 rows on 1501 keys, 4 pairs, d = 64, window 300: 31.6 us, of them 2 for
// the difference (with the scores formed twice 40.2; 2048 rows of 8 pairs, causal: 240
// and 295).  The bound is that of window_f32.cu, the issue of split products.
#include "attn_diff.cuh"
#include "attn_internal.cuh"

namespace lr {
namespace {

constexpr int NT = 128;

// The maps' outputs in the workspace, row i of a half of map m: [B][H][map][Tq][2 D],
// or [B][H][map][half][Tq][D] at D = 128.
__host__ __device__ constexpr int kept_halves(int d) { return d == 128 ? 2 : 1; }

// A warp per row of a pair.
template <int D>
__global__ void __launch_bounds__(NT) diff_join_kernel(DiffArgs a, const float *maps) {
    constexpr int PL = D / 32;
    constexpr bool APART = kept_halves(D) == 2;
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)a.B * a.H * a.Tq;
    const long long r = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int i = (int)(r % a.Tq), bh = (int)(r / a.Tq), b = bh / a.H, h = bh - b * a.H;
    bool bad = false;  // reported by the maps' own kernels
    if (i >= clamp_len(a.q_len, b, a.Tq, &bad)) return;
    const float lambda = a.lambda[h];
    float y[2][PL], sum = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int c = 0; c < PL; ++c) {
            const float *x = maps + lane + 32 * c +
                             (APART ? (((long long)bh * 4 + half) * a.Tq + i) * D
                                    : ((long long)bh * 2 * a.Tq + i) * 2 * D + half * D);
            y[half][c] = fmaf(-lambda, x[2ll * a.Tq * D], x[0]);
            sum = fmaf(y[half][c], y[half][c], sum);
        }
    const float f = a.norm ? diff_rms(warp_sum(sum), D, a.eps) : 1.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float *o = static_cast<float *>(a.o) + b * a.os.b + (2 * h + half) * a.os.h + i * a.os.t + lane;
#pragma unroll
        for (int c = 0; c < PL; ++c)
            o[32 * c] = y[half][c] * f * (a.norm && a.weight ? a.weight[half * D + lane + 32 * c] : 1.f);
    }
}

template <int D>
void join(const DiffArgs &a, const float *maps, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.H * a.Tq;
    diff_join_kernel<D><<<(unsigned)((rows + NT / 32 - 1) / (NT / 32)), NT, 0, stream>>>(a, maps);
}

}  // namespace

size_t diff_f32_workspace_bytes(int B, int H, int Tq, int d) { return (size_t)B * H * Tq * d * 16; }

cudaError_t launch_diff_f32(const DiffArgs &a, int d, void *ws, cudaStream_t stream) {
    float *maps = static_cast<float *>(ws);
    const int heads = 2 * kept_halves(d), width = 4 * d / heads;  // outputs of a pair, their channels
    WindowArgs w{a.q, a.k, a.v, maps, a.qs, a.ks, a.vs, {}, a.q_len, a.k_len, a.B, heads * a.H, a.Hk, a.Tq, a.Tk,
                 a.window, a.sinks, a.scale, 1};
    w.os = {4ll * a.H * a.Tq * d, (long long)a.Tq * width, width};
    const cudaError_t e = launch_window_f32(w, d, stream);
    if (e != cudaSuccess) return e;
    if (d == 32) join<32>(a, maps, stream);
    else if (d == 64) join<64>(a, maps, stream);
    else join<128>(a, maps, stream);
    return cudaGetLastError();
}

}  // namespace lr
