// Declarations shared by the attention translation units of liblr (the
// operators of include/lr_attn.h).
#pragma once

#include "lr_attn.h"
#include "lr_internal.cuh"

namespace lr {

// Error word of the attention kernels: bits set by any of them, read and
// cleared by lr_device_status.  Each translation unit has its own copy in its
// module; attn_errors() collects them.
constexpr unsigned kAttnIndex = 1u;    // a page or a length out of range
constexpr unsigned kAttnTimeout = 2u;  // a bounded wait gave up

// Keys that the query at position p sees: [0, s1) and [lo, hi), with
// s1 <= lo (lo == 0 or s1 == 0 where one run covers all).
struct SeenKeys {
    int s1, lo, hi;
};
__host__ __device__ __forceinline__ SeenKeys seen_keys(int p, int klen, int window, int sinks) {
    SeenKeys s;
    s.hi = p + 1 < klen ? p + 1 : klen;
    if (s.hi < 0) s.hi = 0;
    const long long l = (long long)p - window + 1;
    s.lo = l < 0 ? 0 : (int)l;
    if (s.lo > s.hi) s.lo = s.hi;
    s.s1 = sinks < s.lo ? sinks : s.lo;
    return s;
}

// Lengths as the kernels use them; *bad when one was out of range.
__device__ __forceinline__ int clamp_len(const int *len, int b, int most, bool *bad) {
    if (!len) return most;
    const int x = len[b];
    if (x < 0 || x > most) *bad = true;
    return x < 0 ? 0 : (x > most ? most : x);
}

// A score enters as sign * (q . k), formed in fp32 before any scale, and its
// weight is 2^(c (score - maximum)): no finite scale can push a finite score
// out of range.  Scale 0 gives sign 0: scores of zero, so that masked ones can
// stay -inf (their product with a factor of 0 would be NaN).
struct ScoreFactor {
    float sign, c;
};
__host__ __device__ __forceinline__ ScoreFactor score_factor(float scale) {
    // scale 0: all scores are zero, whatever c is
    return {scale > 0.f ? 1.f : (scale < 0.f ? -1.f : 0.f),
            scale == 0.f ? 1.f : fminf(fabsf(scale) * 1.4426950408889634f, 3.402823466e38f)};
}

// ------------------------------------------------------------------ arithmetic
// 2^x, results below the normal range zero
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// two values rounded to bf16, `lo` in the lower half
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

struct QkMaps {
    const float *qw, *kw;
    const double *inv_freq;
    float eps;
    int rot;
    unsigned flags;
};

// ------------------------------------------------------------------ launchers
cudaError_t launch_qk_norm_rope(const void *q, lr_strides qs, const void *k, lr_strides ks,
                                const int *positions, const QkMaps &maps, void *q_out, void *k_out,
                                const void *v, lr_strides vs, const lr_paged *cache, int B, int T,
                                int Hq, int Hk, int d, lr_dtype dt, cudaStream_t stream);

constexpr int kMostCluster = 8;  // CTAs of the largest cluster that is always allowed
// CTAs of clusters of 1, 2, .. 8 that find room on the GPU at once with one to
// four of them on an SM (the occupancy calculator's answers on a GPU of 152 SMs:
// a cluster stays within one of the GPU's groups of SMs, which it does not
// always fill).  Another chip may have other SMs of a group switched off: plans
// then meet a second round that they meant to avoid, and results stay the same.
// A table, so that plans and workspace sizes need no device.
constexpr int kClusterRoom[4][kMostCluster + 1] = {{0, 152, 152, 138, 144, 140, 138, 105, 120},
                                                   {0, 304, 304, 291, 296, 290, 276, 266, 288},
                                                   {0, 456, 456, 444, 440, 435, 444, 413, 408},
                                                   {0, 608, 608, 582, 592, 585, 582, 567, 592}};

struct WindowArgs {
    const void *q, *k, *v;
    void *o;
    lr_strides qs, ks, vs, os;
    const int *q_len, *k_len;
    int B, Hq, Hk, Tq, Tk, window, sinks;
    float scale;
};
// fp32, Tk >= 1 (window_f32.cu).
cudaError_t launch_window_f32(const WindowArgs &a, int d, cudaStream_t stream);
// Tensor cores, bf16, Tk >= 1 (window_tc.cu).
cudaError_t launch_window_tc(const WindowArgs &a, int d, cudaStream_t stream);
// Zeros in every row that is written (Tk == 0), either type (window_f32.cu).
cudaError_t launch_window_zero(const WindowArgs &a, int d, lr_dtype dt, cudaStream_t stream);

struct StepArgs {
    const void *q, *k, *v;
    void *o;
    const int *table, *lens;
    int N, Hq, Hk, max_len, window, sinks, num_pages, page_log2, max_pages;
    float scale;
    int fill;  // rows that are not computed are zeros
};
// How a step's keys are cut: chunks of `chunk` keys, at most `splits` of them,
// joined by a cluster or by a second kernel.
struct StepPlan {
    int chunk, splits;
    bool cluster;
};
StepPlan step_plan(int N, int Hq, int Hk, int d, int max_len, int window, int sinks, lr_dtype dt);
size_t step_workspace_bytes(int N, int Hq, int d, const StepPlan &p);
cudaError_t launch_step_paged(const StepArgs &a, int d, lr_dtype dt, void *ws, cudaStream_t stream);

// Return and clear the error bits of each unit (-1: the device could not be read).
int attn_errors_rope();
int attn_errors_window_f32();
int attn_errors_window_tc();
int attn_errors_step();

}  // namespace lr
