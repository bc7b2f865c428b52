// What the two tensor-core kernels of differential attention share: the pieces of
// work (128 query rows of a pair of heads), their order, and rows put right.
#pragma once

#include <algorithm>

#include "attn_diff.cuh"
#include "attn_internal.cuh"
#include "attn_rows.cuh"
#include "attn_tc.cuh"

namespace lr {

constexpr int kDiffRows = 128, kDiffKeys = 128;

struct DiffTcArgs {
    DiffArgs a;
    float c;          // the scores' factor, positive
    unsigned negate;  // idesc bit: scores of -Q (scale < 0)
    int group;        // pairs of heads that share keys
    int tiles;        // row blocks of a pair
    int span;         // pairs of all batches that are worked on together
    int pieces;
};

// A piece of work, kept in shared memory.  Key tile `it` is a sink tile (it <
// sink_tiles), whose keys all rows see, or window tile it - sink_tiles; those
// that all rows see entirely form one run [all0, all1).
struct DiffItem {
    int b, h, hk, i0, rows, p0, kl;
    int all0, all1, sink_keys, sink_tiles, lo, hi;
    int n;      // key tiles; 0: no rows
    int valid;  // 0: no work is left

    __device__ __forceinline__ int key0(int it) const {
        return it < sink_tiles ? it * kDiffKeys : lo + (it - sink_tiles) * kDiffKeys;
    }
    __device__ __forceinline__ int limit(int it) const { return it < sink_tiles ? sink_keys : hi; }
    // columns that the tile needs, a multiple of 32
    __device__ __forceinline__ int width(int it) const {
        const int w = limit(it) - key0(it);
        return w >= kDiffKeys ? kDiffKeys : (w < 32 ? 32 : (w + 31) & ~31);
    }
};
static_assert(sizeof(DiffItem) <= 128, "shared memory layout");

__device__ __forceinline__ void make_diff_item(const DiffTcArgs &g, int block, DiffItem &x, bool *bad) {
    const DiffArgs &a = g.a;
    // the last rows see the most keys: of the pairs whose keys and values the L2
    // cache holds together, all longest tiles start first
    const unsigned size = g.span * g.tiles, span = (unsigned)block / size, in = block - span * size;
    const unsigned wide = min(g.span, a.B * a.H - (int)span * g.span), deep = in / wide;
    const int tile = g.tiles - 1 - (int)deep, bh = span * g.span + in - deep * wide;
    x.b = (unsigned)bh / (unsigned)a.H;
    x.h = bh - x.b * a.H;
    x.hk = (unsigned)x.h / (unsigned)g.group;
    const int ql = clamp_len(a.q_len, x.b, a.Tq, bad), kl = clamp_len(a.k_len, x.b, a.Tk, bad);
    x.kl = kl;
    x.i0 = tile * kDiffRows;
    x.rows = max(0, min(kDiffRows, ql - x.i0));
    x.p0 = kl - ql + x.i0;
    const SeenKeys f = seen_keys(x.p0, kl, a.window, a.sinks),
                   e = seen_keys(x.p0 + x.rows - 1, kl, a.window, a.sinks);
    x.lo = f.lo, x.hi = e.hi;
    x.sink_keys = min(e.s1, f.lo);
    x.sink_tiles = (x.sink_keys + kDiffKeys - 1) / kDiffKeys;
    x.n = x.sink_tiles + (x.hi > x.lo ? (x.hi - x.lo + kDiffKeys - 1) / kDiffKeys : 0);
    // no key for any row: one tile with everything masked gives the zeros
    x.n = x.rows > 0 ? max(x.n, 1) : 0;
    // positions and keys lie within +-2^30, so differences of two fit an int
    const int far = x.p0 + kDiffRows - min(a.window, 1 << 30) - x.lo;  // first key of the last row
    x.all0 = x.sink_tiles + (far > 0 ? (far + kDiffKeys - 1) / kDiffKeys : 0);
    const int end = min(x.hi, x.p0 + 1) - x.lo;
    x.all1 = x.sink_tiles + (end > 0 ? end / kDiffKeys : 0);
}

// What follows the difference of a row, for the sum of its squares (`squares`; of the
// thread's own values where there is no norm): NaN for a row that is to be put right.  Such
// a row leaves as NaN in all of its channels, which marks it for mend_marked.
__device__ __forceinline__ float diff_scale(bool norm, float squares, int d, float eps) {
    return norm ? diff_rms(squares, d, eps) : (squares == squares ? 1.f : NAN);
}
// The squares' sum of N values: NaN where one of them is not finite.  Squares of finite
// values may pass the range; the row is then divided by infinity, as the formula has it.
template <int N>
__device__ __forceinline__ float marked_squares(const float (&y)[N], float squares) {
    if (squares < INFINITY) return squares;
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) odd = fmaf(y[i], 0.f, odd);
    return odd == 0.f ? INFINITY : NAN;
}

// Rows that the pieces of this CTA (or cluster), number `me` of `all`, left marked, put
// right by its eight softmax warps.  It comes last, when no other warp waits for these in
// a loop that gives up: a row takes two passes over its keys.  Warp w of warpgroup t wrote
// rows 32 w .. 32 w + 31 of each piece, channels c0 + t n .. of n; here the warpgroups take
// every other of these rows, with both their channels.  marked: the warp left such a row.
template <int D>
__device__ __forceinline__ void mend_marked(const DiffTcArgs &g, bool marked, int me, int all, int c0, int n) {
    using E = __nv_bfloat16;
    constexpr int PL = D / 32;
    const DiffArgs &a = g.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row0 = 32 * (warp & 3);
    uint32_t some;  // of all eight, which are through with their pieces
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(some)
        : "r"((uint32_t)marked)
        : "memory");
    if (!some) return;
#pragma unroll 1
    for (int i = 0;; ++i) {
        const long long block = (long long)i * all + (i & 1 ? all - 1 - me : me);
        if (block >= g.pieces) break;
        bool bad = false;
        DiffItem x;
        make_diff_item(g, (int)block, x, &bad);
        E *o = static_cast<E *>(a.o) + x.b * a.os.b + 2 * x.h * a.os.h + (long long)(x.i0 + row0) * a.os.t;
        // a mark for either warpgroup's channels
        bool odd[2] = {false, false};
        if (row0 + lane < x.rows && (lane & 1) == warp >> 2)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int ch = c0 + t * n;
                const float mark = to_f<E>(o[ch / D * a.os.h + lane * a.os.t + ch % D]);
                odd[t] = mark != mark;
            }
        const unsigned again[2] = {__ballot_sync(0xffffffffu, odd[0]), __ballot_sync(0xffffffffu, odd[1])};
        unsigned rows = again[0] | again[1];
#pragma unroll 1
        while (rows) {
            const int row = __ffs(rows) - 1;
            rows &= rows - 1;
            const bool put[2] = {(again[0] >> row & 1u) != 0, (again[1] >> row & 1u) != 0};
            const E *q = static_cast<const E *>(a.q) + x.b * a.qs.b + 2 * x.h * a.qs.h +
                         (long long)(x.i0 + row0 + row) * a.qs.t;
            const E *k = static_cast<const E *>(a.k) + x.b * a.ks.b + 2 * x.hk * a.ks.h;
            const E *v = static_cast<const E *>(a.v) + x.b * a.vs.b + 2 * x.hk * a.vs.h;
            float y[2][PL];
            mend_diff<E, D>(
                q, q + a.qs.h,
                [&](int map, int half, int j, const E *&kj, const E *&vj) {
                    kj = k + map * a.ks.h + j * a.ks.t, vj = v + half * a.vs.h + j * a.vs.t;
                    return true;
                },
                a.lambda[x.h], a.norm, a.weight, a.eps, seen_keys(x.p0 + row0 + row, x.kl, a.window, a.sinks),
                score_factor(a.scale), (put[0] ? 1u << c0 / D : 0u) | (put[1] ? 1u << (c0 + n) / D : 0u), y);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int c = 0; c < PL; ++c) {
                    const int in = lane * PL + c, ch = half * D + in - c0;  // of the CTA's 2 n
                    if (ch >= 0 && ch < 2 * n && put[ch >= n]) o[half * a.os.h + row * a.os.t + in] = from_f<E>(y[half][c]);
                }
        }
    }
}

inline DiffTcArgs diff_tc_args(const DiffArgs &a, int d) {
    DiffTcArgs g;
    g.a = a;
    // scale 0: as in window_tc.cu
    g.c = a.scale == 0.f ? 0x1p-149f : score_factor(a.scale).c;
    g.negate = a.scale < 0.f ? 1u << 13 : 0u;
    g.group = a.H / a.Hk;
    g.tiles = (a.Tq + kDiffRows - 1) / kDiffRows;
    // keys and values of the pairs in flight stay within 48 MB of the L2's 129
    const long long kv = 8ll * d * a.Tk, pairs = (long long)a.B * a.H;
    const long long span = (48ll << 20) / kv;
    g.span = (int)(span < 1 ? 1 : (span < pairs ? span : pairs));
    g.pieces = (int)(pairs * g.tiles);
    return g;
}

}  // namespace lr
