// lr_fwd_window in bf16 on the tensor cores (tcgen05), one pass over the keys
// with the running maximum and sum of the softmax.
//
// A CTA takes two 128-row query tiles that read the same keys: the same rows
// of two heads that share a key head, or, where the heads of a group are odd
// in number, consecutive rows of one head.  Per 128-key tile and query tile:
//
//     S = Q K^T        (tcgen05.mma, both operands in shared memory, S in TMEM)
//     P = exp2(c S - m) row by row: one softmax thread per row reads its 128
//                      scores, so maximum and sum need no exchange; P goes
//                      back to TMEM in bf16, over the scores
//     O += P V         (tcgen05.mma, P from TMEM, V from shared memory MN-major)
//
// The two query tiles alternate on the tensor pipe (P0 V, Q0 K', P1 V, Q1 K'),
// so that one tile's softmax runs while the other's products do, and each key
// tile is loaded once for 256 rows: at 1024 tensor cycles per 128 x 128 tile
// (d = 128) the loads then need 32 bytes per cycle and SM, half of what a
// single tile would.
//
// The maximum is raised only when a row's new one exceeds the one in use by a
// factor of 2^8 (a weight is then at most 2^8, which costs fp32 sums and bf16
// weights no precision); only then O in TMEM is rescaled, by the softmax warp itself: the commit that
// announced the scores also covers the tile's earlier products.
//
// A weight is one fma and one exponential, 2^(c s - b) with b = c m rounded.
// What was summed before is rescaled by the difference of the rounded b, so
// all weights of a row refer to the same b exactly.  b is off from c m by up to
// half a step, 2^5 where |c m| < 2^30, and the row's largest weight by as many
// powers of two: a sum below 2^-40, or one that is not finite, tells of larger
// ones, and such rows are computed again (attn_rows.cuh).  Differences first
// would take a second instruction for every score.
//
// Key tiles: the sinks' (before the window of every row), then the window's
// from the first key that any row sees.  A tile that all rows of a query tile
// see entirely skips the mask; one that none sees is skipped; a short one
// takes fewer columns.  Masked weights are exact zeros, so only a non-finite
// masked value row can disturb a result; rows whose output is not finite are
// put right one by one (attn_rows.cuh).  Padding behind a sequence's last key
// is set to zero as it is loaded.
//
// Few rows and many keys: where the pieces of work would leave most SMs idle, a
// cluster of up to eight CTAs takes one piece, each a run of its key tiles, and
// joins the parts through distributed shared memory (16 rows of 8 heads on
// 8192 keys: 88 -> 23 us).
//
// Roles of the 384 threads: warps 0-3 softmax and output of query tile 0,
// warps 4-7 of tile 1, warps 8 and 9 issue the products of tiles 0 and 1, warp
// 10 the TMA loads, warp 11 fetches the next piece of work.
// Every wait is bounded (lr_device_status).
//
// Measured (d = 128): 16384 causal rows of 16 heads on 4 in 620 to 670 us, 1.64
// to 1.77 PFLOP/s of visible work (by the clock under the power limit); with a
// window of 1024 and 4 sinks 125 us; 4096 causal rows of 32 heads 110.5 us.  A pair of tiles takes 2690 cycles for 2048
// of the tensor pipe: the chain of a tile is scores -> first half of the weights
// (1100) -> its turn on the pipe (200) -> its 16 products (930) -> scores (460).
#include <algorithm>

#include "attn_internal.cuh"
#include "attn_join.cuh"
#include "attn_rows.cuh"
#include "attn_tc.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

using namespace tc;

__device__ unsigned g_wtc_error = 0;

constexpr int BM = 128, BN = 128;
// Threads and their registers: launched with 168 each (64,512 in all); the
// softmax warpgroups take 216, the third one keeps 72.
constexpr int NT = 384, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther <= NT * 168, "register shares");

template <int D>
struct Layout {
    static constexpr int KB = D > 64 ? 2 : 1;        // 64-column blocks of a tile
    static constexpr int TILE = KB * 128 * 128;      // bytes of a 128-row tile
    static constexpr int NS = D > 64 ? 4 : 8;        // key and value tiles in flight
    static constexpr int Q = 0;
    static constexpr int KV = 2 * TILE;
    static constexpr int OUT = KV + NS * TILE;       // 2 KB per softmax warp: rows on their way out,
                                                     // or (maximum, sum) of the rows of a part
    static constexpr int CLC = OUT + 8 * 2048;       // answer to a request for work, 16 bytes
    static constexpr int BAR = CLC + 16;
    static constexpr int ITEM = BAR + 384;           // two of struct Item
    static constexpr int BYTES = ITEM + 2 * 128;
    static constexpr int ALLOC = BYTES + 1024;
};

struct Barriers {
    uint64_t qfull[2], qempty[2], sfull[2], pready[2][2], ofull[2], oempty[2], fin[2];
    uint64_t full[8], empty[8];
    uint64_t ifull[2], iempty[2], clc, loaded, pad;
    uint32_t tmem, pipe;  // pipe: 1 while a warp issues products
};

constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S0, S1 (P over them), then O0, O1

struct TcArgs {
    WindowArgs w;
    float c;          // the scores' factor, positive
    unsigned negate;  // idesc bit: scores of -Q (scale < 0)
    int pair_heads;   // the two query tiles are two heads, else consecutive rows
    int group;        // query heads of a key head
    int tiles;        // row blocks of a head (pair)
    int span;         // heads (pairs) of all batches that are worked on together
    int splits;       // CTAs that share a piece (a cluster)
};

// A piece of work, kept in shared memory.  Key
// tile `it` is a sink tile (it < sink_tiles) or window tile it - sink_tiles.
// Sink tiles lie before the window of every row, so all rows see their keys.
// Window tiles that query tile t needs form one run [act0, act1), those that
// all its rows see entirely one inside it [all0, all1).
struct Item {
    int b, hk, head[2], i0[2];  // first row of each query tile
    int rows[2], p0[2];         // valid rows, position of the first
    int act0[2], act1[2], all0[2], all1[2];
    int last[2];                // last key tile that the query tile needs, -1: none
    int kl, sink_keys, sink_tiles, lo, hi;
    int first, n;               // the piece's key tiles: [first, n)
    int valid;                  // 0: no work is left

    __device__ __forceinline__ int key0(int it) const {
        return it < sink_tiles ? it * BN : lo + (it - sink_tiles) * BN;
    }
    __device__ __forceinline__ int limit(int it) const { return it < sink_tiles ? sink_keys : hi; }
    // columns that the tile needs, a multiple of 32
    __device__ __forceinline__ int width(int it) const {
        const int w = limit(it) - key0(it);
        return w >= BN ? BN : (w < 32 ? 32 : (w + 31) & ~31);
    }
};

// rank: of the CTA among those that share the piece (0 of 1: the whole piece).
template <bool SPLIT>
__device__ __forceinline__ void make_item(const TcArgs &g, int block, int rank, Item &x, bool *bad) {
    const WindowArgs &a = g.w;
    const int groups = g.pair_heads ? a.Hq / 2 : a.Hq;
    // the last rows see the most keys: of the heads whose keys and values the
    // L2 cache holds together, all longest tiles start first
    const unsigned size = g.span * g.tiles, span = (unsigned)block / size, in = block - span * size;
    const unsigned wide = min(g.span, a.B * groups - (int)span * g.span), deep = in / wide;
    const int tile = g.tiles - 1 - (int)deep, bh = span * g.span + in - deep * wide;
    const int batch = (unsigned)bh / (unsigned)groups, gh = bh - batch * groups;
    x.b = batch;
    const int ql = clamp_len(a.q_len, batch, a.Tq, bad), kl = clamp_len(a.k_len, batch, a.Tk, bad);
    x.kl = kl;
    if (g.pair_heads) {
        x.head[0] = 2 * gh, x.head[1] = 2 * gh + 1;
        x.i0[0] = x.i0[1] = tile * BM;
    } else {
        x.head[0] = x.head[1] = gh;
        x.i0[0] = tile * 2 * BM, x.i0[1] = x.i0[0] + BM;
    }
    x.hk = (unsigned)x.head[0] / (unsigned)g.group;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        x.rows[t] = max(0, min(BM, ql - x.i0[t]));
        x.p0[t] = kl - ql + x.i0[t];
    }
    const int last = x.rows[1] > 0 ? x.p0[1] + x.rows[1] - 1 : x.p0[0] + x.rows[0] - 1;
    const SeenKeys f = seen_keys(x.p0[0], kl, a.window, a.sinks),
                   e = seen_keys(last, kl, a.window, a.sinks);
    x.lo = f.lo, x.hi = e.hi;
    x.sink_keys = min(e.s1, f.lo);
    x.sink_tiles = (x.sink_keys + BN - 1) / BN;
    x.n = x.rows[0] > 0 ? x.sink_tiles + (x.hi > x.lo ? (x.hi - x.lo + BN - 1) / BN : 0) : 0;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
        // positions and keys lie within +-2^30, so differences of two fit an int
        const int p = x.p0[t], lo = x.lo, far = min(a.window, 1 << 30);
        // first key that the tile's first row sees; sinks inside the window tiles keep all
        const int k = a.sinks > lo ? 0 : p - far + 1 - lo;
        x.act0[t] = x.sink_tiles + (max(k, 0) / BN);
        const int last_p = p + x.rows[t] - 1 - lo;
        x.act1[t] = min(x.n, x.sink_tiles + (last_p < 0 ? 0 : last_p / BN + 1));
        const int f = p + BM - far - lo;  // first key of the last row
        x.all0[t] = min(x.n, x.sink_tiles + (f > 0 ? (f + BN - 1) / BN : 0));
        const int e = min(x.hi, p + 1) - lo;
        x.all1[t] = x.sink_tiles + (e > 0 ? e / BN : 0);
        if (!SPLIT && x.rows[t] > 0 && x.sink_tiles == 0 && x.act1[t] <= x.act0[t]) {
            // no key for any row: one tile with everything masked gives the zeros
            x.n = max(x.n, 1);
            x.act0[t] = 0, x.act1[t] = 1, x.all0[t] = x.all1[t] = 0;
        }
        x.last[t] = x.rows[t] == 0 ? -1 : (x.act1[t] > x.act0[t] ? x.act1[t] : x.sink_tiles) - 1;
    }
    x.first = 0;
    if (SPLIT) {
        const int n = x.n;
        x.first = (int)((long long)n * rank / g.splits);
        x.n = (int)((long long)n * (rank + 1) / g.splits);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            const int w = min(x.act1[t], x.n), k = min(x.sink_tiles, x.n);
            x.last[t] = x.rows[t] == 0                     ? -1
                        : w > max(x.act0[t], x.first)      ? w - 1
                        : k > x.first                      ? k - 1
                                                           : -1;
        }
    }
}

static_assert(sizeof(Item) <= 128 && sizeof(Barriers) <= 384, "shared memory layout");

// Ask for the index of a block that has not started, to do its work here; the
// answer (16 bytes at `dst`) is counted on `bar`.
__device__ __forceinline__ void request_block(void *dst, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(dst)),
        "r"(smem_u32(bar))
        : "memory");
}
// The index in the answer, -1 where no block was left.
__device__ __forceinline__ int granted_block(const void *src) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(src))
        : "memory");
    return got ? (int)x : -1;
}

// Joins the parts of a piece, which the CTAs left as join_row wants them: one
// warp per row, the rows shared out over the cluster.
template <int D>
__device__ __forceinline__ void join_parts(const TcArgs &g, const Item &x, uint32_t part, uint32_t stats) {
    const WindowArgs &a = g.w;
    const int warp = threadIdx.x >> 5, rank = (int)cluster_rank();
    for (int r = rank * (NT / 32) + warp; r < 2 * BM; r += g.splits * (NT / 32)) {
        const int t = r >> 7, row = r & (BM - 1);
        if (row >= x.rows[t]) continue;
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.o) + x.b * a.os.b + x.head[t] * a.os.h +
                            (long long)(x.i0[t] + row) * a.os.t;
        float sum;
        // the parts' maxima come in powers of two
        if (join_row<__nv_bfloat16, D>(part, stats, r, g.splits, 1.f, to, sum)) continue;
        mend_row<__nv_bfloat16, D>(
            static_cast<const __nv_bfloat16 *>(a.q) + x.b * a.qs.b + x.head[t] * a.qs.h +
                (long long)(x.i0[t] + row) * a.qs.t,
            static_cast<const __nv_bfloat16 *>(a.k) + x.b * a.ks.b + x.hk * a.ks.h,
            static_cast<const __nv_bfloat16 *>(a.v) + x.b * a.vs.b + x.hk * a.vs.h, a.ks.t, a.vs.t, to,
            seen_keys(x.p0[t] + row, x.kl, a.window, a.sinks), score_factor(a.scale), isfinite(sum));
    }
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(NT, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const TcArgs g) {
    using L = Layout<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Barriers *bars = reinterpret_cast<Barriers *>(sm + L::BAR);
    Item *items = reinterpret_cast<Item *>(sm + L::ITEM);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WindowArgs &a = g.w;

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->qfull[t], 1);
            mbar_init(&bars->qempty[t], 1);
            mbar_init(&bars->sfull[t], 1);
            mbar_init(&bars->pready[t][0], 4);  // the first 64 columns of P
            mbar_init(&bars->pready[t][1], 4);  // the others
            mbar_init(&bars->ofull[t], 1);
            mbar_init(&bars->oempty[t], 4);
            mbar_init(&bars->fin[t], 1);
            mbar_init(&bars->ifull[t], 1);
            mbar_init(&bars->iempty[t], 11);  // softmax, product and load warps
        }
        bars->pipe = 0;
        mbar_init(&bars->clc, 1);
        mbar_init(&bars->loaded, 1);
        mbar_init(&bars->pad, 1);
        for (int s = 0; s < L::NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 2);  // both query tiles
        }
        fence_mbar_init();
    }
    if (warp == 10 && lane == 0) {
        for (const CUtensorMap *map : {&tmq, &tmk, &tmv})
            asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    if (warp == 8) {
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    bool ok = true;

    // A role's next piece of work (whole warp); null at the end or on a wait that gave up.
    int piece = 0;
    auto take = [&]() -> const Item * {
        ok = __all_sync(0xffffffffu, ok && wait_bar(&bars->ifull[piece & 1], (piece >> 1) & 1));
        return ok && items[piece & 1].valid ? &items[piece & 1] : nullptr;
    };
    auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->iempty[piece & 1]);
        ++piece;
    };

    if (warp >= 8) regs_down<kRegsOther>();
    if (warp == 11) {
        // ==================================================== pieces of work
        // The block's own, then those of blocks that have not started: the
        // grid holds one block per piece, longest first, and each running CTA
        // takes the next one once the loads of its last have been issued (not
        // at once, or blocks that are about to start would be taken from idle
        // SMs).
        if (lane == 0) {
            int block = SPLIT ? blockIdx.x / g.splits : blockIdx.x;
            for (int i = 0; ok; ++i) {
                if (i >= 2) ok = wait_bar(&bars->iempty[i & 1], ((i >> 1) - 1) & 1);
                if (!ok) break;
                if (SPLIT && i > 0) {
                    block = -1;  // one piece for a cluster
                } else if (i > 0) {
                    ok = wait_bar(&bars->loaded, (i - 1) & 1);
                    if (!ok) break;
                    fence_async_smem();  // the last answer was read
                    mbar_expect_tx(&bars->clc, 16);
                    request_block(sm + L::CLC, &bars->clc);
                    ok = wait_bar(&bars->clc, (i - 1) & 1);
                    if (!ok) break;
                    block = granted_block(sm + L::CLC);
                }
                Item &x = items[i & 1];
                if (block >= 0) {
                    bool bad = false;
                    make_item<SPLIT>(g, block, SPLIT ? blockIdx.x % g.splits : 0, x, &bad);
                    if (bad) atomicOr(&g_wtc_error, kAttnIndex);
                }
                x.valid = block >= 0;
                mbar_arrive(&bars->ifull[i & 1]);
                if (block < 0) break;
            }
        }
    } else if (warp == 10) {
        // ============================================================ loads
        int seq = 0, used[2] = {0, 0}, pads = 0;
        while (const Item *px = take()) {
            const Item &x = *px;
#pragma unroll 1
            for (int t = 0; t < 2 && ok; ++t) {
                if (x.last[t] < 0) continue;
                if (used[t] > 0) ok = __all_sync(0xffffffffu, wait_bar(&bars->qempty[t], (used[t] - 1) & 1));
                if (!ok) break;
                ++used[t];
                if (lane == 0) {
                    mbar_expect_tx(&bars->qfull[t], L::TILE);
                    for (int kb = 0; kb < L::KB; ++kb)
                        tma_load_4d(sm + L::Q + t * L::TILE + kb * 16384, &tmq, kb * 64, x.i0[t],
                                    x.head[t], x.b, &bars->qfull[t]);
                }
            }
            const int n = x.n;
#pragma unroll 1
            for (int i = 2 * x.first; i < 2 * n && ok; ++i, ++seq) {
                const int s = seq % L::NS, k0 = x.key0(i >> 1);
                if (seq >= L::NS)
                    ok = __all_sync(0xffffffffu, wait_bar(&bars->empty[s], (seq / L::NS - 1) & 1));
                if (!ok) break;
                uint8_t *to = sm + L::KV + s * L::TILE;
                // values behind the last key: zeros, whatever the padding holds
                const bool pad = (i & 1) && x.kl < a.Tk && k0 + BN > x.kl;
                uint64_t *bar = pad ? &bars->pad : &bars->full[s];
                if (lane == 0) {
                    mbar_expect_tx(bar, L::TILE);
                    for (int kb = 0; kb < L::KB; ++kb)
                        tma_load_4d(to + kb * 16384, i & 1 ? &tmv : &tmk, kb * 64, k0, x.hk, x.b, bar);
                }
                if (pad) {
                    ok = __all_sync(0xffffffffu, wait_bar(&bars->pad, pads & 1));
                    ++pads;
                    const int from = max(0, x.kl - k0) * 8;  // 16-byte units of 128-byte rows
#pragma unroll 1
                    for (int u = from + lane; u < BN * 8; u += 32)
                        for (int kb = 0; kb < L::KB; ++kb)
                            *reinterpret_cast<uint4 *>(to + kb * 16384 + u * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->full[s]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->loaded);
            give_back();
        }
        // never leave with copies into shared memory in flight
        if (lane == 0) {
            for (int t = 0; t < 2; ++t)
                if (used[t] > 0 && !wait_bar(&bars->qfull[t], (used[t] - 1) & 1)) ok = false;
            if (pads > 0 && !wait_bar(&bars->pad, (pads - 1) & 1)) ok = false;
            for (int i = max(0, seq - L::NS); i < seq; ++i)
                if (!wait_bar(&bars->full[i % L::NS], (i / L::NS) & 1)) ok = false;
        }
    } else if (warp == 8 || warp == 9) {
        // ========================================================= products
        // One warp per query tile.  It walks and waits as a whole; one elected
        // lane issues.  What a step needs is worked out before its wait for P,
        // so that the products of a step follow the wait at once.
        const int t = warp - 8;
        const uint32_t q_s = smem_u32(sm + L::Q) + t * L::TILE, kv_s = smem_u32(sm + L::KV);
        const uint32_t s_t = tmem + kS + t * BN, o_t = tmem + kO + t * 128;
        const uint32_t id_o = idesc_bf16_f32_mn(BM, D, false, true);
        const uint64_t dq = tile_desc(q_s, 128, 0, 0);
        const bool lead = elect_one();
        int done_stages = 0;  // of earlier pieces
        int done = 0;   // key tiles multiplied
        int used = 0;   // pieces with any
        auto stage_wait = [&](int seq) {
            return __all_sync(0xffffffffu, wait_bar(&bars->full[seq % L::NS], (seq / L::NS) & 1));
        };
        while (const Item *px = take()) {
            const Item &x = *px;
            const int n = x.n, sink_tiles = x.sink_tiles, act0 = x.act0[t], act1 = x.act1[t], last = x.last[t];
            const int seq0 = done_stages - 2 * x.first;  // stage of key tile 0
            const int w_last = n > 0 ? x.width(n - 1) : 0, w_sink = sink_tiles ? x.width(sink_tiles - 1) : BN;
            auto active = [&](int it) {
                return last >= 0 && (it < sink_tiles || (it >= act0 && it < act1));
            };
            auto width = [&](int it) { return it == n - 1 ? w_last : (it == sink_tiles - 1 ? w_sink : BN); };
            // a tile that the query tile skips: its stages are free for it once loaded
            auto skip = [&](int it) {
#pragma unroll 1
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    const int seq = seq0 + 2 * it + kv;
                    ok = stage_wait(seq);
                    if (lead && ok) mbar_arrive(&bars->empty[seq % L::NS]);
                }
            };
            // S = Q K(it)^T
            auto scores = [&](int it, int s, uint64_t dk, uint32_t id) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16(s_t, kdesc_step(dq, 128, ks), kdesc_step(dk, 128, ks), id, ks > 0);
                mma_commit(&bars->sfull[t]);
                mma_commit(&bars->empty[s]);
                if (it == last) mma_commit(&bars->qempty[t]);
            };
            int it = x.first;
#pragma unroll 1
            for (; it < n && ok && !active(it); ++it) skip(it);
            if (it < n && ok) {
                const int seq = seq0 + 2 * it, s = seq % L::NS;
                ok = __all_sync(0xffffffffu, wait_bar(&bars->qfull[t], used & 1)) && stage_wait(seq);
                if (lead && ok)
                    scores(it, s, tile_desc(kv_s + s * L::TILE, 128, 0, 0),
                           idesc_bf16_f32(BM, width(it)) | g.negate);
                __syncwarp();
            }
            bool first = true;
            while (it < n && ok) {
                int nx = it + 1;
#pragma unroll 1
                for (; nx < n && ok && !active(nx); ++nx) skip(nx);
                if (ok && nx < n) ok = stage_wait(seq0 + 2 * nx);
                if (ok) ok = stage_wait(seq0 + 2 * it + 1);
                const int sk = (seq0 + 2 * nx) % L::NS, sv = (seq0 + 2 * it + 1) % L::NS;
                const uint64_t dk = tile_desc(kv_s + sk * L::TILE, 128, 0, 0),
                               dv = tile_desc_mn(kv_s + sv * L::TILE, 128, 0);
                const uint32_t id_s = idesc_bf16_f32(BM, width(nx)) | g.negate;
                const int steps = width(it) >> 4;
                // the last piece's output has left O
                if (ok && first && used > 0)
                    ok = __all_sync(0xffffffffu, wait_bar(&bars->oempty[t], (used - 1) & 1));
                if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->pready[t][0], done & 1));
                if (!ok) break;
                tc_fence_after();
                // O += P V, 64 keys at a time as P comes
                if (lead) {
                    take_pipe(&bars->pipe);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps)
                            mma_bf16_ta(o_t, s_t + 8 * ks, mndesc_step(dv, ks), id_o, ks > 0 || !first);
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, wait_bar(&bars->pready[t][1], done & 1));
                if (!ok) break;
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int ks = 4; ks < BN / 16; ++ks)
                        if (ks < steps) mma_bf16_ta(o_t, s_t + 8 * ks, mndesc_step(dv, ks), id_o, 1);
                    mma_commit(&bars->empty[sv]);
                    if (nx < n) scores(nx, sk, dk, id_s);
                    else mma_commit(&bars->ofull[t]);
                    free_pipe(&bars->pipe);
                }
                __syncwarp();
                first = false;
                ++done;
                it = nx;
            }
            if (!first) ++used;
            done_stages += 2 * (n - x.first);
            give_back();
        }
        if (lead) mma_commit(&bars->fin[t]);
        __syncwarp();
        if (!wait_bar(&bars->fin[t], 0)) ok = false;
    } else if (warp < 8) {
        // ========================================= softmax, then the output
        regs_up<kRegsSoftmax>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + kS + t * BN, to = tmem + lanes + kO + t * 128;
        const float2 c2 = make_float2(g.c, g.c);
        int seen = 0, used = 0;
        while (const Item *px = take()) {
            const Item &x = *px;
            const int sink_tiles = x.sink_tiles, act0 = x.act0[t], all0 = x.all0[t],
                      all1 = x.all1[t], n = x.last[t] + 1;
            const int p = x.p0[t] + row;
            const long long plo = (long long)p - a.window + 1;
            const int rlo = plo < 0 ? 0 : (int)plo;
            float m = -INFINITY, l = 0.f;
            for (int it = x.first; it < n && ok; ++it) {
                if (it >= sink_tiles && it < act0) continue;
                const bool whole = it >= all0 && it < all1;
                const int k0 = x.key0(it), end = min(p + 1, x.limit(it));
                ok = __all_sync(0xffffffffu, wait_bar(&bars->sfull[t], seen & 1));
                if (!ok) break;
                tc_fence_after();
                // raise the maximum in use, rescaling the sum and O, where a row needs it
                auto raise = [&](float mn) {
                    const bool grow = mn > m && (m == -INFINITY || (mn - m) * g.c > 8.f);
                    // a row that has seen nothing yet has l = 0 and zeros in O (or O unset)
                    if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
                        // no fma here: both products as `base` has them
                        const float f = grow && m != -INFINITY
                                            ? ex2(__fsub_rn(__fmul_rn(m, g.c), __fmul_rn(mn, g.c)))
                                            : 1.f;
                        l *= f;
#pragma unroll 1
                        for (int ch = 0; ch < D / 16; ++ch) {
                            float v[16];
                            tmem_ld16(to + 16 * ch, v);
                            tmem_ld_wait(v);
                            uint32_t r[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i] * f);
                            tmem_st16(to + 16 * ch, r);
                        }
                    }
                    if (grow) m = mn;
                    return m == -INFINITY ? 0.f : -__fmul_rn(m, g.c);
                };
                float2 sum[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
                // weights of 32 columns: P over the first half of the scores' place
                auto weights = [&](int ch, const float (&s)[32], float2 b2) {
                    uint32_t r[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = fma2(make_float2(s[2 * i], s[2 * i + 1]), c2, b2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        sum[i & 3] = add2(sum[i & 3], e);
                        r[i] = pack2(e.x, e.y);
                    }
                    tmem_st16(ts + 16 * ch, r);
                };
                auto top = [&](float (&mx)[4], const float (&s)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[i], s[i + 1]);
                };
                if (!whole) {
                    // A tile at the edge of what the rows see, or a narrow one:
                    // -inf over the scores that a row does not see, in TMEM, so
                    // that one code serves all tiles (unrolled code of its own
                    // fell out of the instruction cache between its uses).
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        const int kc = k0 + 32 * ch;
                        const uint32_t keep = low_bits(end - kc) & (~low_bits(rlo - kc) | low_bits(a.sinks - kc));
                        if (__all_sync(0xffffffffu, keep == 0xffffffffu)) continue;
                        float s[32];
                        tmem_ld32(ts + 32 * ch, s);
                        tmem_ld_wait(s);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((keep >> i) & 1u)) s[i] = -INFINITY;
                        tmem_st32(ts + 32 * ch, s);
                    }
                    tmem_st_wait();
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto publish = [&](int half) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->pready[t][half]);
                };
                float s[4][32];
                tmem_ld32(ts, s[0]);
                tmem_ld32(ts + 32, s[1]);
                tmem_ld32(ts + 64, s[2]);
                tmem_ld32(ts + 96, s[3]);
                tmem_ld_wait(s[0], s[1], s[2], s[3]);
                top(mx, s[0]);
                top(mx, s[1]);
                top(mx, s[2]);
                top(mx, s[3]);
                const float base = raise(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                const float2 b2 = make_float2(base, base);
                weights(0, s[0], b2);
                weights(1, s[1], b2);
                publish(0);
                weights(2, s[2], b2);
                weights(3, s[3], b2);
                publish(1);
                const float2 two = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += two.x + two.y;
                ++seen;
            }
            // the rounding of the exponent's base took the weights' range
            if (m != -INFINITY && !(l >= 0x1p-40f)) l = NAN;
            if (SPLIT) {
                // the part, once the products of both query tiles have read their operands
                for (int u = 0; u < 2; ++u)
                    if (x.last[u] >= 0 && ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->ofull[u], 0));
                tc_fence_after();
                *reinterpret_cast<float2 *>(sm + L::OUT + (t * BM + row) * 8) = make_float2(__fmul_rn(m, g.c), l);
                if (n > 0 && ok) {
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        float v[32];
                        tmem_ld32(to + 32 * ch, v);
                        tmem_ld_wait(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4 *>(sm + part_at<D>(t * BM + row, 8 * ch + i)) =
                                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                give_back();
                continue;
            }
            if (n == 0) {
                give_back();
                continue;
            }
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->ofull[t], used & 1));
            ++used;
            if (!ok) break;
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;  // no key, or only scores of -inf
            // Rows leave through the warp's shared memory, 32 channels at a time,
            // so that a store writes whole 64-byte pieces of eight rows (with a
            // row per lane it touched 32 lines at once).
            uint8_t *out = sm + L::OUT + warp * 2048;
            const int w0 = 32 * (warp & 3), rows = x.rows[t], r8 = lane >> 2, c8 = lane & 3;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + x.b * a.os.b + x.head[t] * a.os.h +
                               (long long)(x.i0[t] + w0 + r8) * a.os.t + 8 * c8;
            const long long next8 = 8 * a.os.t;
            float odd[4] = {0.f, 0.f, 0.f, 0.f};  // NaN once a value is not finite
            int last_ch;      // hidden from the compiler, which would unroll the last turn
            asm volatile("mov.u32 %0, %1;" : "=r"(last_ch) : "n"(D / 32 - 1));
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                float v[32];
                tmem_ld32(to + 32 * ch, v);
                tmem_ld_wait(v);
                if (ch == last_ch) {  // O has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->oempty[t]);
                }
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float y0 = v[2 * i] * inv, y1 = v[2 * i + 1] * inv;
                    odd[i & 3] = fmaf(y0, 0.f, fmaf(y1, 0.f, odd[i & 3]));
                    w[i] = pack2(y0, y1);
                }
                __syncwarp();  // the last channels have left
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(out + lane * 64 + (i ^ ((lane >> 1) & 3)) * 16) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                __syncwarp();
                __nv_bfloat16 *oc = o + 32 * ch;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = 8 * i + r8;
                    const uint4 y = *reinterpret_cast<const uint4 *>(out + rr * 64 + (c8 ^ ((rr >> 1) & 3)) * 16);
                    if (w0 + rr < rows) *reinterpret_cast<uint4 *>(oc) = y;
                    oc += next8;
                }
            }
            unsigned again = __ballot_sync(0xffffffffu, row < rows && !(odd[0] + odd[1] + odd[2] + odd[3] == 0.f));
            if (again) {
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + x.b * a.qs.b +
                                         x.head[t] * a.qs.h + (long long)x.i0[t] * a.qs.t;
                const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + x.b * a.ks.b + x.hk * a.ks.h;
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + x.b * a.vs.b + x.hk * a.vs.h;
                __nv_bfloat16 *ot = static_cast<__nv_bfloat16 *>(a.o) + x.b * a.os.b + x.head[t] * a.os.h +
                                    (long long)x.i0[t] * a.os.t;
                __syncwarp();
                while (again) {
                    const int src = __ffs(again) - 1, rr = w0 + src;
                    again &= again - 1;
                    mend_row<__nv_bfloat16, D>(q + rr * a.qs.t, k, v, a.ks.t, a.vs.t, ot + rr * a.os.t,
                                               seen_keys(x.p0[t] + rr, x.kl, a.window, a.sinks), score_factor(a.scale),
                                               isfinite(__shfl_sync(0xffffffffu, l, src)));
                }
            }
            give_back();
        }
    }

    if (!ok) atomicOr(&g_wtc_error, kAttnTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (SPLIT) {
        cluster_sync_all();
        join_parts<D>(g, items[0], smem_u32(sm), smem_u32(sm + L::OUT));
        cluster_sync_all();  // no CTA leaves while another reads its part
    }
}

template <int D>
cudaError_t launch(const WindowArgs &a, int slot, cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    cudaError_t e = rows_map(&mq, a.q, a.qs, a.B, a.Hq, a.Tq, D);
    if (e == cudaSuccess) e = rows_map(&mk, a.k, a.ks, a.B, a.Hk, a.Tk, D);
    if (e == cudaSuccess) e = rows_map(&mv, a.v, a.vs, a.B, a.Hk, a.Tk, D);
    if (e != cudaSuccess) return e;
    TcArgs g;
    g.w = a;
    // The queries reach the products as they are, so for scale 0 c is fp32's
    // smallest value: 2^(c s) is 1 within 2^-20 for every finite score, and a
    // masked -inf stays one
    g.c = a.scale == 0.f ? 0x1p-149f : score_factor(a.scale).c;
    g.negate = a.scale < 0.f ? 1u << 13 : 0u;
    g.group = a.Hq / a.Hk;
    g.pair_heads = g.group % 2 == 0;
    const int rows = g.pair_heads ? BM : 2 * BM;
    g.tiles = (a.Tq + rows - 1) / rows;
    // keys and values of the heads in flight stay within 48 MB of the L2's 129
    const long long kv = 4ll * D * a.Tk, pairs = (long long)a.B * (g.pair_heads ? a.Hq / 2 : a.Hq);
    const long long span = (48ll << 20) / kv;
    g.span = (int)(span < 1 ? 1 : (span < pairs ? span : pairs));
    const long long pieces = pairs * g.tiles;
    // Key tiles of a piece at most.  All clusters have to run at once: a second
    // round would cost as much as the first.  The join takes as long as four
    // tiles (64 rows of 32 heads on 4096 keys: 49 us alone, 20.6 by 6; 4 heads,
    // d = 128, 100 rows: on 1024 keys 15.7 alone, 15.2 by 2, 10.9 by 8; on 512
    // 10.6 alone, 12.5 by 2).
    const long long most = std::min<long long>(a.Tk, (long long)a.window + (g.pair_heads ? 1 : 2) * BM);
    const int tiles = (int)((most + BN - 1) / BN) + (std::min(a.sinks, a.Tk) + BN - 1) / BN;
    g.splits = 1;
    for (int s = 2, least = tiles; s <= kMostCluster && s <= tiles; ++s) {
        const int cost = (tiles + s - 1) / s + 4;
        if (pieces * s <= kClusterRoom[0][s] && cost < least) g.splits = s, least = cost;
    }
    auto *fn = g.splits > 1 ? window_tc_kernel<D, true> : window_tc_kernel<D, false>;
    e = ensure_smem_attr(reinterpret_cast<const void *>(fn), Layout<D>::ALLOC, slot + (g.splits > 1 ? 3 : 0));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pieces * g.splits));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = Layout<D>::ALLOC;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)g.splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = g.splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, mq, mk, mv, g);
}

}  // namespace

// ensure_smem_attr slots 214..219 belong to this file.
cudaError_t launch_window_tc(const WindowArgs &a, int d, cudaStream_t stream) {
    if (d == 32) return launch<32>(a, 214, stream);
    if (d == 64) return launch<64>(a, 215, stream);
    return launch<128>(a, 216, stream);
}

int attn_errors_window_tc() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_wtc_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_wtc_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
