// lr_fwd_diff in bf16 on the tensor cores (tcgen05): both softmax maps of a pair
// of heads in one pass over the keys, their difference and its norm in the
// epilogue (attn_diff.cuh has the formula).
//
// A CTA takes 128 query rows of a pair.  Per 128-key tile and map m:
//
//     S_m = Q_m K_m^T   (tcgen05.mma, both operands in shared memory, S in TMEM)
//     P_m = exp2(c S_m - b) row by row, one softmax thread per row (softmax_tile)
//     O_m += P_m V      (P from TMEM, V from shared memory MN-major, 2 d columns)
//
// The maps alternate on the tensor pipe, one's softmax under the other's
// products, and share the value tile.  Both outputs stay in tensor memory, so
// the difference is formed there in fp32 and rounded once: at the end each of
// the two softmax warpgroups reads half of the channels of both outputs.
//
// The difference takes away what the maps have in common, but not the rounding of their
// weights to bf16, so what that rounding left is multiplied as well, as bf16 weights of its
// own in the other half of the score tile: a weight counts with 16 bits, and the error of
// a result is that of 32-bit weights (without the rest 1.53 times that; lr_fwd_window:
// 1.35).  It costs twice the value products: 8192 causal tokens of 8 pairs, d = 64, 156 us
// without, 206 with it; d = 32 148 and 208.
//
// Measured: those 206 us are 1000 TFLOP/s of visible products, 1670 of those formed.  What
// bounds it is a map's chain, softmax of a tile, its last products, its next scores, which
// the tensor pipe takes behind them: some 3000 cycles a tile of both maps, whose products
// need 2560 (1536 at d = 32).
//
// Tensor memory holds 2 x 128 columns of scores and 2 x 128 of output, so d is 32
// or 64 here (diff_wide_tc.cu: 128).
//
// A row's non-finite values, padding and the rounding of the exponent's base are
// dealt with as in window_tc.cu.
//
// Roles of the 384 threads: warps 0-3 softmax of map 0 and the first half of the
// channels, warps 4-7 of map 1 and the second half, warps 8 and 9 issue the
// products of maps 0 and 1, warp 10 the TMA loads, warp 11 works out the pieces.
// The CTAs stay and take every n-th piece, longest first and in turning order, so
// that loads and products of the next piece run under the last one's epilogue.
// Every wait is bounded (lr_device_status).
#include <algorithm>

#include "attn_diff_tc.cuh"
#include "attn_internal.cuh"
#include "attn_tc.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

using namespace tc;

__device__ unsigned g_diff_error = 0;

constexpr int BM = kDiffRows, BN = kDiffKeys;
// Threads and their registers: launched with 168 each (64,512 in all); the
// softmax warpgroups take 216, the third one keeps 72.
constexpr int NT = 384, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther <= NT * 168, "register shares");

template <int D>
struct Layout {
    static constexpr int DV = 2 * D;                 // value channels
    static constexpr int TILE = 128 * 128;           // bytes of a query or key tile: one 64-column block
    static constexpr int VTILE = 2 * 128 * 128;      // of a value tile: a block for each half
    static constexpr int NK = 2, NV = 2;             // key tiles (per map) and value tiles in flight
    static constexpr int Q = 0;
    static constexpr int K = 2 * TILE;               // [slot][map]
    static constexpr int V = K + 2 * NK * TILE;
    static constexpr int OUT = V + NV * VTILE;       // 2 KB per softmax warp: rows on their way out
    static constexpr int SUM = OUT + 8 * 2048;       // [2][map][128] sums of weights
    static constexpr int SQ = SUM + 2 * 2 * 128 * 4; // [2][2][128] sums of squares
    static constexpr int W = SQ + 2 * 2 * 128 * 4;   // [2 D] weights of the norm
    static constexpr int BAR = W + 2 * D * 4;
    static constexpr int ITEM = BAR + 384;           // two of struct DiffItem
    static constexpr int BYTES = ITEM + 2 * 128;
    static constexpr int ALLOC = BYTES + 1024;
};

struct Barriers {
    uint64_t qfull, qempty, sfull[2], pready[2][2], ofull[2], oempty, fin[2];
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
    uint64_t ifull[2], iempty[2], lfull, sqready, pad;
    uint32_t tmem, pipe;  // pipe: 1 while a warp issues products
};

static_assert(sizeof(Barriers) <= 384, "shared memory layout");

constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S0, S1 (P over them), then O0, O1

template <int D>
__global__ void __launch_bounds__(NT, 1)
    diff_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const DiffTcArgs g) {
    using L = Layout<D>;
    constexpr int NK = L::NK, NV = L::NV, DV = L::DV;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Barriers *bars = reinterpret_cast<Barriers *>(sm + L::BAR);
    DiffItem *items = reinterpret_cast<DiffItem *>(sm + L::ITEM);
    float *wsm = reinterpret_cast<float *>(sm + L::W);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DiffArgs &a = g.a;

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->sfull[t], 1);
            mbar_init(&bars->pready[t][0], 4);  // the first 64 columns of P
            mbar_init(&bars->pready[t][1], 4);  // the others
            mbar_init(&bars->ofull[t], 1);
            mbar_init(&bars->fin[t], 1);
            mbar_init(&bars->ifull[t], 1);
            mbar_init(&bars->iempty[t], 11);  // softmax, product and load warps
        }
        for (int s = 0; s < NK; ++s) {
            mbar_init(&bars->kfull[s], 1);
            mbar_init(&bars->kempty[s], 2);  // both maps
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&bars->vfull[s], 1);
            mbar_init(&bars->vempty[s], 2);
        }
        mbar_init(&bars->qfull, 1);
        mbar_init(&bars->qempty, 2);
        mbar_init(&bars->oempty, 8);
        mbar_init(&bars->lfull, 8);
        mbar_init(&bars->sqready, 8);
        mbar_init(&bars->pad, 1);
        bars->pipe = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < 2 * D; i += NT) wsm[i] = a.norm && a.weight ? a.weight[i] : 1.f;
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
    auto take = [&]() -> const DiffItem * {
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
        if (lane == 0) {
            const int me = blockIdx.x, all = gridDim.x;
            for (int i = 0; ok; ++i) {
                if (i >= 2) ok = wait_bar(&bars->iempty[i & 1], ((i >> 1) - 1) & 1);
                if (!ok) break;
                const long long block = (long long)i * all + (i & 1 ? all - 1 - me : me);
                DiffItem &x = items[i & 1];
                const bool some = block < g.pieces;
                if (some) {
                    bool bad = false;
                    make_diff_item(g, (int)block, x, &bad);
                    if (bad) atomicOr(&g_diff_error, kAttnIndex);
                }
                x.valid = some;
                mbar_arrive(&bars->ifull[i & 1]);
                if (!some) break;
            }
        }
    } else if (warp == 10) {
        // ============================================================ loads
        int queries = 0, keys = 0, done = 0, pads = 0;  // asked for: pairs of query and key tiles, value tiles
        while (const DiffItem *px = take()) {
            const DiffItem &x = *px;
            const int n = x.n;
            if (n > 0) {
                if (queries > 0) ok = __all_sync(0xffffffffu, wait_bar(&bars->qempty, (queries - 1) & 1));
                if (ok) {
                    ++queries;
                    if (lane == 0) {
                        mbar_expect_tx(&bars->qfull, 2 * L::TILE);
                        tma_load_5d(sm + L::Q, &tmq, 0, x.i0, 0, 2 * x.h, x.b, &bars->qfull);
                    }
                }
            }
#pragma unroll 1
            for (int it = 0; it < n && ok; ++it) {
                const int k0 = x.key0(it), ks = done % NK, vs = done % NV;
                if (done >= NK) ok = __all_sync(0xffffffffu, wait_bar(&bars->kempty[ks], (done / NK - 1) & 1));
                if (!ok) break;
                ++keys;
                if (lane == 0) {
                    mbar_expect_tx(&bars->kfull[ks], 2 * L::TILE);
                    tma_load_5d(sm + L::K + ks * 2 * L::TILE, &tmk, 0, k0, 0, 2 * x.hk, x.b, &bars->kfull[ks]);
                }
                if (done >= NV) ok = __all_sync(0xffffffffu, wait_bar(&bars->vempty[vs], (done / NV - 1) & 1));
                if (!ok) break;
                uint8_t *to = sm + L::V + vs * L::VTILE;
                // values behind the last key: zeros, whatever the padding holds
                const bool pad = x.kl < a.Tk && k0 + BN > x.kl;
                uint64_t *bar = pad ? &bars->pad : &bars->vfull[vs];
                if (lane == 0) {
                    mbar_expect_tx(bar, L::VTILE);
                    tma_load_5d(to, &tmv, 0, k0, 0, 2 * x.hk, x.b, bar);
                }
                if (pad) {
                    ok = __all_sync(0xffffffffu, wait_bar(&bars->pad, pads & 1));
                    ++pads;
                    const int from = max(0, x.kl - k0) * 8;  // 16-byte units of 128-byte rows
#pragma unroll 1
                    for (int u = from + lane; u < BN * 8; u += 32)
                        for (int j = 0; j < 2; ++j)
                            *reinterpret_cast<uint4 *>(to + j * 16384 + u * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->vfull[vs]);
                }
                ++done;
            }
            give_back();
        }
        // never leave with copies into shared memory in flight: the last phases
        // of every barrier that this warp armed
        if (lane == 0) {
            if (queries > 0 && !wait_bar(&bars->qfull, (queries - 1) & 1)) ok = false;
            for (int i = max(0, keys - NK); i < keys; ++i)
                if (!wait_bar(&bars->kfull[i % NK], (i / NK) & 1)) ok = false;
            for (int i = max(0, done - NV); i < done; ++i)
                if (!wait_bar(&bars->vfull[i % NV], (i / NV) & 1)) ok = false;
            if (pads > 0 && !wait_bar(&bars->pad, (pads - 1) & 1)) ok = false;
        }
    } else if (warp == 8 || warp == 9) {
        // ========================================================= products
        // One warp per map.  It walks and waits as a whole; one elected lane
        // issues.  What a step needs is worked out before its wait for P.
        const int t = warp - 8;
        const uint32_t s_t = tmem + kS + t * BN, o_t = tmem + kO + t * 128;
        // d = 32: the halves' 32 columns lie in two 64-column blocks, a product each
        constexpr int NO = D == 32 ? 2 : 1;
        const uint32_t id_o = idesc_bf16_f32_mn(BM, DV / NO, false, true);
        const uint64_t dq = tile_desc(smem_u32(sm + L::Q) + t * L::TILE, 128, 0, 0);
        const uint32_t k_s = smem_u32(sm + L::K) + t * L::TILE, v_s = smem_u32(sm + L::V);
        const bool lead = elect_one();
        int done = 0, used = 0;  // key tiles and pieces multiplied
        auto k_wait = [&](int i) {
            return __all_sync(0xffffffffu, wait_bar(&bars->kfull[i % NK], (i / NK) & 1));
        };
        while (const DiffItem *px = take()) {
            const DiffItem &x = *px;
            const int n = x.n;
            if (n == 0) {
                give_back();
                continue;
            }
            const int w_last = x.width(n - 1), w_sink = x.sink_tiles ? x.width(x.sink_tiles - 1) : BN;
            const int sink_tiles = x.sink_tiles;
            auto width = [&](int it) { return it == n - 1 ? w_last : (it == sink_tiles - 1 ? w_sink : BN); };
            // S = Q K(it)^T; i: tiles multiplied before it
            auto scores = [&](int it, int i) {
                const uint64_t dk = tile_desc(k_s + (i % NK) * 2 * L::TILE, 128, 0, 0);
                const uint32_t id = idesc_bf16_f32(BM, width(it)) | g.negate;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16(s_t, kdesc_step(dq, 128, ks), kdesc_step(dk, 128, ks), id, ks > 0);
                mma_commit(&bars->sfull[t]);
                mma_commit(&bars->kempty[i % NK]);
                if (it == n - 1) mma_commit(&bars->qempty);
            };
            ok = __all_sync(0xffffffffu, wait_bar(&bars->qfull, used & 1)) && k_wait(done);
            if (lead && ok) scores(0, done);
            __syncwarp();
#pragma unroll 1
            for (int it = 0; it < n && ok; ++it) {
                if (it + 1 < n) ok = k_wait(done + 1);
                if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->vfull[done % NV], (done / NV) & 1));
                const uint64_t dv = tile_desc_mn(v_s + (done % NV) * L::VTILE, 128, 0);
                const int steps = width(it) >> 4;
                // 16 keys: their weights, and what the weights' rounding left
                auto values = [&](int ks) {
#pragma unroll
                    for (int rest = 0; rest < 2; ++rest)
#pragma unroll
                        for (int j = 0; j < NO; ++j)
                            mma_bf16_ta(o_t + j * (DV / NO), s_t + 64 * rest + 8 * ks,
                                        mndesc_step(dv, ks) + j * (16384u >> 4), id_o, rest || ks > 0 || it > 0);
                };
                // the last piece's outputs have left
                if (ok && it == 0 && used > 0)
                    ok = __all_sync(0xffffffffu, wait_bar(&bars->oempty, (used - 1) & 1));
                if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->pready[t][0], done & 1));
                if (!ok) break;
                tc_fence_after();
                // O += P V, 64 keys at a time as P comes
                if (lead) {
                    take_pipe(&bars->pipe);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps) values(ks);
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, wait_bar(&bars->pready[t][1], done & 1));
                if (!ok) break;
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int ks = 4; ks < BN / 16; ++ks)
                        if (ks < steps) values(ks);
                    mma_commit(&bars->vempty[done % NV]);
                    if (it + 1 < n) scores(it + 1, done + 1);
                    else mma_commit(&bars->ofull[t]);
                    free_pipe(&bars->pipe);
                }
                __syncwarp();
                ++done;
            }
            ++used;
            give_back();
        }
        if (lead) mma_commit(&bars->fin[t]);
        __syncwarp();
        if (!wait_bar(&bars->fin[t], 0)) ok = false;
    } else if (warp < 8) {
        // ========================== softmax, then the difference and its norm
        regs_up<kRegsSoftmax>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + kS + t * BN, to = tmem + lanes + kO + t * 128;
        constexpr int CH = DV / 2;  // channels of this warpgroup
        const int col = t * CH;     // the first of them in the outputs
        const int half = col / D, in_half = col - half * D;
        int seen = 0, used = 0;
        bool marked = false;  // a row of the warp is to be put right
        while (const DiffItem *px = take()) {
            const DiffItem &x = *px;
            const int n = x.n, all0 = x.all0, all1 = x.all1;
            if (n == 0) {
                give_back();
                continue;
            }
            const int p = x.p0 + row;
            const long long plo = (long long)p - a.window + 1;
            const int rlo = plo < 0 ? 0 : (int)plo;
            float m = -INFINITY, l = 0.f;
            for (int it = 0; it < n && ok; ++it) {
                const bool whole = it >= all0 && it < all1;
                const int k0 = x.key0(it), end = min(p + 1, x.limit(it));
                ok = __all_sync(0xffffffffu, wait_bar(&bars->sfull[t], seen & 1));
                if (!ok) break;
                tc_fence_after();
                auto keep = [&](int ch) {
                    const int kc = k0 + 32 * ch;
                    return low_bits(end - kc) & (~low_bits(rlo - kc) | low_bits(a.sinks - kc));
                };
                softmax_tile<DV, true>(ts, to, g.c, whole, keep, m, l, &bars->pready[t][0], &bars->pready[t][1]);
                ++seen;
            }
            // the rounding of the exponent's base took the weights' range
            if (m != -INFINITY && !(l >= 0x1p-40f)) l = NAN;
            const int slot = used & 1;
            float *sums = reinterpret_cast<float *>(sm + L::SUM) + slot * 256;
            sums[t * 128 + row] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->lfull);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->lfull, used & 1));
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->ofull[0], used & 1));
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->ofull[1], used & 1));
            if (!ok) break;
            tc_fence_after();
            const float l0 = sums[row], l1 = sums[128 + row];
            // no key, or only scores of -inf: zeros
            const float f0 = l0 == 0.f ? 0.f : 1.f / l0, f1 = (l1 == 0.f ? 0.f : 1.f / l1) * -a.lambda[x.h];
            float y[CH], squares = 0.f;
#pragma unroll
            for (int c = 0; c < CH; c += 32) {
                float u[32], w[32];
                tmem_ld32(tmem + lanes + kO + col + c, u);
                tmem_ld32(tmem + lanes + kO + 128 + col + c, w);
                tmem_ld_wait(u, w);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    // each product rounded, so that equal maps cancel exactly
                    y[c + i] = __fadd_rn(__fmul_rn(u[i], f0), __fmul_rn(w[i], f1));
                    squares = fmaf(y[c + i], y[c + i], squares);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->oempty);
            squares = marked_squares(y, squares);
            if (a.norm) {
                // the other channels' sum of this row, from the other warpgroup
                float *sq = reinterpret_cast<float *>(sm + L::SQ) + slot * 256;
                sq[t * 128 + row] = squares;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->sqready);
                ok = __all_sync(0xffffffffu, wait_bar(&bars->sqready, used & 1));
                if (!ok) break;
                squares = sq[row] + sq[128 + row];
            }
            const float scale = diff_scale(a.norm, squares, D, a.eps);
            marked = marked || (row < x.rows && scale != scale);
            ++used;
            // Rows leave through the warp's shared memory, 32 channels at a time,
            // so that a store writes whole 64-byte pieces of eight rows.
            uint8_t *out = sm + L::OUT + warp * 2048;
            const int w0 = 32 * (warp & 3), rows = x.rows, r8 = lane >> 2, c8 = lane & 3;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + x.b * a.os.b + (2 * x.h + half) * a.os.h +
                               (long long)(x.i0 + w0 + r8) * a.os.t + in_half + 8 * c8;
            const float4 *weight = reinterpret_cast<const float4 *>(wsm + col);
#pragma unroll
            for (int c = 0; c < CH; c += 32) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 z = weight[c / 4 + i];
                    const float *yi = y + c + 4 * i;
                    w[2 * i] = pack2(yi[0] * scale * z.x, yi[1] * scale * z.y);
                    w[2 * i + 1] = pack2(yi[2] * scale * z.z, yi[3] * scale * z.w);
                }
                __syncwarp();  // the last channels have left
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(out + lane * 64 + (i ^ ((lane >> 1) & 3)) * 16) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = 8 * i + r8;
                    const uint4 z = *reinterpret_cast<const uint4 *>(out + rr * 64 + (c8 ^ ((rr >> 1) & 3)) * 16);
                    if (w0 + rr < rows) *reinterpret_cast<uint4 *>(o + 8 * i * a.os.t + c) = z;
                }
            }
            give_back();
        }
        mend_marked<D>(g, __any_sync(0xffffffffu, ok && marked), blockIdx.x, gridDim.x, 0, CH);
    }

    if (!ok) atomicOr(&g_diff_error, kAttnTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const DiffArgs &a, int slot, cudaStream_t stream) {
    using L = Layout<D>;
    CUtensorMap mq, mk, mv;
    cudaError_t e = blocks_map(&mq, a.q, a.qs, a.B, 2 * a.H, a.Tq, D, BM, 2);
    if (e == cudaSuccess) e = blocks_map(&mk, a.k, a.ks, a.B, 2 * a.Hk, a.Tk, D, BN, 2);
    if (e == cudaSuccess) e = blocks_map(&mv, a.v, a.vs, a.B, 2 * a.Hk, a.Tk, D, BN, 2);
    if (e != cudaSuccess) return e;
    const DiffTcArgs g = diff_tc_args(a, D);
    auto *fn = diff_tc_kernel<D>;
    e = ensure_smem_attr(reinterpret_cast<const void *>(fn), L::ALLOC, slot);
    if (e != cudaSuccess) return e;
    fn<<<(unsigned)std::min(g.pieces, 152), NT, L::ALLOC, stream>>>(mq, mk, mv, g);
    return cudaGetLastError();
}

}  // namespace

// ensure_smem_attr slots 224 and 225 belong to this file.
cudaError_t launch_diff_tc(const DiffArgs &a, int d, cudaStream_t stream) {
    if (d == 32) return launch<32>(a, 224, stream);
    if (d == 64) return launch<64>(a, 225, stream);
    return launch_diff_wide_tc(a, stream);
}

int attn_errors_diff_tc() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_diff_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_diff_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
