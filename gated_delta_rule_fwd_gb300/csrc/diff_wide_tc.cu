// lr_fwd_diff in bf16 at d = 128, where a pair's value row has 256 channels: both
// maps' outputs of 128 rows would take all of tensor memory.  A cluster of two
// CTAs takes 128 query rows of a pair, a CTA a map:
//
//     S = Q_m K_m^T   128 keys at a time, two buffers of 128 columns
//     P = exp2(c S - b)
//     O += P V        all 256 channels (products of N = 256)
//
// Scores are formed once, a buffer ahead: their products, the softmax of the other
// buffer and the value products run at the same time.  The pipe gets them in the order
// P V of tile i, S of tile i + 2, P V of tile i + 1: scores that wait behind the next value
// products hold up their softmax (an earlier version: 200 instead of 181 us).  Scores of
// tile i + 2 overwrite the weights of tile i and wait until the products that read these
// are done.  Each CTA loads the values for itself.  Two softmax threads share a row, 64
// keys each; they exchange the tile's maximum, so that both raise the one in use together.
// At the end a CTA takes over the rows' 128 channels of its half: the CTAs send each other
// the other half of their output, scaled, through distributed shared memory (over queries
// and keys, which are free from the last scores on), and the rows' sums of squares.
//
// Weights count with 16 bits as in diff_tc.cu (2 x 4096 causal tokens of 8 pairs: 171 us
// without their rest, 218 with it); a row's non-finite values, padding and the rounding of
// the exponent's base are dealt with as in window_tc.cu.
//
// Roles of the 384 threads: warps 0-3 softmax of a tile's first 64 keys and the first
// half of the CTA's channels, warps 4-7 of the others, warp 8 issues the value
// products, warp 9 the scores', warp 10 loads the values, warp 11 works out the pieces
// and loads their queries and keys.
//
// A load warp's work per copy counts: its code is cold each time it wakes (two copies
// a tile by the whole warp took longer than the tile's products), hence one lane in
// short loops, few barriers, whole boxes.  Every wait is bounded (lr_device_status).
//
// Measured: those 218 us are 945 TFLOP/s of visible products, 1575 of those formed (16384
// tokens of 8 pairs: 1154 and 1923, all that the pipe gives).  Beside its tiles a piece
// costs the wait for its last products, the exchange (64 KB each way at some 32 bytes a
// cycle), two rounds between the CTAs and the stores: the share of that falls with length.
#include <algorithm>

#include "attn_diff_tc.cuh"
#include "attn_internal.cuh"
#include "attn_join.cuh"
#include "attn_tc.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

using namespace tc;

__device__ unsigned g_diff_wide_error = 0;

constexpr int D = 128, DV = 256;
constexpr int BM = kDiffRows;
// Threads and their registers: launched with 168 each (64,512 in all); the
// softmax warpgroups take 216, the third one keeps 72.
constexpr int NT = 384, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther <= NT * 168, "register shares");

constexpr int BLOCK = 128 * 128;                // bytes of 128 rows' 64 columns
constexpr int VHALF = 4 * 64 * 128;             // of 64 value rows: four 64-column blocks
constexpr int NK = 3, NV = 4;                   // blocks of keys, halves of values in flight
constexpr int XBYTES = 128 * 128 * 4;           // what a CTA is sent: 128 channels of all rows
constexpr int SM_Q = 0;
constexpr int SM_K = 2 * BLOCK;                 // [NK] blocks of a tile's columns
constexpr int SM_V = SM_K + NK * BLOCK;         // [NV] halves of a tile's rows
constexpr int SM_X = SM_V - XBYTES;             // received outputs between two pieces, [channel / 4][128 rows]
static_assert(SM_X >= SM_Q, "received outputs over queries and keys");
constexpr int SM_OUT = SM_V + NV * VHALF;       // 1 KB per softmax warp: rows on their way out
constexpr int SM_MAX = SM_OUT + 8 * 1024;       // [2][warpgroup][128] maxima of a tile
constexpr int SM_SUM = SM_MAX + 2 * 2 * 128 * 4;  // [2][warpgroup][128] sums of weights
constexpr int SM_SQ = SM_SUM + 2 * 2 * 128 * 4;   // [2][2 CTAs x 2][128] sums of squares
constexpr int SM_W = SM_SQ + 2 * 4 * 128 * 4;     // [256] weights of the norm
constexpr int SM_BAR = SM_W + DV * 4;
constexpr int SM_ITEM = SM_BAR + 448;             // two of struct DiffItem
constexpr int SM_ALLOC = SM_ITEM + 2 * 128 + 1024;
static_assert(SM_ALLOC <= 227 * 1024, "shared memory of a CTA");

struct Barriers {
    uint64_t qfull, qempty, kfull[2], kempty[2], vfull[NV], vempty[NV];
    uint64_t sfull[2], pready[2], vdone[2], ofull, oempty;
    uint64_t ifull[2], iempty[2], pair[4], lfull, xfull, xempty, xdone, sqfull[2], pad[NV], fin[2];
    uint32_t tmem;
};
static_assert(sizeof(Barriers) <= 448, "shared memory layout");

constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: two score buffers (P over them), then O
constexpr uint32_t kSqBytes = 4 * 128 * 4;

// Arrive (count 1) on the mbarrier at cluster address `bar`.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__global__ void __launch_bounds__(NT, 1)
    diff_wide_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const DiffTcArgs g) {
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Barriers *bars = reinterpret_cast<Barriers *>(sm + SM_BAR);
    DiffItem *items = reinterpret_cast<DiffItem *>(sm + SM_ITEM);
    float *wsm = reinterpret_cast<float *>(sm + SM_W);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DiffArgs &a = g.a;
    const int rank = (int)cluster_rank();  // the CTA's map, and the half of the channels it writes

    if (tid == 0) {
        for (uint64_t *bar : {&bars->qfull, &bars->qempty, &bars->ofull, &bars->xfull}) mbar_init(bar, 1);
        for (int s = 0; s < 2; ++s) {
            for (uint64_t *bar : {&bars->sfull[s], &bars->vdone[s], &bars->ifull[s], &bars->sqfull[s], &bars->fin[s]})
                mbar_init(bar, 1);
            mbar_init(&bars->kfull[s], 2);  // a tile's two blocks
            mbar_init(&bars->kempty[s], 1);
            mbar_init(&bars->pready[s], 9);  // softmax warps, and the next scores are queued
            mbar_init(&bars->iempty[s], 11);  // softmax, product and value load warps
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&bars->vfull[s], 1);
            mbar_init(&bars->pad[s], 1);
            mbar_init(&bars->vempty[s], 1);
        }
        for (int s = 0; s < 4; ++s) mbar_init(&bars->pair[s], 2);
        mbar_init(&bars->oempty, 8);
        mbar_init(&bars->lfull, 8);
        mbar_init(&bars->xempty, 8);  // the other CTA's softmax warps
        mbar_init(&bars->xdone, 8);
        fence_mbar_init();
        for (int s = 0; s < 2; ++s) mbar_expect_tx(&bars->sqfull[s], kSqBytes);
        mbar_expect_tx(&bars->xfull, XBYTES);
    }
    for (int i = tid; i < DV; i += NT) wsm[i] = a.norm && a.weight ? a.weight[i] : 1.f;
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
    cluster_sync_all();  // the other CTA's barriers stand before it is sent anything
    const uint32_t tmem = bars->tmem;
    bool ok = true;

    // A role's next piece of work (whole warp); null at the end or on a wait that gave up.
    int piece = 0;
    auto wait = [&](uint64_t *bar, int phase) { return (bool)__all_sync(0xffffffffu, wait_bar(bar, phase & 1)); };
    auto take = [&]() -> const DiffItem * {
        ok = __all_sync(0xffffffffu, ok) && wait(&bars->ifull[piece & 1], piece >> 1);
        return ok && items[piece & 1].valid ? &items[piece & 1] : nullptr;
    };
    auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->iempty[piece & 1]);
        ++piece;
    };

    if (warp >= 8) regs_down<kRegsOther>();
    if (warp == 11) {
        // ============================= pieces of work, their queries and keys
        // One lane throughout: a wait that is over and a copy cost a whole warp twice
        // as much, and what the loads take a tile bounds all else.
        if (lane == 0) {
            const int me = blockIdx.x / 2, all = gridDim.x / 2;
            int queries = 0, slot = 0;  // tiles asked for; the next block's slot
            int blocks = 0;             // of keys asked for
            for (int i = 0; ok; ++i) {
                if (i >= 2) ok = wait_bar(&bars->iempty[i & 1], ((i >> 1) - 1) & 1);
                if (!ok) break;
                const long long block = (long long)i * all + (i & 1 ? all - 1 - me : me);
                DiffItem &x = items[i & 1];
                const bool some = block < g.pieces;
                if (some) {
                    bool bad = false;
                    make_diff_item(g, (int)block, x, &bad);
                    if (bad) atomicOr(&g_diff_wide_error, kAttnIndex);
                }
                x.valid = some;
                mbar_arrive(&bars->ifull[i & 1]);
                if (!some) break;
                const int n = x.n, b = x.b, hk = 2 * x.hk + rank;
                if (n == 0) continue;
                if (queries > 0) {
                    ok = wait_bar(&bars->qempty, (queries - 1) & 1);
                    // the last piece's received outputs have been read
                    if (ok) ok = wait_bar(&bars->xdone, (queries - 1) & 1);
                }
                if (!ok) break;
                ++queries;
                mbar_expect_tx(&bars->qfull, 2 * BLOCK);
                tma_load_5d(sm + SM_Q, &tmq, 0, x.i0, 0, 2 * x.h + rank, b, &bars->qfull);
                const int jump = 2 * x.sink_tiles, lo = x.lo;
                int k0 = jump > 0 ? 0 : lo;
#pragma unroll 1
                for (int j = 0; j < 2 * n; ++j, ++blocks) {
                    if (blocks >= NK) {
                        const int last = (blocks - NK) >> 1;  // the slot's last tile
                        ok = wait_bar(&bars->kempty[last & 1], (last >> 1) & 1);
                        if (!ok) break;
                    }
                    uint64_t *bar = &bars->kfull[(blocks >> 1) & 1];
                    mbar_expect_tx(bar, BLOCK);
                    tma_load_5d(sm + SM_K + slot * BLOCK, &tmk, 0, k0, j & 1, hk, b, bar);
                    slot = slot == NK - 1 ? 0 : slot + 1;
                    if (j & 1) k0 = j + 1 == jump ? lo : k0 + kDiffKeys;
                }
            }
            // never leave with copies into shared memory in flight: the last phases
            // of every barrier that was armed here
            if (queries > 0 && !wait_bar(&bars->qfull, (queries - 1) & 1)) ok = false;
            for (int i = max(0, blocks - NK); i < blocks; ++i)
                if (!wait_bar(&bars->kfull[(i >> 1) & 1], (i >> 2) & 1)) ok = false;
        }
    } else if (warp == 10) {
        // ============================================================ values
        uint32_t asked = 0, turn = 0, padded = 0, pad_turn = 0;  // a bit a slot: ever, phase of the last time
        int slot = 0;                                            // of the next half
        // one lane throughout: see above
        auto ask = [&](int k0, int hv, int b, uint64_t *bar) {  // both heads' channels by one copy
            const uint32_t bit = 1u << slot;
            if (asked & bit) {
                ok = wait_bar(&bars->vempty[slot], (turn >> slot) & 1);
                if (!ok) return;
                turn ^= bit;
            }
            asked |= bit;
            mbar_expect_tx(&bar[slot], VHALF);
            tma_load_5d(sm + SM_V + slot * VHALF, &tmv, 0, k0, 0, hv, b, &bar[slot]);
        };
        while (const DiffItem *px = take()) {
            const DiffItem &x = *px;
            const int b = x.b, hv = 2 * x.hk, kl = x.kl, jump = 2 * x.sink_tiles, lo = x.lo, all = 2 * x.n;
            // halves that reach behind the last key, where padding follows, get zeros there: the
            // last ones (or some, behind sinks that end near it)
            int plain = kl < a.Tk && x.sink_tiles * kDiffKeys > kl ? 0 : all;
            if (kl < a.Tk)
                while (plain > 0 && x.key0((plain - 1) >> 1) + 64 * ((plain - 1) & 1) + 64 > kl) --plain;
            const int first = slot;
            if (lane == 0) {
                int k0 = jump > 0 ? 0 : lo;
#pragma unroll 1
                for (int half = 0; half < plain && ok;) {
                    ask(k0, hv, b, bars->vfull);
                    slot = (slot + 1) % NV;
                    k0 = ++half == jump ? lo : k0 + 64;
                }
            }
            slot = (first + plain) % NV;
            ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
            for (int half = plain; half < all && ok; ++half, slot = (slot + 1) % NV) {
                const int k0 = x.key0(half >> 1) + 64 * (half & 1);
                const uint32_t bit = 1u << slot;
                const bool pad = k0 + 64 > kl;
                uint8_t *to = sm + SM_V + slot * VHALF;
                if (lane == 0) ask(k0, hv, b, pad ? bars->pad : bars->vfull);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (!pad) continue;
                if (padded & bit) pad_turn ^= bit;
                padded |= bit;
                ok = wait(&bars->pad[slot], pad_turn >> slot);
                const int from = max(0, kl - k0) * 8;  // 16-byte units of 128-byte rows
#pragma unroll 1
                for (int u = from + lane; u < 64 * 8; u += 32)
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(to + c * 8192 + u * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->vfull[slot]);
            }
            __syncwarp();
            give_back();
        }
        // never leave with copies into shared memory in flight
        if (lane == 0) {
            for (int s = 0; s < NV; ++s) {
                if ((padded >> s & 1) && !wait_bar(&bars->pad[s], pad_turn >> s & 1)) ok = false;
                if ((asked >> s & 1) && !wait_bar(&bars->vfull[s], turn >> s & 1)) ok = false;
            }
        }
    } else if (warp == 9) {
        // ===================================================== scores' products
        const bool lead = elect_one();
        const uint64_t dq = tile_desc(smem_u32(sm + SM_Q), 128, 0, 0);
        int done = 0, used = 0;           // tiles and pieces multiplied
        int slot = 0;                     // of the next block of keys
        while (const DiffItem *px = take()) {
            const DiffItem &x = *px;
            const int n = x.n;
            if (n > 0) ok = wait(&bars->qfull, used);
#pragma unroll 1
            for (int it = 0; it < n && ok; ++it) {
                const int u = done & 1;
                const uint32_t id = idesc_bf16_f32(BM, x.width(it)) | g.negate;
                const int slot1 = slot == NK - 1 ? 0 : slot + 1;
                ok = wait(&bars->kfull[u], done >> 1);
                // the products that read the buffer's weights are done: another warp issued
                // them, and nothing but their completion orders them with these
                if (ok && done >= 2) ok = wait(&bars->vdone[u], (done >> 1) - 1);
                if (!ok) break;
                tc_fence_after();
                if (lead) {
                    const uint64_t dk = tile_desc(smem_u32(sm + SM_K), 128, 0, 0);
                    const uint64_t dk0 = dk + (uint64_t)(slot * (BLOCK >> 4)), dk1 = dk + (uint64_t)(slot1 * (BLOCK >> 4));
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_bf16(tmem + kS + 128 * u, kdesc_step(dq, 128, ks), kdesc_step(ks < 4 ? dk0 : dk1, 128, ks & 3), id,
                                 ks > 0);
                    // the last tile's value products may follow
                    if (it > 0) mbar_arrive(&bars->pready[u ^ 1]);
                    if (it == n - 1) mbar_arrive(&bars->pready[u]);
                    mma_commit(&bars->sfull[u]);
                    mma_commit(&bars->kempty[u]);
                    if (it == n - 1) mma_commit(&bars->qempty);
                }
                __syncwarp();
                slot = slot1 == NK - 1 ? 0 : slot1 + 1;
                ++done;
            }
            if (n > 0) ++used;
            give_back();
        }
        if (lead) mma_commit(&bars->fin[1]);
        __syncwarp();
        if (!wait_bar(&bars->fin[1], 0)) ok = false;
    } else if (warp == 8) {
        // ====================================================== value products
        const bool lead = elect_one();
        constexpr uint32_t id_o = idesc_bf16_f32_mn(BM, DV, false, true);
        const uint64_t dv = tile_desc_mn(smem_u32(sm + SM_V), 64, 0);
        const uint32_t o = tmem + kO;
        // 16 keys: their weights, and what the weights' rounding left
        auto values = [&](uint32_t p, uint64_t v, bool add) {
            mma_bf16_ta(o, p, v, id_o, add);
            mma_bf16_ta(o, p + 32, v, id_o, 1);
        };
        int done = 0, used = 0;  // tiles and pieces multiplied
        while (const DiffItem *px = take()) {
            const DiffItem &x = *px;
            const int n = x.n;
#pragma unroll 1
            for (int it = 0; it < n && ok; ++it) {
                const int u = done & 1, steps = x.width(it) >> 4;
                const uint32_t p = tmem + kS + 128 * u;
                const int slot0 = 2 * u, slot1 = 2 * u + 1;
                const uint64_t dv0 = dv + (uint64_t)(slot0 * (VHALF >> 4)), dv1 = dv + (uint64_t)(slot1 * (VHALF >> 4));
                ok = wait(&bars->vfull[slot0], done >> 1);
                // the last piece's output has left
                if (ok && it == 0 && used > 0) ok = wait(&bars->oempty, used - 1);
                if (ok) ok = wait(&bars->pready[u], done >> 1);
                if (!ok) break;
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps) values(p + 8 * ks, mndesc_step(dv0, ks), ks > 0 || it > 0);
                    mma_commit(&bars->vempty[slot0]);
                }
                __syncwarp();
                ok = wait(&bars->vfull[slot1], done >> 1);
                if (!ok) break;
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int ks = 4; ks < 8; ++ks)
                        if (ks < steps) values(p + 64 + 8 * (ks - 4), mndesc_step(dv1, ks - 4), true);
                    mma_commit(&bars->vempty[slot1]);
                    mma_commit(&bars->vdone[u]);
                    if (it == n - 1) mma_commit(&bars->ofull);
                }
                __syncwarp();
                ++done;
            }
            if (n > 0) ++used;
            give_back();
        }
        if (lead) mma_commit(&bars->fin[0]);
        __syncwarp();
        if (!wait_bar(&bars->fin[0], 0)) ok = false;
    } else if (warp < 8) {
        // ========================== softmax, then the difference and its norm
        regs_up<kRegsSoftmax>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, base_o = tmem + lanes + kO;
        const float2 c2 = make_float2(g.c, g.c);
        float *maxima = reinterpret_cast<float *>(sm + SM_MAX);
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
                const int u = seen & 1;
                const uint32_t ts = tmem + lanes + kS + 128 * u + 64 * t;
                const bool whole = it >= all0 && it < all1;
                const int k0 = x.key0(it) + 64 * t, end = min(p + 1, x.limit(it));
                ok = wait(&bars->sfull[u], seen >> 1);
                if (!ok) break;
                tc_fence_after();
                // the last scores are there: no product reads the keys that the other CTA
                // writes its outputs over
                if (it == n - 1 && lane == 0) arrive_remote(map_to_rank(smem_u32(&bars->xempty), rank ^ 1));
                if (!whole) {
                    // -inf over the scores that a row does not see, in tensor memory, so
                    // that one code serves all tiles
#pragma unroll 1
                    for (int ch = 0; ch < 2; ++ch) {
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
                float s[2][32];
                tmem_ld32(ts, s[0]);
                tmem_ld32(ts + 32, s[1]);
                tmem_ld_wait(s[0], s[1]);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[ch][i], s[ch][i + 1]);
                // the other 64 keys' maximum, from the warp of the same rows
                const float own = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                maxima[(u * 2 + t) * 128 + row] = own;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->pair[warp & 3]);
                ok = wait(&bars->pair[warp & 3], seen);
                if (!ok) break;
                const float mn = fmaxf(own, maxima[(u * 2 + (t ^ 1)) * 128 + row]);
                const bool grow = mn > m && (m == -INFINITY || (mn - m) * g.c > 8.f);
                // a row that has seen nothing yet has l = 0 and zeros in O (or O unset)
                if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
                    // the last tile's products are in O; this warpgroup's half of it
                    ok = wait(&bars->vdone[u ^ 1], (seen - 1) >> 1);
                    if (!ok) break;
                    tc_fence_after();
                    // no fma here: both products as the exponent's base has them
                    const float f = grow && m != -INFINITY ? ex2(__fsub_rn(__fmul_rn(m, g.c), __fmul_rn(mn, g.c))) : 1.f;
                    l *= f;
#pragma unroll 1
                    for (int ch = 0; ch < DV / 32; ++ch) {
                        float v[16];
                        tmem_ld16(base_o + 128 * t + 16 * ch, v);
                        tmem_ld_wait(v);
                        uint32_t r[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i] * f);
                        tmem_st16(base_o + 128 * t + 16 * ch, r);
                    }
                }
                if (grow) m = mn;
                const float base = m == -INFINITY ? 0.f : -__fmul_rn(m, g.c);
                const float2 b2 = make_float2(base, base);
                float2 sum[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    uint32_t r[16], rest[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = fma2(make_float2(s[ch][2 * i], s[ch][2 * i + 1]), c2, b2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        sum[i & 3] = add2(sum[i & 3], e);
                        r[i] = pack2_rest(e, rest[i]);
                    }
                    tmem_st16(ts + 16 * ch, r);
                    tmem_st16(ts + 32 + 16 * ch, rest);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->pready[u]);
                const float2 two = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += two.x + two.y;
                ++seen;
            }
            const int slot = used & 1;
            float *sums = reinterpret_cast<float *>(sm + SM_SUM) + slot * 256;
            sums[t * 128 + row] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->lfull);
            if (ok) ok = wait(&bars->lfull, used);
            if (!ok) break;
            l = sums[row] + sums[128 + row];
            // the rounding of the exponent's base took the weights' range
            if (m != -INFINITY && !(l >= 0x1p-40f)) l = NAN;
            // no key, or only scores of -inf: zeros
            const float f = (l == 0.f ? 0.f : 1.f / l) * (rank ? -a.lambda[x.h] : 1.f);
            // rows of a warp side by side, so that a store of it writes 512 bytes in a row
            uint8_t *got = sm + SM_X + (t * 16 * 128 + row) * 16;
            const uint32_t peer = map_to_rank(smem_u32(got), rank ^ 1),
                           peer_bar = map_to_rank(smem_u32(&bars->xfull), rank ^ 1);
            ok = wait(&bars->xempty, used);
            if (ok) ok = wait(&bars->ofull, used);
            if (!ok) break;
            tc_fence_after();
            // what is sent leaves at some 32 bytes a cycle; the CTA's own channels meanwhile
            float y[64];
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float v[32], own[32];
                tmem_ld32(base_o + 128 * (rank ^ 1) + 64 * t + c, v);
                tmem_ld32(base_o + 128 * rank + 64 * t + c, own);
                tmem_ld_wait(v, own);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    st_async_v4(peer + (uint32_t)((c / 4 + i) * 2048), __fmul_rn(v[4 * i], f), __fmul_rn(v[4 * i + 1], f),
                                __fmul_rn(v[4 * i + 2], f), __fmul_rn(v[4 * i + 3], f), peer_bar);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[c + i] = __fmul_rn(own[i], f);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->oempty);
            ok = wait(&bars->xfull, used);
            if (!ok) break;
            if (tid == 0) mbar_expect_tx(&bars->xfull, XBYTES);  // the next piece's
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 z = *reinterpret_cast<const float4 *>(got + i * 2048);
                // each product rounded, so that equal maps cancel exactly
                y[4 * i] = __fadd_rn(y[4 * i], z.x), y[4 * i + 1] = __fadd_rn(y[4 * i + 1], z.y);
                y[4 * i + 2] = __fadd_rn(y[4 * i + 2], z.z), y[4 * i + 3] = __fadd_rn(y[4 * i + 3], z.w);
            }
            fence_async_smem();  // queries and keys come there next
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->xdone);
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; ++i) part[i & 3] = fmaf(y[i], y[i], part[i & 3]);
            float squares = marked_squares(y, (part[0] + part[1]) + (part[2] + part[3]));
            if (a.norm) {
                // the row's other channels: every warp sends its rows' sums to both CTAs,
                // four a lane
                const float *sq = reinterpret_cast<const float *>(sm + SM_SQ) + slot * 4 * 128;
                float four[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) four[i] = __shfl_sync(0xffffffffu, squares, (4 * lane + i) & 31);
                if (lane < 8) {
                    const uint32_t dst = smem_u32(sq + (rank * 2 + t) * 128 + (row & ~31) + 4 * lane);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        st_async_v4(map_to_rank(dst, r), four[0], four[1], four[2], four[3],
                                    map_to_rank(smem_u32(&bars->sqfull[slot]), r));
                }
                ok = wait(&bars->sqfull[slot], used >> 1);
                if (!ok) break;
                squares = (sq[row] + sq[128 + row]) + (sq[256 + row] + sq[384 + row]);
                // the slot's next use is two pieces on (its sums may come before it is armed)
                if (tid == 0) mbar_expect_tx(&bars->sqfull[slot], kSqBytes);
            }
            const float scale = diff_scale(a.norm, squares, D, a.eps);
            marked = marked || (row < x.rows && scale != scale);
            ++used;
            // Rows leave through the warp's shared memory, 16 channels at a time, so that a
            // store writes whole 32-byte sectors of 16 rows.
            uint8_t *out = sm + SM_OUT + warp * 1024;
            const int w0 = 32 * (warp & 3), rows = x.rows, r16 = lane >> 1, c2 = lane & 1;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + x.b * a.os.b + (2 * x.h + rank) * a.os.h +
                               (long long)(x.i0 + w0 + r16) * a.os.t + 64 * t + 8 * c2;
            const float4 *weight = reinterpret_cast<const float4 *>(wsm + 128 * rank + 64 * t);
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 z = weight[c / 4 + i];
                    const float *yi = y + c + 4 * i;
                    w[2 * i] = pack2(yi[0] * scale * z.x, yi[1] * scale * z.y);
                    w[2 * i + 1] = pack2(yi[2] * scale * z.z, yi[3] * scale * z.w);
                }
                __syncwarp();  // the last channels have left
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4 *>(out + lane * 32 + (i ^ ((lane >> 2) & 1)) * 16) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rr = 16 * i + r16;
                    const uint4 z = *reinterpret_cast<const uint4 *>(out + rr * 32 + (c2 ^ ((rr >> 2) & 1)) * 16);
                    if (w0 + rr < rows) *reinterpret_cast<uint4 *>(o + 16 * i * a.os.t + c) = z;
                }
            }
            give_back();
        }
        mend_marked<D>(g, __any_sync(0xffffffffu, ok && marked), blockIdx.x / 2, gridDim.x / 2, 128 * rank, 64);
    }

    if (!ok) atomicOr(&g_diff_wide_error, kAttnTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
    cluster_sync_all();  // no CTA leaves while another may send to it
}

}  // namespace

// ensure_smem_attr slot 226 belongs to this file.
cudaError_t launch_diff_wide_tc(const DiffArgs &a, cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    cudaError_t e = blocks_map(&mq, a.q, a.qs, a.B, 2 * a.H, a.Tq, D, BM, 1);
    if (e == cudaSuccess) e = blocks_map(&mk, a.k, a.ks, a.B, 2 * a.Hk, a.Tk, D, kDiffKeys, 1, true);
    if (e == cudaSuccess) e = blocks_map(&mv, a.v, a.vs, a.B, 2 * a.Hk, a.Tk, D, 64, 2);
    if (e != cudaSuccess) return e;
    const DiffTcArgs g = diff_tc_args(a, D);
    auto *fn = diff_wide_kernel;
    e = ensure_smem_attr(reinterpret_cast<const void *>(fn), SM_ALLOC, 226);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(std::min(g.pieces, kClusterRoom[0][2] / 2) * 2));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = SM_ALLOC;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, mq, mk, mv, g);
}

int attn_errors_diff_wide() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_diff_wide_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_diff_wide_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
