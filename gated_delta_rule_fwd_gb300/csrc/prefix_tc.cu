// lr_step_paged_prefix in bf16 on the tensor cores (tcgen05): the part of a
// step's attention that lies in the prefix shared by the batch.
//
// The query rows of all sequences that read one key head (N times Hq / Hk) are
// worked on as one matrix, so the prefix's keys and values are read once for
// them instead of once per sequence.  A CTA takes up to two 128-row query tiles
// and a run of 128-key tiles of the prefix; the tiles alternate on the tensor
// pipe as in window_tc.cu:
//
//     S = Q K^T,   P = exp2(c S - b) (softmax_tile),   O += P V
//
// It leaves (maximum, sum, unnormalised output) of its run for each row; the
// step over each sequence's own keys joins them (step_paged.cu).  Parts refer
// to the exact maximum: weights 2^(c s - b), b = c m rounded, are rescaled by
// 2^(b - c m) on their way out.
//
// With few rows the bound is the read of the prefix, with many the tensor pipe.
// Measured (d = 128, 32 heads on 8): 128 sequences behind 16384 tokens 36 us, 1.5 us a key
// tile of both query tiles (70 % of the pipe's rate; the chain is that of diff_tc.cu) and
// 14 us to start, to write 19 MB of parts and to read them; 4 sequences behind 2048, with
// their own tokens, 12.5 us.  Tiles in 64-key halves: 44 instead of 37 us.
// Pages: a tile is copied in boxes of min(page, 128) rows.  Rows of the last page
// behind the prefix are set to zero as they are loaded; a page outside the pool is
// read as page 0 and masked.
//
// Roles of the 384 threads: warps 0-3 queries, softmax and output of query tile
// 0, warps 4-7 of tile 1, warps 8 and 9 issue the products of tiles 0 and 1, warp
// 10 the TMA loads.  Every wait is bounded (lr_device_status).
#include <limits.h>

#include "attn_internal.cuh"
#include "attn_step.cuh"
#include "attn_tc.cuh"
#include "tc_common.cuh"

namespace lr {
namespace {

using namespace tc;

__device__ unsigned g_prefix_error = 0;

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
    static constexpr int KV = 2 * TILE;              // also the rows on their way out, 4 KB a softmax warp
    static constexpr int BAR = KV + NS * TILE;
    static constexpr int BYTES = BAR + 384;
    static constexpr int ALLOC = BYTES + 1024;
};

struct Barriers {
    uint64_t qfull[2], sfull[2], pready[2][2], ofull[2], fin[2];
    uint64_t full[8], empty[8], pad;
    uint32_t tmem, pipe;  // pipe: 1 while a warp issues products
    int broken;           // a page of the run lies outside the pool
};
static_assert(sizeof(Barriers) <= 384, "shared memory layout");

constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S0, S1 (P over them), then O0, O1

struct TcArgs {
    StepArgs a;
    PrefixPlan plan;
    float c;          // the scores' factor, positive
    unsigned negate;  // idesc bit: scores of -Q (scale < 0)
    int zero;         // scale 0: scores count as zeros
};

template <int D>
__global__ void __launch_bounds__(NT, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const TcArgs g) {
    using L = Layout<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Barriers *bars = reinterpret_cast<Barriers *>(sm + L::BAR);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const StepArgs &a = g.a;
    const PrefixPlan &plan = g.plan;
    const int G = a.Hq / a.Hk, rows = a.N * G;
    int id = blockIdx.x;
    const int run = id % plan.parts;
    id /= plan.parts;
    const int hk = id % a.Hk, row0 = id / a.Hk * 2 * BM;
    const int active = rows - row0 > BM ? 2 : 1;  // query tiles with rows
    const int begin = run * plan.chunk, n = max(0, min(plan.tiles, begin + plan.chunk) - begin);
    auto key0 = [&](int it) {
        it += begin;
        return BN * (it < plan.sink_tiles ? it : it - plan.sink_tiles + plan.first);
    };
    // columns that the tile needs, a multiple of 32
    auto width = [&](int it) {
        const int w = a.plen - key0(it);
        return w >= BN ? BN : (w + 31) & ~31;
    };

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->qfull[t], 4);
            mbar_init(&bars->sfull[t], 1);
            mbar_init(&bars->pready[t][0], 4);  // the first 64 columns of P
            mbar_init(&bars->pready[t][1], 4);  // the others
            mbar_init(&bars->ofull[t], 1);
            mbar_init(&bars->fin[t], 1);
        }
        for (int s = 0; s < L::NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], active);
        }
        mbar_init(&bars->pad, 1);
        bars->pipe = 0;
        bars->broken = 0;
        fence_mbar_init();
    }
    if (warp == 10 && lane == 0) {
        for (const CUtensorMap *map : {&tmk, &tmv}) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    if (warp == 8) {
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    let_next_start();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    bool ok = true;

    if (warp >= 8) regs_down<kRegsOther>();
    if (warp == 10) {
        // ============================================================ loads
        int pads = 0, seq = 0;
        const int box = min(1 << a.page_log2, BN), in_page = (1 << a.page_log2) - 1;
#pragma unroll 1
        for (; seq < 2 * n && ok; ++seq) {
            const int s = seq % L::NS, k0 = key0(seq >> 1);
            if (seq >= L::NS) ok = __all_sync(0xffffffffu, wait_bar(&bars->empty[s], (seq / L::NS - 1) & 1));
            if (!ok) break;
            uint8_t *to = sm + L::KV + s * L::TILE;
            const int keys = min(BN, a.plen - k0), boxes = (keys + box - 1) / box;
            // values behind the prefix: zeros, whatever the last page or the buffer holds
            const bool pad = (seq & 1) && keys < BN;
            uint64_t *bar = pad ? &bars->pad : &bars->full[s];
            if (lane == 0) mbar_expect_tx(bar, boxes * box * 128 * L::KB);
            __syncwarp();
            if (lane < boxes) {  // a box a lane: at most eight
                const int key = k0 + lane * box;
                int page = a.ptable[key >> a.page_log2];
                if (page < 0 || page >= a.num_pages) page = 0;
                // the copies of whole tiles bring both blocks of columns
                for (int kb = 0; kb < (box == BN ? 1 : L::KB); ++kb)
                    tma_load_5d(to + kb * 16384 + lane * box * 128, seq & 1 ? &tmv : &tmk, 0, key & in_page, kb, hk, page,
                                bar);
            }
            __syncwarp();
            if (pad) {
                ok = __all_sync(0xffffffffu, wait_bar(&bars->pad, pads & 1));
                ++pads;
#pragma unroll 1
                for (int u = keys * 8 + lane; u < BN * 8; u += 32)  // 16-byte units of 128-byte rows
                    for (int kb = 0; kb < L::KB; ++kb)
                        *reinterpret_cast<uint4 *>(to + kb * 16384 + u * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->full[s]);
            }
        }
        // never leave with copies into shared memory in flight
        if (lane == 0) {
            if (pads > 0 && !wait_bar(&bars->pad, (pads - 1) & 1)) ok = false;
            for (int i = max(0, seq - L::NS); i < seq; ++i)
                if (!wait_bar(&bars->full[i % L::NS], (i / L::NS) & 1)) ok = false;
        }
    } else if ((warp == 8 || warp == 9) && warp - 8 < active) {
        // ========================================================= products
        const int t = warp - 8;
        const uint32_t s_t = tmem + kS + t * BN, o_t = tmem + kO + t * 128, kv_s = smem_u32(sm + L::KV);
        const uint32_t id_o = idesc_bf16_f32_mn(BM, D, false, true);
        const uint64_t dq = tile_desc(smem_u32(sm + L::Q) + t * L::TILE, 128, 0, 0);
        const bool lead = elect_one();
        auto stage_wait = [&](int seq) {
            return __all_sync(0xffffffffu, wait_bar(&bars->full[seq % L::NS], (seq / L::NS) & 1));
        };
        auto scores = [&](int it) {
            const int s = 2 * it % L::NS;
            const uint64_t dk = tile_desc(kv_s + s * L::TILE, 128, 0, 0);
            const uint32_t id_s = idesc_bf16_f32(BM, width(it)) | g.negate;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                mma_bf16(s_t, kdesc_step(dq, 128, ks), kdesc_step(dk, 128, ks), id_s, ks > 0);
            mma_commit(&bars->sfull[t]);
            mma_commit(&bars->empty[s]);
        };
        if (n > 0) {
            ok = __all_sync(0xffffffffu, wait_bar(&bars->qfull[t], 0)) && stage_wait(0);
            if (lead && ok) scores(0);
            __syncwarp();
        }
#pragma unroll 1
        for (int it = 0; it < n && ok; ++it) {
            if (it + 1 < n) ok = stage_wait(2 * it + 2);
            if (ok) ok = stage_wait(2 * it + 1);
            const int sv = (2 * it + 1) % L::NS, steps = width(it) >> 4;
            const uint64_t dv = tile_desc_mn(kv_s + sv * L::TILE, 128, 0);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->pready[t][0], it & 1));
            if (!ok) break;
            tc_fence_after();
            // O += P V, 64 keys at a time as P comes
            if (lead) {
                take_pipe(&bars->pipe);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    if (ks < steps) mma_bf16_ta(o_t, s_t + 8 * ks, mndesc_step(dv, ks), id_o, ks > 0 || it > 0);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, wait_bar(&bars->pready[t][1], it & 1));
            if (!ok) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
                for (int ks = 4; ks < BN / 16; ++ks)
                    if (ks < steps) mma_bf16_ta(o_t, s_t + 8 * ks, mndesc_step(dv, ks), id_o, 1);
                mma_commit(&bars->empty[sv]);
                if (it + 1 < n) scores(it + 1);
                else mma_commit(&bars->ofull[t]);
                free_pipe(&bars->pipe);
            }
            __syncwarp();
        }
        if (lead) mma_commit(&bars->fin[t]);
        __syncwarp();
        if (!wait_bar(&bars->fin[t], 0)) ok = false;
    } else if (warp < 8 && warp >> 2 < active) {
        // ============================ queries, softmax, then the run's part
        regs_up<kRegsSoftmax>();
        const int t = warp >> 2, row = row0 + t * BM + (tid & 127);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + kS + t * BN, to = tmem + lanes + kO + t * 128;
        const int seq = min(row, rows - 1) / G, len = a.lens[seq];
        // a row that is not computed sees nothing and leaves nothing
        const bool on = row < rows && len >= 0 && len <= a.max_len;
        const int head = seq * a.Hq + hk * G + row - seq * G;
        const int lo = on ? window_start(a.plen + len - 1, a.window) : INT_MAX, sinks = min(a.all_sinks, a.plen);
        const int lo_most = __reduce_max_sync(0xffffffffu, on ? lo : 0);
        {
            // the row into the swizzled query tile; zeros behind the last row
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + (size_t)head * D);
            uint8_t *qt = sm + L::Q + t * L::TILE;
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch)
                *reinterpret_cast<uint4 *>(qt + sw128_offset(tid & 127, 8 * ch, 128)) =
                    row < rows ? q[ch] : make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->qfull[t]);
        }
        // pages of the run, 16 keys at a time, while the first tiles are on their way
        for (int i = tid; i < n * (BN / 16); i += active * BM) {
            const int key = key0(i / (BN / 16)) + i % (BN / 16) * 16;
            if (key >= a.plen) continue;
            const int page = a.ptable[key >> a.page_log2];
            if (page < 0 || page >= a.num_pages) {
                bars->broken = 1;
                atomicOr(&g_prefix_error, kAttnIndex);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"r"(active * BM) : "memory");  // the softmax warps
        const bool broken = bars->broken;
        float m = -INFINITY, l = 0.f;
        for (int it = 0; it < n && ok; ++it) {
            const int k0 = key0(it);
            const bool whole = k0 + BN <= a.plen && (k0 >= lo_most || k0 + BN <= sinks) && !broken;
            ok = __all_sync(0xffffffffu, wait_bar(&bars->sfull[t], it & 1));
            if (!ok) break;
            tc_fence_after();
            auto keep = [&](int ch) {
                const int kc = k0 + 32 * ch;
                uint32_t see = low_bits(a.plen - kc) & (~low_bits(lo - kc) | low_bits(sinks - kc));
                if (broken)
                    for (int i = 0; i < 2; ++i) {
                        const int key = kc + 16 * i, page = key < a.plen ? a.ptable[key >> a.page_log2] : 0;
                        if (page < 0 || page >= a.num_pages) see &= i ? 0x0000ffffu : 0xffff0000u;
                    }
                return see;
            };
            softmax_tile<D, false>(ts, to, g.c, whole, keep, m, l, &bars->pready[t][0], &bars->pready[t][1]);
        }
        // every product of both tiles has read its operands: their place is free
        for (int u = 0; u < active; ++u)
            if (n > 0 && ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->ofull[u], 0));
        if (ok && n > 0) {
            tc_fence_after();
            // weights relative to the exact maximum
            const float b = __fmul_rn(m, g.c), shift = m == -INFINITY ? 1.f : ex2(-fmaf(m, g.c, -b));
            l *= shift;
            if (m != -INFINITY && !(l >= 0x1p-40f)) l = NAN;  // the rounding of b took the weights' range
            const size_t at = (size_t)head * plan.parts + run;
            if (on) a.pml[at] = make_float2(g.zero && m != -INFINITY ? 0.f : m, l);
            uint8_t *out = sm + L::KV + warp * 4096;
            const int r8 = lane >> 3, c8 = lane & 7, mine = on ? head : -1;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                float v[32];
                tmem_ld32(to + 32 * ch, v);
                tmem_ld_wait(v);
                __syncwarp();  // the last channels have left
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(out + lane * 128 + (i ^ (lane & 7)) * 16) = make_float4(
                        v[4 * i] * shift, v[4 * i + 1] * shift, v[4 * i + 2] * shift, v[4 * i + 3] * shift);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = 4 * i + r8, to_head = __shfl_sync(0xffffffffu, mine, rr);
                    const float4 x = *reinterpret_cast<const float4 *>(out + rr * 128 + (c8 ^ (rr & 7)) * 16);
                    if (to_head >= 0)
                        *reinterpret_cast<float4 *>(a.po + ((size_t)to_head * plan.parts + run) * D + 32 * ch + 4 * c8) = x;
                }
            }
        }
    }

    if (!ok) atomicOr(&g_prefix_error, kAttnTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const StepArgs &a, const PrefixPlan &plan, int slot, cudaStream_t stream) {
    using L = Layout<D>;
    CUtensorMap mk, mv;
    const int page = 1 << a.page_log2, box = page < 128 ? page : 128;
    cudaError_t e = pool_map(&mk, a.k, D, page, a.Hk, a.num_pages, box, 1, box < BN);
    if (e == cudaSuccess) e = pool_map(&mv, a.v, D, page, a.Hk, a.num_pages, box, 1, box < BN);
    if (e != cudaSuccess) return e;
    TcArgs g;
    g.a = a;
    g.plan = plan;
    // scale 0: as in window_tc.cu
    g.c = a.scale == 0.f ? 0x1p-149f : score_factor(a.scale).c;
    g.negate = a.scale < 0.f ? 1u << 13 : 0u;
    g.zero = a.scale == 0.f;
    auto *fn = prefix_tc_kernel<D>;
    e = ensure_smem_attr(reinterpret_cast<const void *>(fn), L::ALLOC, slot);
    if (e != cudaSuccess) return e;
    const long long blocks = ((long long)a.N * (a.Hq / a.Hk) + 2 * BM - 1) / (2 * BM);
    fn<<<(unsigned)(blocks * a.Hk * plan.parts), NT, L::ALLOC, stream>>>(mk, mv, g);
    return cudaGetLastError();
}

}  // namespace

// ensure_smem_attr slots 230..232 belong to this file.
cudaError_t launch_prefix_tc(const StepArgs &a, const PrefixPlan &plan, int d, cudaStream_t stream) {
    if (d == 32) return launch<32>(a, plan, 230, stream);
    if (d == 64) return launch<64>(a, plan, 231, stream);
    return launch<128>(a, plan, 232, stream);
}

int attn_errors_prefix_tc() {
    unsigned h = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&h, g_prefix_error, sizeof(h)) != cudaSuccess) return -1;
    if (h) cudaMemcpyToSymbol(g_prefix_error, &zero, sizeof(h));
    return (int)h;
}

}  // namespace lr
