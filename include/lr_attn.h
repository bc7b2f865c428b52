/*
 * lr_attn.h -- C ABI of liblr's softmax-attention operators: the layers that
 * hybrid stacks place between the fixed-size memories of lr.h.
 *
 *   lr_qk_norm_rope   RMS norm of every query and key head and the position
 *                     rotation in one pass, with an optional write of keys
 *                     and values into a paged cache
 *   lr_qk_norm_rope_axes  the same with positions of several axes (time, height,
 *                     width), as prompts with images and video have them
 *   lr_fwd_window     causal attention over whole sequences, limited to a
 *                     sliding window and a few first tokens (sinks)
 *   lr_step_paged     the same attention for one new token per sequence over
 *                     the paged cache
 *   lr_step_paged_prefix  that step for a batch that shares a long prefix, whose
 *                     keys and values are read once for all
 *   lr_fwd_diff       differential attention over whole sequences: the
 *                     difference of two softmax maps, with its norm
 *   lr_step_paged_diff  the same for one new token per sequence over the paged
 *                     cache
 *
 * Conventions are those of lr.h: device pointers owned by the caller, 16-byte
 * aligned (int32 arrays: 4-byte); arguments validated on the host before any launch, so that a call
 * that returns an error has launched nothing; work enqueued on `stream` of
 * the current device without synchronising; no allocation, no state kept
 * between calls, no exceptions.  Values are fp32 or bf16 (lr_dtype); sums,
 * norms, rotations and softmax statistics are fp32, and each result is
 * rounded once when it is stored.  One rounding more: where the type is bf16,
 * a softmax weight is rounded to bf16 for its product with a value (the sum of
 * the weights takes it unrounded), which moves an output by up to 2^-8 of the
 * weighted mean of |v|; against weights of 32 bits the error of a result is
 * 1.2 to 1.4 times as large.
 *
 * Scores: q . k is formed in fp32, and the scale applies to differences of it,
 * so a finite scale takes no finite q . k out of range.  A key whose q . k
 * times the scale's sign is -inf weighs nothing; one where it is NaN or +inf
 * makes its rows NaN.  With all scores in range, a channel in which a row sees
 * an infinite value is that infinity however small the weight, with both signs
 * or a NaN it is NaN, and finite values average without overflow.
 *
 * Heads: Hq query heads share Hk key/value heads, Hq a multiple of Hk; query
 * head h reads key head h / (Hq / Hk).  Head widths d: 32, 64, 128.
 *
 * Values that live on the device (positions, lengths, block tables) cannot be
 * checked on the host.  The kernels bound every address that they form from
 * them: a page outside the pool or a length beyond its limit is left out, and
 * lr_device_status then reports LR_ERR_INDEX.
 */
#ifndef LR_ATTN_H_
#define LR_ATTN_H_

#include "lr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides, in elements, of a [B, H, T, d] tensor whose channels are
 * contiguous: any order of batch, head and token, as a fused projection
 * leaves them.  Each stride is positive and a multiple of 16 bytes where its
 * size is above 1 (else LR_ERR_ALIGN; not positive: LR_ERR_SHAPE). */
typedef struct {
    long long b, h, t;
} lr_strides;

/* A paged key/value cache: pools [num_pages, Hk, page, d] and, per sequence,
 * the page numbers of its tokens in order.  Token p of sequence n is row
 * p % page of page table[n][p / page].  Sequences may share pages that are
 * only read. */
typedef struct {
    void *k, *v;       /* [num_pages, Hk, page, d], contiguous                    */
    const int *table;  /* [B, max_pages] int32                                    */
    int num_pages;     /* >= 1                                                    */
    int page;          /* tokens per page: 16, 32, 64, 128 or 256                 */
    int max_pages;     /* >= 1; page * max_pages <= 2^30                          */
} lr_paged;

#define LR_QK_NORM 0x1u        /* y = weight * x / sqrt(mean(x^2) + eps), per head */
#define LR_QK_INTERLEAVED 0x2u /* rotate channels (2i, 2i+1), else (i, i + rot/2)  */
#define LR_QK_ZERO_Q 0x8u      /* padding's rows of q_out are written as zeros     */
#define LR_QK_ZERO_K 0x10u     /* the same for k_out (where it is given)           */

typedef struct {
    unsigned flags;          /* OR of LR_QK_*                                       */
    const float *q_weight;   /* [d] fp32, or NULL for ones (LR_QK_NORM)             */
    const float *k_weight;   /* [d] fp32, or NULL for ones (LR_QK_NORM)             */
    float eps;               /* >= 0, finite                                        */
    int rot;                 /* rotated channels, the first of each head: a
                                multiple of 16 up to d; 0: no rotation              */
    const double *inv_freq;  /* [rot / 2] fp64, radians per position (finite)       */
} lr_qk_maps;

/*
 * For every token t of sequence b, at position p = positions[b][t]:
 *
 *     y   = x, or its RMS norm over the d channels times the weight
 *     (a', b') = (a cos th - b sin th, b cos th + a sin th),  th = p inv_freq[i],
 *                for the rot/2 channel pairs (a, b) of y; other channels pass
 *
 * for each query and key head.  Squares are summed in fp32: a head whose
 * values pass 1.8e19 has a norm beyond it and comes out as zeros.  Angles are
 * formed from the product taken modulo a full turn in 64-bit fixed point, so
 * they stay accurate to fp32 at every position an int holds and every frequency
 * up to 2^50.
 *
 *   q, qs      [B, Hq, T, d] with strides qs
 *   k, ks      [B, Hk, T, d] with strides ks
 *   positions  [B, T] int32, or NULL for p = t.  A negative position marks
 *              padding: nothing of that token is written anywhere, but for the
 *              zeros that LR_QK_ZERO_Q and LR_QK_ZERO_K ask for.
 *   q_out      [B, Hq, T, d] contiguous, written
 *   k_out      [B, Hk, T, d] contiguous, written, or NULL
 *   v, vs      [B, Hk, T, d] with strides vs: with a cache only, else NULL
 *   cache      NULL, or the pools that receive the keys and v at row p of
 *              their sequence (table [B, max_pages])
 *
 * k_out may be NULL only with a cache.  The positions of a sequence in one
 * call are distinct (of two equal ones either may end in the cache).  Outputs
 * overlap neither the inputs nor each other.  B, T, Hq, Hk >= 1 (T == 0 does
 * nothing).  One kernel.
 */
lr_status lr_qk_norm_rope(const void *q, lr_strides qs, const void *k, lr_strides ks,
                          const int *positions, const lr_qk_maps *maps, void *q_out, void *k_out,
                          const void *v, lr_strides vs, const lr_paged *cache, int B, int T,
                          int Hq, int Hk, int d, lr_dtype dt, cudaStream_t stream);

#define LR_MAX_AXES 16

/*
 * lr_qk_norm_rope with positions of several axes: channel pair i of a token is
 * turned by th = positions[axis[i]][b][t] inv_freq[i].  Where a token's keys go
 * in the cache is a matter of its place in the sequence, not of its positions:
 *
 *   positions  [axes, B, T] int32, any values; 1 <= axes <= LR_MAX_AXES
 *   axis       [rot / 2] int32, 0..axes-1 (others count as 0 and are reported
 *              as LR_ERR_INDEX); positions and axis are not read where rot is 0
 *   places     [B, T] int32, the cache row of the token, or NULL for t.  A
 *              negative place marks padding, as a negative position does there.
 *
 * All else is as for lr_qk_norm_rope.  The places of a sequence in one call are
 * distinct.
 */
lr_status lr_qk_norm_rope_axes(const void *q, lr_strides qs, const void *k, lr_strides ks,
                               const int *positions, const int *axis, int axes, const int *places,
                               const lr_qk_maps *maps, void *q_out, void *k_out, const void *v,
                               lr_strides vs, const lr_paged *cache, int B, int T, int Hq, int Hk,
                               int d, lr_dtype dt, cudaStream_t stream);

/*
 * Causal attention with a sliding window and sinks.  Query row i of sequence
 * b stands at position p = k_len[b] - q_len[b] + i (the queries are the last
 * tokens of the keys' sequence) and sees key j iff
 *
 *     0 <= j < k_len[b],  j <= p,  and  (j > p - window  or  j < sinks);
 *
 *     o_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys it sees.
 *
 * A row that sees no key (p < 0, or an empty sequence), or only keys whose
 * score is -inf, is written as zeros.  Rows i >= q_len[b] are left as they
 * were.  What a row does not see cannot change it, whatever it holds: NaN and
 * infinities in masked rows of k and v are not read into any sum.
 *
 *   q, qs   [B, Hq, Tq, d] with strides     k, ks, v, vs  [B, Hk, Tk, d]
 *   q_len   [B] int32 or NULL (Tq)          k_len         [B] int32 or NULL (Tk)
 *           (lengths outside 0..Tq and 0..Tk are brought into that range and
 *           reported as LR_ERR_INDEX)
 *   o, os   [B, Hq, Tq, d] with strides, written; overlaps no input
 *   window  >= 1; Tk or more: plain causal attention
 *   sinks   >= 0        scale  finite
 *   B, Hq, Hk >= 1; Tq >= 0 (0 does nothing), Tk >= 0 (0: zeros)
 */
lr_status lr_fwd_window(const void *q, lr_strides qs, const void *k, lr_strides ks, const void *v,
                        lr_strides vs, const int *q_len, const int *k_len, void *o, lr_strides os,
                        int B, int Hq, int Hk, int Tq, int Tk, int d, int window, int sinks,
                        float scale, lr_dtype dt, cudaStream_t stream);

/*
 * Differential attention.  H pairs of query heads share Hk pairs of key heads
 * (H a multiple of Hk; pair h reads pair g = h / (H / Hk)).  Pair h has the
 * query heads 2h and 2h + 1, one for each softmax map, and the key heads 2g and
 * 2g + 1 likewise; its value row is the 2 d channels of the value heads 2g and
 * 2g + 1 in that order, and so is its output:
 *
 *     A_m  = softmax_j(scale q_(2h+m),i . k_(2g+m),j)      m = 0, 1
 *     y_i  = sum_j (A_0 - lambda[h] A_1) [v_2g,j  v_(2g+1),j]
 *     [o_2h,i  o_(2h+1),i] = y_i, or weight y_i / sqrt(mean(y_i^2) + eps)
 *
 * over the keys that row i sees, as for lr_fwd_window (window, sinks, lengths,
 * strides and what a masked row may hold are as there).  The difference, its
 * mean square and its norm are formed in fp32.  The difference takes away what the
 * maps have in common, but not the rounding of their weights to bf16 (see above), so
 * lr_fwd_diff and lr_step_paged_diff multiply what that rounding left as well: weights
 * of 16 bits, and the error of 32-bit ones.  Equal maps cancel exactly.
 * A row that sees no key, or whose y is zero, is zeros.  With eps 0, rows below
 * 1e-19 lose digits, as their squares do; a mean that underflows counts as 2^-149.
 * Where a map's row is not finite (lr_fwd_window says when) the formulas hold as
 * fp32 arithmetic has them; a row whose squares sum to more than fp32 holds is
 * divided by infinity.
 */
#define LR_DIFF_NORM 0x1u /* the root-mean-square norm over the pair's 2 d channels */
#define LR_DIFF_FILL 0x2u /* lr_step_paged_diff: rows of unused slots are written as zeros */

typedef struct {
    unsigned flags;       /* OR of LR_DIFF_*                            */
    const float *lambda;  /* [H] fp32, 4-byte aligned                   */
    const float *weight;  /* [2 d] fp32 of the norm, or NULL for ones   */
    float eps;            /* >= 0, finite (LR_DIFF_NORM)                */
} lr_diff_maps;

/*
 *   q, qs  [B, 2 H, Tq, d] with strides    k, ks, v, vs  [B, 2 Hk, Tk, d]
 *   o, os  [B, 2 H, Tq, d] with strides, written; overlaps no input
 *   workspace  lr_fwd_diff_workspace_size(...) bytes, 16-byte aligned (0 in
 *              bf16); its contents on entry do not matter.  Calls that share
 *              one are ordered on one stream.
 * The other arguments are those of lr_fwd_window.  bf16: one kernel.
 */
lr_status lr_fwd_diff(const void *q, lr_strides qs, const void *k, lr_strides ks, const void *v,
                      lr_strides vs, const int *q_len, const int *k_len, const lr_diff_maps *maps,
                      void *o, lr_strides os, int B, int H, int Hk, int Tq, int Tk, int d,
                      int window, int sinks, float scale, lr_dtype dt, void *workspace,
                      size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes lr_fwd_diff needs (0 as well for arguments it would reject). */
size_t lr_fwd_diff_workspace_size(int B, int H, int Hk, int Tq, int Tk, int d, lr_dtype dt);

/*
 * One decode step: the row of position lens[n] - 1 of the attention above,
 * for N sequences whose keys and values (this token's included) are in the
 * paged cache.
 *
 *   q       [N, Hq, d], contiguous
 *   cache   pools and table [N, max_pages]
 *   lens    [N] int32, tokens in the cache.  0: the output row is zeros.
 *           Negative: an unused slot, its row is left as it was.
 *   o       [N, Hq, d], written; overlaps no input
 *   max_len bound on lens, 1 <= max_len <= page * max_pages: it sets how the
 *           work is split, so a tight bound is faster and needs less workspace
 *           (128 sequences of 500 to 8192 tokens, 32 heads on 8, bf16: 351 us
 *           and 16 MB under a bound of 8192, 369 us and 65 MB under 32768, 465
 *           us and 260 MB under 131072).  A longer sequence is reported as
 *           LR_ERR_INDEX and its row is left as it was.
 *   workspace   lr_step_paged_workspace_size(...) bytes, 16-byte aligned (0
 *           where the work is not split, or its parts are joined on the chip);
 *           its contents on entry do not matter.  Calls that share one are
 *           ordered on one stream.
 *
 * The keys a sequence sees are cut into chunks of equal size, which the CTAs
 * of a cluster or a second kernel join in a fixed order: a repeated call gives
 * the same bits.  Up to 16 query heads of a key head in bf16, and 4 in fp32,
 * share one read of its keys and values; more are worked on in parts that each
 * read them.
 */
lr_status lr_step_paged(const void *q, const lr_paged *cache, const int *lens, void *o, int N,
                        int Hq, int Hk, int d, int max_len, int window, int sinks, float scale,
                        lr_dtype dt, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* lr_step_paged for an output that held nothing before: the rows that it would
 * leave as they were (unused slots, lengths beyond max_len) are zeros. */
lr_status lr_step_paged_fill(const void *q, const lr_paged *cache, const int *lens, void *o, int N,
                             int Hq, int Hk, int d, int max_len, int window, int sinks, float scale,
                             lr_dtype dt, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream);

/* Workspace bytes lr_step_paged and lr_step_paged_fill need (0 as well for
 * arguments they would reject). */
size_t lr_step_paged_workspace_size(int N, int Hq, int Hk, int d, int max_len, int window,
                                    int sinks, lr_dtype dt);

#define LR_STEP_FILL 0x1u /* rows of unused slots are written as zeros */

/*
 * One decode step of lr_step_paged for N sequences that begin with the same
 * prefix_len tokens, held once in the pages of `prefix`; a sequence's own tokens
 * follow in its pages of the cache's table.  The row of sequence n stands at
 * position prefix_len + lens[n] - 1 of the whole sequence; window and sinks count
 * in it.  What it sees and returns is what lr_step_paged would for the pages of
 * prefix and own tokens one behind the other.
 *
 *   prefix      [ceil(prefix_len / page)] int32 page numbers on the device, in
 *               the cache's pools; NULL where prefix_len is 0.  Rows of its last
 *               page behind the prefix are not read into any sum.
 *   prefix_len  0 <= prefix_len, prefix_len + max_len <= 2^30
 *   lens        [N] int32 own tokens, this one included (0: the row is that of the
 *               prefix's last token, zeros where there is none; negative: an
 *               unused slot, its row is left as it was)
 *   max_len     bound on lens, as for lr_step_paged
 *   flags       OR of LR_STEP_*
 *   workspace   lr_step_paged_prefix_workspace_size(...) bytes, 16-byte aligned
 *
 * The other arguments are those of lr_step_paged.  The prefix is read once for up
 * to 256 rows of a key head in bf16 and 64 in fp32 (a row: a sequence and one of
 * the Hq / Hk query heads), by a kernel of its own; the own tokens' kernel joins
 * both.  A repeated call gives the same bits.
 */
lr_status lr_step_paged_prefix(const void *q, const lr_paged *cache, const int *prefix,
                               int prefix_len, const int *lens, void *o, int N, int Hq, int Hk,
                               int d, int max_len, int window, int sinks, float scale,
                               unsigned flags, lr_dtype dt, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes lr_step_paged_prefix needs (0 as well for arguments it would reject). */
size_t lr_step_paged_prefix_workspace_size(int N, int Hq, int Hk, int d, int prefix_len,
                                           int max_len, int window, int sinks, lr_dtype dt);

/*
 * One decode step of lr_fwd_diff, as lr_step_paged is one of lr_fwd_window.
 *
 *   q       [N, 2 H, d], contiguous
 *   cache   pools [num_pages, 2 Hk, page, d]: the keys of both maps, and the two
 *           halves of every value row, as lr_qk_norm_rope writes them from 2 Hk
 *           heads
 *   o       [N, 2 H, d], written; overlaps no input
 *   lens, max_len, window, sinks, scale as for lr_step_paged (with LR_DIFF_FILL
 *           the rows that it would leave as they were are zeros)
 *   workspace   lr_step_paged_diff_workspace_size(...) bytes, 16-byte aligned
 *
 * A repeated call gives the same bits.  Up to 8 pairs of query heads of a pair
 * of key heads in bf16, and 2 in fp32, share one read of the cache.
 */
lr_status lr_step_paged_diff(const void *q, const lr_paged *cache, const int *lens,
                             const lr_diff_maps *maps, void *o, int N, int H, int Hk, int d,
                             int max_len, int window, int sinks, float scale, lr_dtype dt,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes lr_step_paged_diff needs (0 as well for arguments it would reject). */
size_t lr_step_paged_diff_workspace_size(int N, int H, int Hk, int d, int max_len, int window,
                                         int sinks, lr_dtype dt);

#ifdef __cplusplus
}
#endif

#endif /* LR_ATTN_H_ */
