// Host side of include/lr_attn.h: validation before any launch, dispatch,
// status mapping.
#include <math.h>

#include "attn_internal.cuh"

using namespace lr;

namespace {

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi)
};
Span span(const void *p, size_t bytes) {
    Span s;
    if (p && bytes) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + bytes;
    }
    return s;
}
bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr long long kMostElements = 1ll << 40;

// a * b * c * d as elements one device can hold; all factors >= 0
bool count_ok(long long a, long long b, long long c, long long d) {
    long long x = 1;
    for (long long f : {a, b, c, d}) {
        if (f == 0) return true;
        if (x > kMostElements / f) return false;
        x *= f;
    }
    return true;
}

lr_status check_types(int d, lr_dtype dt) {
    if (dt != LR_DT_F32 && dt != LR_DT_BF16) return LR_ERR_DTYPE;
    if (d < 1) return LR_ERR_SHAPE;
    if (d != 32 && d != 64 && d != 128) return LR_ERR_UNSUPPORTED;
    return LR_OK;
}

size_t esize(lr_dtype dt) { return dt == LR_DT_F32 ? 4 : 2; }

// Strides of a [B, H, T, d] tensor: positive and whole 16-byte units where
// the size is above 1 (a size of 1 never uses its stride: it is replaced by 0).
lr_status check_strides(lr_strides *s, int B, int H, int T, lr_dtype dt) {
    const long long unit = 16 / (long long)esize(dt);
    long long *st[3] = {&s->b, &s->h, &s->t};
    const int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) {
            *st[i] = 0;
            continue;
        }
        if (*st[i] <= 0 || *st[i] > kMostElements / n[i]) return LR_ERR_SHAPE;
        if (*st[i] % unit) return LR_ERR_ALIGN;
    }
    return LR_OK;
}
Span strided_span(const void *p, const lr_strides &s, int B, int H, int T, int d, lr_dtype dt) {
    if (!B || !H || !T) return Span{};
    const size_t last = (size_t)s.b * (B - 1) + (size_t)s.h * (H - 1) + (size_t)s.t * (T - 1);
    return span(p, (last + d) * esize(dt));
}
// No two elements of a written tensor share an address: sorted by stride,
// each stride covers the extent of the smaller ones.
bool distinct_rows(const lr_strides &s, int B, int H, int T, int d) {
    long long st[3] = {s.b, s.h, s.t};
    int n[3] = {B, H, T};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (st[j] > st[j + 1]) {
                const long long x = st[j];
                st[j] = st[j + 1];
                st[j + 1] = x;
                const int y = n[j];
                n[j] = n[j + 1];
                n[j + 1] = y;
            }
    long long extent = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < extent) return false;
        extent = st[i] * (n[i] - 1) + extent;
    }
    return true;
}

// The cache's own fields; its pools as spans.
lr_status check_paged(const lr_paged *c, int B, int Hk, int d, lr_dtype dt, Span *k, Span *v,
                      Span *table) {
    if (c->num_pages < 1 || c->max_pages < 1) return LR_ERR_SHAPE;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
        return LR_ERR_UNSUPPORTED;
    if ((long long)c->page * c->max_pages > (1ll << 30)) return LR_ERR_SHAPE;
    if (!count_ok(c->num_pages, Hk, c->page, d) || !count_ok(B, c->max_pages, 1, 1))
        return LR_ERR_SHAPE;
    if (!c->k || !c->v || !c->table) return LR_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->table)) return LR_ERR_ALIGN;
    const size_t pool = (size_t)c->num_pages * Hk * c->page * d * esize(dt);
    *k = span(c->k, pool);
    *v = span(c->v, pool);
    *table = span(c->table, (size_t)B * c->max_pages * 4);
    return LR_OK;
}

lr_status check_heads(int Hq, int Hk) {
    if (Hq < 1 || Hk < 1 || Hq % Hk) return LR_ERR_SHAPE;
    return LR_OK;
}

int log2_of(int page) {
    int l = 0;
    while ((1 << l) < page) ++l;
    return l;
}

lr_status done(cudaError_t e) { return e == cudaSuccess ? LR_OK : LR_ERR_CUDA; }

// Sizes of a step; shared by the call and its workspace query.
lr_status check_step_sizes(int N, int Hq, int Hk, int d, int max_len, int window, int sinks,
                           lr_dtype dt) {
    const lr_status st = check_types(d, dt);
    if (st != LR_OK) return st;
    const lr_status hs = check_heads(Hq, Hk);
    if (hs != LR_OK) return hs;
    if (N < 1 || max_len < 1 || window < 1 || sinks < 0) return LR_ERR_SHAPE;
    if (max_len > (1 << 30) || !count_ok(N, Hq, d, 1)) return LR_ERR_SHAPE;
    // CTAs of one launch
    const StepPlan p = step_plan(N, Hq, Hk, d, max_len, window, sinks, dt);
    if (!count_ok(N, Hq, p.splits, 1) || (long long)N * Hq * p.splits > 0x7fffffffll)
        return LR_ERR_SHAPE;
    return LR_OK;
}

lr_status step_paged(const void *q, const lr_paged *cache, const int *lens, void *o, int N, int Hq,
                     int Hk, int d, int max_len, int window, int sinks, float scale, lr_dtype dt,
                     void *workspace, size_t workspace_bytes, bool fill, cudaStream_t stream) {
    lr_status st = check_step_sizes(N, Hq, Hk, d, max_len, window, sinks, dt);
    if (st != LR_OK) return st;
    if (!isfinite(scale)) return LR_ERR_SHAPE;
    if (!q || !cache || !lens || !o) return LR_ERR_NULL;
    Span ck, cv, ct;
    if ((st = check_paged(cache, N, Hk, d, dt, &ck, &cv, &ct)) != LR_OK) return st;
    if ((long long)max_len > (long long)cache->page * cache->max_pages) return LR_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(o) || !aligned4(lens)) return LR_ERR_ALIGN;
    const size_t need = lr_step_paged_workspace_size(N, Hq, Hk, d, max_len, window, sinks, dt);
    if (need > 0 && (!workspace || workspace_bytes < need)) return LR_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return LR_ERR_ALIGN;
    const size_t rows = (size_t)N * Hq * d * esize(dt);
    const Span so = span(o, rows), sq = span(q, rows), sl = span(lens, (size_t)N * 4);
    const Span sw = span(need > 0 ? workspace : nullptr, need);
    for (const Span &i : {sq, sl, ck, cv, ct, sw})
        if (overlap(so, i)) return LR_ERR_ALIAS;
    for (const Span &i : {sq, sl, ck, cv, ct})
        if (overlap(sw, i)) return LR_ERR_ALIAS;
    const StepArgs a{q, cache->k, cache->v, o, cache->table, lens, N, Hq, Hk, max_len, window,
                     sinks, cache->num_pages, log2_of(cache->page), cache->max_pages, scale, fill,
                     nullptr, 0, sinks, 0, nullptr, nullptr};
    return done(launch_step_paged(a, d, dt, workspace, stream));
}

// Sizes of differential attention; shared by the call and its workspace query.
lr_status check_diff_sizes(int B, int H, int Hk, int Tq, int Tk, int d, lr_dtype dt) {
    const lr_status st = check_types(d, dt);
    if (st != LR_OK) return st;
    if (check_heads(H, Hk) != LR_OK || B < 1 || Tq < 0 || Tk < 0 || H > (1 << 29)) return LR_ERR_SHAPE;
    if (Tq > (1 << 30) || Tk > (1 << 30) || !count_ok(B, 2ll * H, Tq, 2ll * d) ||
        !count_ok(B, 2ll * Hk, Tk, d))
        return LR_ERR_SHAPE;
    // row tiles of both maps over both halves of the values, counted as CTAs of one launch
    if (!count_ok(B, 4ll * H, Tq / 64 + 1, 1) || 4ll * B * H * (Tq / 64 + 1) > 0x7fffffffll)
        return LR_ERR_SHAPE;
    return LR_OK;
}
// fp32 keeps the maps' own outputs
size_t diff_workspace(int B, int H, int Tq, int Tk, int d, lr_dtype dt) {
    return dt == LR_DT_F32 && Tk > 0 ? diff_f32_workspace_bytes(B, H, Tq, d) : 0;
}

lr_status check_diff_maps(const lr_diff_maps *m, unsigned known, int H, int d, Span *lambda, Span *weight) {
    if (!m) return LR_ERR_NULL;
    if (m->flags & ~known) return LR_ERR_FUSE;
    const bool norm = m->flags & LR_DIFF_NORM;
    if (norm && !(m->eps >= 0.f && m->eps <= 3.4e38f)) return LR_ERR_FUSE;
    if (!m->lambda) return LR_ERR_NULL;
    if (!aligned4(m->lambda) || !aligned4(m->weight)) return LR_ERR_ALIGN;
    *lambda = span(m->lambda, (size_t)H * 4);
    *weight = span(norm ? m->weight : nullptr, (size_t)d * 8);
    return LR_OK;
}

// Sinks among a sequence's own tokens.
int own_sinks(int sinks, int prefix_len) { return sinks > prefix_len ? sinks - prefix_len : 0; }

lr_status check_prefix_sizes(int N, int Hq, int Hk, int d, int prefix_len, int max_len, int window, int sinks,
                             lr_dtype dt) {
    if (prefix_len < 0 || sinks < 0 || (long long)prefix_len + max_len > (1ll << 30)) return LR_ERR_SHAPE;
    const lr_status st = check_step_sizes(N, Hq, Hk, d, max_len, window, own_sinks(sinks, prefix_len), dt);
    if (st != LR_OK) return st;
    // rows as an int, CTAs of one launch and the parts' elements
    const PrefixPlan p = prefix_plan(N, Hq, Hk, d, prefix_len, window, sinks, dt);
    if ((long long)N * Hq > (1ll << 30) || !count_ok(N, Hq, p.parts, d) ||
        ((long long)N * (Hq / Hk) / 64 + 1) * Hk > 0x7fffffffll / (p.parts ? p.parts : 1))
        return LR_ERR_SHAPE;
    return LR_OK;
}

lr_status check_diff_step_sizes(int N, int H, int Hk, int d, int max_len, int window, int sinks, lr_dtype dt) {
    const lr_status st = check_types(d, dt);
    if (st != LR_OK) return st;
    if (check_heads(H, Hk) != LR_OK || N < 1 || max_len < 1 || window < 1 || sinks < 0) return LR_ERR_SHAPE;
    if (max_len > (1 << 30) || H > (1 << 29) || !count_ok(N, 2ll * H, 2ll * d, 1)) return LR_ERR_SHAPE;
    // CTAs of one launch
    const StepPlan p = diff_step_plan(N, H, Hk, d, max_len, window, sinks, dt);
    if (!count_ok(N, H, p.splits, 1) || (long long)N * H * p.splits > 0x7fffffffll) return LR_ERR_SHAPE;
    return LR_OK;
}

// axes.count 0: positions of one axis; else `positions` are the tokens' places.
lr_status qk_norm_rope(const void *q, lr_strides qs, const void *k, lr_strides ks,
                       const int *positions, const QkAxes &axes, const lr_qk_maps *maps, void *q_out,
                       void *k_out, const void *v, lr_strides vs, const lr_paged *cache, int B, int T,
                       int Hq, int Hk, int d, lr_dtype dt, cudaStream_t stream) {
    lr_status st = check_types(d, dt);
    if (st != LR_OK) return st;
    if (B < 1 || T < 0 || Hq < 1 || Hk < 1) return LR_ERR_SHAPE;
    // the kernel's head index runs up to 4 x 64 beyond the last head
    if (!count_ok(B, T, Hq > Hk ? Hq : Hk, d) || (long long)B * T > (1ll << 30) ||
        Hq > (1 << 30) || Hk > (1 << 30))
        return LR_ERR_SHAPE;
    if (!maps) return LR_ERR_NULL;
    if (maps->flags & ~(LR_QK_NORM | LR_QK_INTERLEAVED | LR_QK_ZERO_Q | LR_QK_ZERO_K))
        return LR_ERR_FUSE;
    const bool norm = maps->flags & LR_QK_NORM;
    if (norm && !(maps->eps >= 0.f && maps->eps <= 3.4e38f)) return LR_ERR_FUSE;
    if (maps->rot < 0 || maps->rot > d || maps->rot % 16) return LR_ERR_UNSUPPORTED;
    if (maps->rot && !maps->inv_freq) return LR_ERR_NULL;
    const bool turned = axes.count && maps->rot;  // by several axes
    if (turned && !axes.axis) return LR_ERR_NULL;
    Span ck, cv, ct;
    if (cache) {
        st = check_paged(cache, B, Hk, d, dt, &ck, &cv, &ct);
        if (st != LR_OK) return st;
    }
    if (T == 0) return LR_OK;
    if (!q || !k || !q_out || (!k_out && !cache) || (cache && !v)) return LR_ERR_NULL;
    if (turned && !axes.positions) return LR_ERR_NULL;
    if (!cache) v = nullptr;
    for (const void *p : {q, k, v, (const void *)q_out, (const void *)k_out,
                          (const void *)maps->inv_freq, (const void *)maps->q_weight,
                          (const void *)maps->k_weight})
        if (!aligned16(p)) return LR_ERR_ALIGN;
    if (!aligned4(positions)) return LR_ERR_ALIGN;
    if (turned && (!aligned4(axes.positions) || !aligned4(axes.axis))) return LR_ERR_ALIGN;
    if ((st = check_strides(&qs, B, Hq, T, dt)) != LR_OK) return st;
    if ((st = check_strides(&ks, B, Hk, T, dt)) != LR_OK) return st;
    if (cache && (st = check_strides(&vs, B, Hk, T, dt)) != LR_OK) return st;

    const size_t es = esize(dt), rows = (size_t)B * T;
    const Span in[] = {strided_span(q, qs, B, Hq, T, d, dt),
                       strided_span(k, ks, B, Hk, T, d, dt),
                       cache ? strided_span(v, vs, B, Hk, T, d, dt) : Span{},
                       span(positions, rows * 4),
                       span(maps->rot ? maps->inv_freq : nullptr, (size_t)maps->rot / 2 * 8),
                       span(norm ? maps->q_weight : nullptr, (size_t)d * 4),
                       span(norm ? maps->k_weight : nullptr, (size_t)d * 4),
                       span(turned ? axes.positions : nullptr, (size_t)axes.count * rows * 4),
                       span(turned ? axes.axis : nullptr, (size_t)maps->rot / 2 * 4),
                       ct};
    const Span out[] = {span(q_out, rows * Hq * d * es), span(k_out, rows * Hk * d * es), ck, cv};
    for (int a = 0; a < 4; ++a) {
        for (const Span &i : in)
            if (overlap(out[a], i)) return LR_ERR_ALIAS;
        for (int b = 0; b < a; ++b)
            if (overlap(out[a], out[b])) return LR_ERR_ALIAS;
    }
    QkMaps m;
    m.qw = norm ? maps->q_weight : nullptr;
    m.kw = norm ? maps->k_weight : nullptr;
    m.inv_freq = maps->inv_freq;
    m.eps = maps->eps;
    m.rot = maps->rot;
    m.flags = maps->flags;
    return done(launch_qk_norm_rope(q, qs, k, ks, positions, axes, m, q_out, k_out, v, vs, cache, B, T,
                                    Hq, Hk, d, dt, stream));
}

}  // namespace

extern "C" {

lr_status lr_qk_norm_rope(const void *q, lr_strides qs, const void *k, lr_strides ks,
                          const int *positions, const lr_qk_maps *maps, void *q_out, void *k_out,
                          const void *v, lr_strides vs, const lr_paged *cache, int B, int T,
                          int Hq, int Hk, int d, lr_dtype dt, cudaStream_t stream) {
    return qk_norm_rope(q, qs, k, ks, positions, QkAxes{nullptr, nullptr, 0}, maps, q_out, k_out, v, vs,
                        cache, B, T, Hq, Hk, d, dt, stream);
}

lr_status lr_qk_norm_rope_axes(const void *q, lr_strides qs, const void *k, lr_strides ks,
                               const int *positions, const int *axis, int axes, const int *places,
                               const lr_qk_maps *maps, void *q_out, void *k_out, const void *v,
                               lr_strides vs, const lr_paged *cache, int B, int T, int Hq, int Hk,
                               int d, lr_dtype dt, cudaStream_t stream) {
    if (axes < 1 || axes > LR_MAX_AXES) return LR_ERR_SHAPE;
    return qk_norm_rope(q, qs, k, ks, places, QkAxes{positions, axis, axes}, maps, q_out, k_out, v, vs,
                        cache, B, T, Hq, Hk, d, dt, stream);
}

lr_status lr_fwd_window(const void *q, lr_strides qs, const void *k, lr_strides ks, const void *v,
                        lr_strides vs, const int *q_len, const int *k_len, void *o, lr_strides os,
                        int B, int Hq, int Hk, int Tq, int Tk, int d, int window, int sinks,
                        float scale, lr_dtype dt, cudaStream_t stream) {
    lr_status st = check_types(d, dt);
    if (st != LR_OK) return st;
    if ((st = check_heads(Hq, Hk)) != LR_OK) return st;
    if (B < 1 || Tq < 0 || Tk < 0 || window < 1 || sinks < 0 || !isfinite(scale))
        return LR_ERR_SHAPE;
    if (Tq > (1 << 30) || Tk > (1 << 30) || !count_ok(B, Hq, Tq, d) || !count_ok(B, Hk, Tk, d))
        return LR_ERR_SHAPE;
    // row tiles, counted as CTAs of one launch
    if (!count_ok(B, Hq, Tq / 64 + 1, 1) || (long long)B * Hq * (Tq / 64 + 1) > 0x7fffffffll)
        return LR_ERR_SHAPE;
    if (Tq == 0) return LR_OK;
    if (!q || !o || (Tk > 0 && (!k || !v))) return LR_ERR_NULL;
    for (const void *p : {q, k, v, (const void *)o})
        if (!aligned16(p)) return LR_ERR_ALIGN;
    if (!aligned4(q_len) || !aligned4(k_len)) return LR_ERR_ALIGN;
    if ((st = check_strides(&qs, B, Hq, Tq, dt)) != LR_OK) return st;
    if ((st = check_strides(&os, B, Hq, Tq, dt)) != LR_OK) return st;
    if ((st = check_strides(&ks, B, Hk, Tk, dt)) != LR_OK) return st;
    if ((st = check_strides(&vs, B, Hk, Tk, dt)) != LR_OK) return st;
    if (!distinct_rows(os, B, Hq, Tq, d)) return LR_ERR_ALIAS;
    const Span so = strided_span(o, os, B, Hq, Tq, d, dt);
    for (const Span &i :
         {strided_span(q, qs, B, Hq, Tq, d, dt), strided_span(k, ks, B, Hk, Tk, d, dt),
          strided_span(v, vs, B, Hk, Tk, d, dt), span(q_len, (size_t)B * 4),
          span(k_len, (size_t)B * 4)})
        if (overlap(so, i)) return LR_ERR_ALIAS;
    const WindowArgs a{q, k, v, o, qs, ks, vs, os, q_len, k_len, B, Hq, Hk, Tq, Tk, window, sinks,
                       scale, 0};
    if (Tk == 0) return done(launch_window_zero(a, d, dt, stream));
    return done(dt == LR_DT_BF16 ? launch_window_tc(a, d, stream)
                                 : launch_window_f32(a, d, stream));
}

lr_status lr_fwd_diff(const void *q, lr_strides qs, const void *k, lr_strides ks, const void *v,
                      lr_strides vs, const int *q_len, const int *k_len, const lr_diff_maps *maps,
                      void *o, lr_strides os, int B, int H, int Hk, int Tq, int Tk, int d,
                      int window, int sinks, float scale, lr_dtype dt, void *workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
    lr_status st = check_diff_sizes(B, H, Hk, Tq, Tk, d, dt);
    if (st != LR_OK) return st;
    if (window < 1 || sinks < 0 || !isfinite(scale)) return LR_ERR_SHAPE;
    Span lambda, weight;
    if ((st = check_diff_maps(maps, LR_DIFF_NORM, H, d, &lambda, &weight)) != LR_OK) return st;
    if (Tq == 0) return LR_OK;
    if (!q || !o || (Tk > 0 && (!k || !v))) return LR_ERR_NULL;
    for (const void *p : {q, k, v, (const void *)o})
        if (!aligned16(p)) return LR_ERR_ALIGN;
    if (!aligned4(q_len) || !aligned4(k_len)) return LR_ERR_ALIGN;
    if ((st = check_strides(&qs, B, 2 * H, Tq, dt)) != LR_OK) return st;
    if ((st = check_strides(&os, B, 2 * H, Tq, dt)) != LR_OK) return st;
    if ((st = check_strides(&ks, B, 2 * Hk, Tk, dt)) != LR_OK) return st;
    if ((st = check_strides(&vs, B, 2 * Hk, Tk, dt)) != LR_OK) return st;
    if (!distinct_rows(os, B, 2 * H, Tq, d)) return LR_ERR_ALIAS;
    const size_t need = diff_workspace(B, H, Tq, Tk, d, dt);
    if (need > 0 && (!workspace || workspace_bytes < need)) return LR_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return LR_ERR_ALIGN;
    const Span so = strided_span(o, os, B, 2 * H, Tq, d, dt), sw = span(need > 0 ? workspace : nullptr, need);
    for (const Span &i :
         {strided_span(q, qs, B, 2 * H, Tq, d, dt), strided_span(k, ks, B, 2 * Hk, Tk, d, dt),
          strided_span(v, vs, B, 2 * Hk, Tk, d, dt), span(q_len, (size_t)B * 4),
          span(k_len, (size_t)B * 4), lambda, weight})
        if (overlap(so, i) || overlap(sw, i)) return LR_ERR_ALIAS;
    if (overlap(so, sw)) return LR_ERR_ALIAS;
    if (Tk == 0) {
        const WindowArgs w{q, k, v, o, qs, ks, vs, os, q_len, k_len, B, 2 * H, 2 * Hk, Tq, Tk, window,
                           sinks, scale, 0};
        return done(launch_window_zero(w, d, dt, stream));
    }
    const DiffArgs a{q, k, v, o, qs, ks, vs, os, q_len, k_len, maps->lambda, maps->weight, B, H, Hk,
                     Tq, Tk, window, sinks, scale, maps->eps, (maps->flags & LR_DIFF_NORM) != 0};
    return done(dt == LR_DT_BF16 ? launch_diff_tc(a, d, stream) : launch_diff_f32(a, d, workspace, stream));
}

size_t lr_fwd_diff_workspace_size(int B, int H, int Hk, int Tq, int Tk, int d, lr_dtype dt) {
    if (check_diff_sizes(B, H, Hk, Tq, Tk, d, dt) != LR_OK) return 0;
    return diff_workspace(B, H, Tq, Tk, d, dt);
}

size_t lr_step_paged_workspace_size(int N, int Hq, int Hk, int d, int max_len, int window,
                                    int sinks, lr_dtype dt) {
    if (check_step_sizes(N, Hq, Hk, d, max_len, window, sinks, dt) != LR_OK) return 0;
    return step_workspace_bytes(N, Hq, d, step_plan(N, Hq, Hk, d, max_len, window, sinks, dt));
}

lr_status lr_step_paged(const void *q, const lr_paged *cache, const int *lens, void *o, int N,
                        int Hq, int Hk, int d, int max_len, int window, int sinks, float scale,
                        lr_dtype dt, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return step_paged(q, cache, lens, o, N, Hq, Hk, d, max_len, window, sinks, scale, dt, workspace,
                      workspace_bytes, false, stream);
}

lr_status lr_step_paged_fill(const void *q, const lr_paged *cache, const int *lens, void *o, int N,
                             int Hq, int Hk, int d, int max_len, int window, int sinks, float scale,
                             lr_dtype dt, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
    return step_paged(q, cache, lens, o, N, Hq, Hk, d, max_len, window, sinks, scale, dt, workspace,
                      workspace_bytes, true, stream);
}

lr_status lr_step_paged_diff(const void *q, const lr_paged *cache, const int *lens,
                             const lr_diff_maps *maps, void *o, int N, int H, int Hk, int d,
                             int max_len, int window, int sinks, float scale, lr_dtype dt,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    lr_status st = check_diff_step_sizes(N, H, Hk, d, max_len, window, sinks, dt);
    if (st != LR_OK) return st;
    if (!isfinite(scale)) return LR_ERR_SHAPE;
    Span lambda, weight;
    if ((st = check_diff_maps(maps, LR_DIFF_NORM | LR_DIFF_FILL, H, d, &lambda, &weight)) != LR_OK) return st;
    if (!q || !cache || !lens || !o) return LR_ERR_NULL;
    Span ck, cv, ct;
    if ((st = check_paged(cache, N, 2 * Hk, d, dt, &ck, &cv, &ct)) != LR_OK) return st;
    if ((long long)max_len > (long long)cache->page * cache->max_pages) return LR_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(o) || !aligned4(lens)) return LR_ERR_ALIGN;
    const size_t need = lr_step_paged_diff_workspace_size(N, H, Hk, d, max_len, window, sinks, dt);
    if (need > 0 && (!workspace || workspace_bytes < need)) return LR_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return LR_ERR_ALIGN;
    const size_t rows = (size_t)N * 2 * H * d * esize(dt);
    const Span so = span(o, rows), sq = span(q, rows), sl = span(lens, (size_t)N * 4);
    const Span sw = span(need > 0 ? workspace : nullptr, need);
    for (const Span &i : {sq, sl, ck, cv, ct, lambda, weight})
        if (overlap(so, i) || overlap(sw, i)) return LR_ERR_ALIAS;
    if (overlap(so, sw)) return LR_ERR_ALIAS;
    const StepArgs a{q, cache->k, cache->v, o, cache->table, lens, N, H, Hk, max_len, window, sinks,
                     cache->num_pages, log2_of(cache->page), cache->max_pages, scale,
                     (maps->flags & LR_DIFF_FILL) != 0, nullptr, 0, sinks, 0, nullptr, nullptr};
    return done(launch_step_diff(a, maps->lambda, maps->weight, maps->eps, (maps->flags & LR_DIFF_NORM) != 0, d, dt,
                                 workspace, stream));
}

size_t lr_step_paged_diff_workspace_size(int N, int H, int Hk, int d, int max_len, int window,
                                         int sinks, lr_dtype dt) {
    if (check_diff_step_sizes(N, H, Hk, d, max_len, window, sinks, dt) != LR_OK) return 0;
    return diff_step_workspace_bytes(N, H, d, diff_step_plan(N, H, Hk, d, max_len, window, sinks, dt));
}

lr_status lr_step_paged_prefix(const void *q, const lr_paged *cache, const int *prefix,
                               int prefix_len, const int *lens, void *o, int N, int Hq, int Hk,
                               int d, int max_len, int window, int sinks, float scale,
                               unsigned flags, lr_dtype dt, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    lr_status st = check_prefix_sizes(N, Hq, Hk, d, prefix_len, max_len, window, sinks, dt);
    if (st != LR_OK) return st;
    if (!isfinite(scale)) return LR_ERR_SHAPE;
    if (flags & ~LR_STEP_FILL) return LR_ERR_FUSE;
    if (!q || !cache || !lens || !o || (prefix_len > 0 && !prefix)) return LR_ERR_NULL;
    Span ck, cv, ct;
    if ((st = check_paged(cache, N, Hk, d, dt, &ck, &cv, &ct)) != LR_OK) return st;
    if ((long long)max_len > (long long)cache->page * cache->max_pages) return LR_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(o) || !aligned4(lens) || !aligned4(prefix)) return LR_ERR_ALIGN;
    const size_t need =
        lr_step_paged_prefix_workspace_size(N, Hq, Hk, d, prefix_len, max_len, window, sinks, dt);
    if (need > 0 && (!workspace || workspace_bytes < need)) return LR_ERR_WORKSPACE;
    if (need > 0 && !aligned16(workspace)) return LR_ERR_ALIGN;
    const size_t rows = (size_t)N * Hq * d * esize(dt), pages = ((size_t)prefix_len + cache->page - 1) / cache->page;
    const Span so = span(o, rows), sq = span(q, rows), sl = span(lens, (size_t)N * 4);
    const Span sp = span(prefix, pages * 4), sw = span(need > 0 ? workspace : nullptr, need);
    for (const Span &i : {sq, sl, ck, cv, ct, sp})
        if (overlap(so, i) || overlap(sw, i)) return LR_ERR_ALIAS;
    if (overlap(so, sw)) return LR_ERR_ALIAS;
    const StepArgs a{q, cache->k, cache->v, o, cache->table, lens, N, Hq, Hk, max_len, window,
                     own_sinks(sinks, prefix_len), cache->num_pages, log2_of(cache->page), cache->max_pages, scale,
                     (flags & LR_STEP_FILL) != 0, prefix, prefix_len, sinks, 0, nullptr, nullptr};
    return done(launch_step_prefix(a, d, dt, workspace, stream));
}

size_t lr_step_paged_prefix_workspace_size(int N, int Hq, int Hk, int d, int prefix_len,
                                           int max_len, int window, int sinks, lr_dtype dt) {
    if (check_prefix_sizes(N, Hq, Hk, d, prefix_len, max_len, window, sinks, dt) != LR_OK) return 0;
    return prefix_workspace_bytes(N, Hq, d, prefix_plan(N, Hq, Hk, d, prefix_len, window, sinks, dt)) +
           step_workspace_bytes(N, Hq, d,
                                step_plan(N, Hq, Hk, d, max_len, window, own_sinks(sinks, prefix_len), dt));
}

}  // extern "C"
