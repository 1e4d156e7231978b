// attn_abi.hip -- the extern "C" boundary of the paged-attention entry points:
// host-side validation, then the launches on the caller's stream.  Nothing here
// allocates, synchronises or reads device memory.  Contracts: include/gdn.h.

#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "gdn.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

gdn_status from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

// log2 of a page size that the kernels take, or -1
int page_shift(int32_t size)
{
    for (int s = 4; s <= 8; ++s)
        if (size == 1 << s)
            return s;
    return -1;
}

gdn_status check_dims(const gdn_attn_dims &d)
{
    if (d.B < 0 || d.T < 0 || d.R < 1 || d.H_q < 1 || d.H_kv < 1 || d.H_q % d.H_kv != 0 || d.N < 1 ||
        d.table_width < 1 || d.max_new < 0 || d.window < 0)
        return GDN_ERR_SHAPE;
    if ((d.d != 64 && d.d != 128 && d.d != 256) || page_shift(d.page_size) < 0 || d.cache_type < 0 ||
        d.cache_type > 1)
        return GDN_ERR_UNSUPPORTED;
    // positions, grids and row counts in 32 bits
    if ((int64_t)d.table_width * d.page_size > INT32_MAX / 2 || (int64_t)d.T * d.H_q > INT32_MAX / 2 ||
        (int64_t)d.H_q + 2 * (int64_t)d.H_kv > 65535 ||
        ((int64_t)d.T * (d.H_q / d.H_kv) / 256 + d.B) * d.H_kv > INT32_MAX / 4)
        return GDN_ERR_SHAPE;
    return GDN_OK;
}

gdn_status check_heads(const gdn_heads &h)
{
    if (h.row_stride < 0 || h.head_stride < 0)
        return GDN_ERR_SHAPE;
    return !aligned(h.data, 16) || h.row_stride % 8 != 0 || h.head_stride % 8 != 0 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn::Heads heads_of(const gdn_heads &h) { return gdn::Heads{h.data, h.row_stride, h.head_stride}; }

gdn_status check_cache(const gdn_kv_cache &c, bool e4m3)
{
    if (!c.k || !c.v || (e4m3 && (!c.k_scale || !c.v_scale)))
        return GDN_ERR_NULL;
    return !aligned(c.k, 16) || !aligned(c.v, 16) ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

constexpr int32_t kMostGroups = 1024; // of a call: a planning workgroup's threads

// What the attention calls share; on GDN_OK with *run set p holds all but the workspace (*run is false when there
// is nothing to do).
gdn_status attn_setup(const gdn_attn_dims *dims, const gdn_heads *q, const gdn_kv_cache *cache, const int32_t *row,
                      const int32_t *cu_seqlens, const gdn_heads *out, float *lse, float scale, void *workspace,
                      gdn::AttnParams &p, bool *run)
{
    *run = false;
    if (!dims)
        return GDN_ERR_NULL;
    const gdn_attn_dims d = *dims;
    if (d.B == 0 || d.T == 0)
        return GDN_OK;
    if (!q || !q->data || !out || !out->data || !cache || !cache->page_table || !cache->kv_len || !row ||
        !cu_seqlens || !workspace)
        return GDN_ERR_NULL;
    gdn_status st = check_dims(d);
    if (st != GDN_OK)
        return st;
    if ((st = check_cache(*cache, d.cache_type == 1)) != GDN_OK || (st = check_heads(*q)) != GDN_OK ||
        (st = check_heads(*out)) != GDN_OK)
        return st;
    if (!aligned(workspace, 256) || !aligned(lse, 4))
        return GDN_ERR_UNSUPPORTED;
    if (!isfinite(scale))
        return GDN_ERR_SHAPE;
    p.q = heads_of(*q);
    p.out = heads_of(*out);
    p.lse = lse;
    p.k_pages = cache->k;
    p.v_pages = cache->v;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.page_table = cache->page_table;
    p.kv_len = cache->kv_len;
    p.row = row;
    p.cu = cu_seqlens;
    p.scale = scale * 1.44269504088896340736f;
    p.B = d.B;
    p.T = d.T;
    p.R = d.R;
    p.H_q = d.H_q;
    p.H_kv = d.H_kv;
    p.G = d.H_q / d.H_kv;
    p.N = d.N;
    p.page_shift = page_shift(d.page_size);
    p.width = d.table_width;
    p.max_new = d.max_new;
    // no position lies further back than the table reaches; the kernels add to a window in 32 bits
    p.window = d.window < (int64_t)d.table_width * d.page_size ? d.window : 0;
    *run = true;
    return GDN_OK;
}

} // namespace

extern "C" {

gdn_status gdn_rope_freqs(int32_t rot, double base, int32_t stretch, double factor, double original, double low,
                          double high, double *out)
{
    if (!out)
        return GDN_ERR_NULL;
    if (rot < 0 || rot % 2 != 0 || !(base > 0) || !isfinite(base) || stretch < 0 || stretch > 3)
        return GDN_ERR_SHAPE;
    if (stretch != 0 && (!(factor > 0) || !isfinite(factor)))
        return GDN_ERR_SHAPE;
    if ((stretch == 2 && rot <= 2) || (stretch == 3 && (!(original > 0) || !isfinite(original) || !(high > low))))
        return GDN_ERR_SHAPE;
    const double from = stretch == 2 ? base * pow(factor, (double)rot / (rot - 2)) : base;
    for (int j = 0; j < rot / 2; ++j) {
        double f = pow(from, -2.0 * j / rot);
        if (stretch == 1) {
            f /= factor;
        } else if (stretch == 3) {
            const double r = original * f / 6.283185307179586477;
            const double g = r >= high ? 1.0 : (r <= low ? 0.0 : (r - low) / (high - low));
            f = g * f + (1.0 - g) * f / factor;
        }
        out[j] = f;
    }
    return GDN_OK;
}

gdn_status attn_prologue(const gdn_attn_dims *dims, const gdn_heads *q, const gdn_heads *k, const gdn_heads *v,
                         const gdn_heads *q_out, const gdn_kv_cache *cache, const int32_t *row,
                         const int32_t *cu_seqlens, const int32_t *positions, const gdn_rope *rope,
                         const gdn_qk_norm *norm, hipStream_t stream)
{
    if (!dims)
        return GDN_ERR_NULL;
    const gdn_attn_dims d = *dims;
    if (d.B == 0 || d.T == 0)
        return GDN_OK;
    const bool has_q = q && q->data, has_kv = k && k->data;
    if (!row || !cu_seqlens || !cache || !cache->kv_len || has_q != (q_out && q_out->data) ||
        has_kv != (v && v->data) || (!has_q && !has_kv) || (rope && rope->rot > 0 && !rope->freqs) ||
        (has_kv && !cache->page_table))
        return GDN_ERR_NULL;
    gdn_status st = check_dims(d);
    if (st != GDN_OK)
        return st;
    // a workgroup of 256 threads a token: a launch counts its threads in 32 bits
    if (d.T > (1 << 24) - 1)
        return GDN_ERR_SHAPE;
    if (has_kv && (st = check_cache(*cache, d.cache_type == 1)) != GDN_OK)
        return st;
    for (const gdn_heads *h : {q, q_out, k, v})
        if (h && h->data && (st = check_heads(*h)) != GDN_OK)
            return st;
    gdn::AttnPrologueParams p{};
    if (rope) {
        if (rope->rot < 0 || rope->rot > d.d || rope->rot % 2 != 0 || !isfinite(rope->scale))
            return GDN_ERR_SHAPE;
        if (!aligned(rope->freqs, 8))
            return GDN_ERR_UNSUPPORTED;
        p.freqs = rope->freqs;
        p.rot = rope->rot;
        p.interleaved = rope->interleaved != 0;
        p.rope_scale = rope->scale;
    }
    if (norm) {
        if (!(norm->eps >= 0.0f) || !isfinite(norm->eps) || !isfinite(norm->add))
            return GDN_ERR_SHAPE;
        if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16))
            return GDN_ERR_UNSUPPORTED;
        p.q_w = norm->q_weight;
        p.k_w = norm->k_weight;
        p.eps = norm->eps;
        p.add = norm->add;
    }
    if (has_q) {
        p.q = heads_of(*q);
        p.q_out = heads_of(*q_out);
    }
    if (has_kv) {
        p.k = heads_of(*k);
        p.v = heads_of(*v);
        p.k_pages = cache->k;
        p.v_pages = cache->v;
        p.k_scale = cache->k_scale;
        p.v_scale = cache->v_scale;
        p.page_table = cache->page_table;
    }
    p.kv_len = cache->kv_len;
    p.row = row;
    p.cu = cu_seqlens;
    p.positions = positions;
    p.B = d.B;
    p.T = d.T;
    p.R = d.R;
    p.H_q = d.H_q;
    p.H_kv = d.H_kv;
    p.N = d.N;
    p.page_shift = page_shift(d.page_size);
    p.width = d.table_width;
    return from_hip(gdn::launch_attn_prologue(p, d.d, d.cache_type == 1, stream));
}

size_t attn_paged_workspace_bytes(const gdn_attn_dims *dims)
{
    if (!dims)
        return 0;
    const gdn_attn_dims d = *dims;
    if (d.B < 0 || d.T < 0 || d.max_new < 0 || d.H_q < 1 || d.H_kv < 1 || d.H_q % d.H_kv != 0 ||
        (d.d != 64 && d.d != 128 && d.d != 256))
        return 0;
    return gdn::attn_paged_layout(d.B, d.T, d.max_new, d.H_kv, d.H_q / d.H_kv, d.d, nullptr, nullptr);
}

gdn_status attn_paged(const gdn_attn_dims *dims, const gdn_heads *q, const gdn_kv_cache *cache, const int32_t *row,
                      const int32_t *cu_seqlens, const gdn_heads *out, float *lse, float scale, void *workspace,
                      size_t workspace_bytes, hipStream_t stream)
{
    gdn::AttnParams p{};
    bool run;
    const gdn_status st = attn_setup(dims, q, cache, row, cu_seqlens, out, lse, scale, workspace, p, &run);
    if (st != GDN_OK || !run)
        return st;
    if (workspace_bytes < gdn::attn_paged_layout(p.B, p.T, p.max_new, p.H_kv, p.G, dims->d, workspace, &p))
        return GDN_ERR_SHAPE;
    return from_hip(gdn::launch_attn_paged(p, dims->d, dims->cache_type == 1, stream));
}

size_t attn_shared_workspace_bytes(const gdn_attn_dims *dims, int32_t groups)
{
    if (!dims || groups < 0 || groups > kMostGroups)
        return 0;
    const gdn_attn_dims d = *dims;
    if (d.B < 0 || d.T < 0 || d.max_new < 0 || d.H_q < 1 || d.H_kv < 1 || d.H_q % d.H_kv != 0 ||
        (d.d != 64 && d.d != 128 && d.d != 256))
        return 0;
    return gdn::attn_shared_layout(d.B, d.T, groups, d.max_new, d.H_kv, d.H_q / d.H_kv, d.d, nullptr, nullptr);
}

gdn_status attn_shared(const gdn_attn_dims *dims, const gdn_heads *q, const gdn_kv_cache *cache, const int32_t *row,
                       const int32_t *cu_seqlens, const int32_t *cu_groups, const int32_t *shared_len, int32_t groups,
                       int32_t least, const gdn_heads *out, float *lse, float scale, void *workspace,
                       size_t workspace_bytes, hipStream_t stream)
{
    gdn::AttnParams p{};
    bool run;
    const gdn_status st = attn_setup(dims, q, cache, row, cu_seqlens, out, lse, scale, workspace, p, &run);
    if (st != GDN_OK || !run)
        return st;
    if (groups < 0 || groups > kMostGroups)
        return GDN_ERR_SHAPE;
    if (groups > 0 && (!cu_groups || !shared_len))
        return GDN_ERR_NULL;
    // the join's grid: an entry is 256 threads of 2^32
    if (((int64_t)p.T * p.G / 128 + (p.B > groups ? p.B : groups)) * p.H_kv >= 1 << 24 ||
        workspace_bytes < gdn::attn_shared_layout(p.B, p.T, groups, p.max_new, p.H_kv, p.G, dims->d, workspace, &p))
        return GDN_ERR_SHAPE;
    p.cu_groups = groups > 0 ? cu_groups : nullptr;
    p.shared_len = shared_len;
    p.K = groups;
    p.least = least < 0 ? -1 : least;
    return from_hip(gdn::launch_attn_shared(p, dims->d, dims->cache_type == 1, stream));
}

size_t kv_page_workspace_bytes(int32_t n, int32_t R, int32_t N)
{
    if (n < 0 || R < 0 || N < 0)
        return 0;
    return ((size_t)R + 4 * (size_t)n + 2 * (size_t)N + 4) * sizeof(int32_t);
}

} // extern "C"

namespace {

// What the bookkeeping calls share: sizes and arrays of the table.
gdn_status table_setup(const gdn_pages *pages, gdn::PageParams &p, bool lengths)
{
    const gdn_pages g = *pages;
    if (!g.page_table || !g.refs || (lengths && !g.kv_len))
        return GDN_ERR_NULL;
    if (g.R < 1 || g.table_width < 1 || g.N < 1 || g.N > 1 << 20)
        return GDN_ERR_SHAPE;
    p.table = g.page_table;
    p.kv_len = g.kv_len;
    p.refs = g.refs;
    p.R = g.R;
    p.width = g.table_width;
    p.N = g.N;
    if (lengths) {
        p.page_shift = page_shift(g.page_size);
        if (p.page_shift < 0)
            return GDN_ERR_UNSUPPORTED;
        if ((int64_t)g.table_width * g.page_size > INT32_MAX / 2)
            return GDN_ERR_SHAPE;
    }
    return GDN_OK;
}

// The arrays of the calls that move pages.
gdn_status move_setup(const gdn_pages *pages, gdn::PageParams &p)
{
    const gdn_pages g = *pages;
    if (!g.k || !g.v)
        return GDN_ERR_NULL;
    if (g.N < 1 || g.layers < 1 || g.page_bytes < 1 || g.layer_stride < 0 ||
        (g.layers > 1 && g.layer_stride / g.N < g.page_bytes))
        return GDN_ERR_SHAPE;
    if (!aligned(g.k, 16) || !aligned(g.v, 16) || g.page_bytes % 16 != 0 || g.layer_stride % 16 != 0)
        return GDN_ERR_UNSUPPORTED;
    p.k = static_cast<uint8_t *>(g.k);
    p.v = static_cast<uint8_t *>(g.v);
    p.layers = g.layers;
    p.layer_stride = g.layer_stride;
    p.page_bytes = g.page_bytes;
    p.N = g.N;
    return GDN_OK;
}

gdn_status scratch_setup(gdn::PageParams &p, int32_t n, int32_t *result, void *workspace, size_t bytes)
{
    if (!result || !workspace)
        return GDN_ERR_NULL;
    if (!aligned(workspace, 256))
        return GDN_ERR_UNSUPPORTED;
    if (bytes < kv_page_workspace_bytes(n, p.R, p.N))
        return GDN_ERR_SHAPE;
    p.result = result;
    p.owner = static_cast<int32_t *>(workspace);
    p.plan = p.owner + p.R;
    return GDN_OK;
}

} // namespace

extern "C" {

gdn_status kv_page_reserve(const gdn_pages *pages, const int32_t *rows, const int32_t *add, int32_t n,
                           int32_t *result, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!pages)
        return GDN_ERR_NULL;
    if (n < 0 || n > 65535)
        return GDN_ERR_SHAPE;
    if (n > 0 && (!rows || !add))
        return GDN_ERR_NULL;
    gdn::PageParams p{};
    gdn_status st = table_setup(pages, p, true);
    if (st != GDN_OK || (st = scratch_setup(p, n, result, workspace, workspace_bytes)) != GDN_OK)
        return st;
    p.a = rows;
    p.b = add;
    p.n = n;
    return from_hip(gdn::launch_kv_reserve(p, stream));
}

gdn_status kv_page_fork(const gdn_pages *pages, const int32_t *src, const int32_t *dst, int32_t n, int32_t *result,
                        void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!pages)
        return GDN_ERR_NULL;
    if (n < 0 || n > 65535)
        return GDN_ERR_SHAPE;
    if (n > 0 && (!src || !dst))
        return GDN_ERR_NULL;
    gdn::PageParams p{};
    gdn_status st = table_setup(pages, p, true);
    if (st != GDN_OK || (st = move_setup(pages, p)) != GDN_OK ||
        (st = scratch_setup(p, n, result, workspace, workspace_bytes)) != GDN_OK)
        return st;
    p.a = src;
    p.b = dst;
    p.n = n;
    return from_hip(gdn::launch_kv_fork(p, stream));
}

gdn_status kv_page_free(const gdn_pages *pages, const int32_t *rows, int32_t n, hipStream_t stream)
{
    if (!pages)
        return GDN_ERR_NULL;
    if (n < 0 || n > 65535)
        return GDN_ERR_SHAPE;
    if (n > 0 && !rows)
        return GDN_ERR_NULL;
    gdn::PageParams p{};
    const gdn_status st = table_setup(pages, p, true);
    if (st != GDN_OK || n == 0)
        return st;
    p.a = rows;
    p.n = n;
    return from_hip(gdn::launch_kv_free(p, stream));
}

gdn_status kv_page_copy(const gdn_pages *pages, const int32_t *src, const int32_t *dst, int32_t n, hipStream_t stream)
{
    if (!pages)
        return GDN_ERR_NULL;
    if (n < 0)
        return GDN_ERR_SHAPE;
    if (n > 0 && (!src || !dst))
        return GDN_ERR_NULL;
    gdn::PageParams p{};
    const gdn_status st = move_setup(pages, p);
    if (st != GDN_OK || n == 0)
        return st;
    p.a = src;
    p.b = dst;
    p.n = n;
    return from_hip(gdn::launch_kv_copy(p, stream));
}

gdn_status kv_page_compact(const gdn_pages *pages, int32_t *remap, int32_t *result, void *workspace,
                           size_t workspace_bytes, hipStream_t stream)
{
    if (!pages || !remap)
        return GDN_ERR_NULL;
    gdn::PageParams p{};
    gdn_status st = table_setup(pages, p, false);
    if (st != GDN_OK || (st = move_setup(pages, p)) != GDN_OK ||
        (st = scratch_setup(p, 0, result, workspace, workspace_bytes)) != GDN_OK)
        return st;
    p.remap = remap;
    return from_hip(gdn::launch_kv_compact(p, stream));
}

} // extern "C"
