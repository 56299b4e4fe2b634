// abi_attn.cu -- the extern "C" entry points of the attention block (declared
// in include/qgemv.h): every argument the host can see is checked before any
// kernel is enqueued.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/qgemv.h"
#include "kv_cache.cuh"

using namespace qg;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool is_16bit(int type) { return type == QG_BF16 || type == QG_F16; }

// The cache's own arguments, and its device view.
int check_cache(const char *fn, const qg_kv_cache *c, KvView *view) {
    if (!c) QG_REFUSE(kEInval, "%s: cache must be non-NULL", fn);
    if (!is_16bit(c->type) && c->type != QG_E4M3)
        QG_REFUSE(kEInval, "%s: cache type %d is not QG_BF16, QG_F16 or QG_E4M3", fn, c->type);
    if (c->n_pages < 1 || c->page_size < 1 || c->n_heads < 1)
        QG_REFUSE(kEInval, "%s: n_pages = %d, page_size = %d and n_heads = %d must be >= 1", fn, c->n_pages,
                  c->page_size, c->n_heads);
    const size_t esz = c->type == QG_E4M3 ? 1 : 2;
    if (c->head_dim < 1 || c->head_dim > 256 || c->head_dim * esz % 16)
        QG_REFUSE(kEShape, "%s: head_dim = %d must be in 1..256 and %d-element lines", fn, c->head_dim,
                  (int)(16 / esz));
    if (!c->k || !c->v) QG_REFUSE(kEInval, "%s: k and v must be non-NULL", fn);
    if (c->type == QG_E4M3 && (!c->k_scale || !c->v_scale))
        QG_REFUSE(kEInval, "%s: an e4m3 cache needs k_scale and v_scale", fn);
    const size_t dim = (size_t)c->head_dim;
    if (c->token_stride < dim || c->head_stride < dim || c->page_stride < dim)
        QG_REFUSE(kEInval, "%s: the cache's strides must be at least head_dim", fn);
    const size_t most = (size_t)1 << 38;   // elements: the copies' strides are below 2^40 bytes
    if (c->token_stride > most || c->head_stride > most || c->page_stride > most ||
        c->page_stride > ((size_t)1 << 60) / c->n_pages || c->head_stride > ((size_t)1 << 60) / c->n_heads ||
        c->token_stride > ((size_t)1 << 60) / c->page_size)
        QG_REFUSE(kEInval, "%s: the cache's strides overflow", fn);
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->token_stride * esz % 16 || c->head_stride * esz % 16 ||
        c->page_stride * esz % 16)
        QG_REFUSE(kEAlign, "%s: k, v and the cache's strides must be whole 16-byte lines", fn);
    if (!aligned(c->weight, 4) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        QG_REFUSE(kEAlign, "%s: weight and the scales must be 4-byte aligned", fn);
    view->k = static_cast<char *>(c->k);
    view->v = static_cast<char *>(c->v);
    view->k_scale = c->k_scale;
    view->v_scale = c->v_scale;
    view->weight = c->weight;
    view->page_b = (long long)(c->page_stride * esz);
    view->head_b = (long long)(c->head_stride * esz);
    view->token_b = (long long)(c->token_stride * esz);
    view->n_pages = c->n_pages;
    view->page = c->page_size;
    view->page_div = fast_div(c->page_size);
    view->n_heads = c->n_heads;
    view->dim = c->head_dim;
    view->type = c->type;
    return kOk;
}

int check_table(const char *fn, const char *name, const int *table, int stride) {
    if (!table) QG_REFUSE(kEInval, "%s: %s must be non-NULL", fn, name);
    if (stride < 1) QG_REFUSE(kEInval, "%s: the stride of %s is %d, must be >= 1", fn, name, stride);
    if (!aligned(table, 4)) QG_REFUSE(kEAlign, "%s: %s must be 4-byte aligned", fn, name);
    return kOk;
}

int check_heads(const char *fn, int n_q_heads, int n_heads) {
    if (n_q_heads < 1 || n_q_heads % n_heads)
        QG_REFUSE(kEInval, "%s: n_q_heads = %d must be a positive multiple of the cache's %d heads", fn, n_q_heads,
                  n_heads);
    if (n_q_heads > 65535) QG_REFUSE(kEInval, "%s: n_q_heads = %d, must be <= 65535", fn, n_q_heads);
    return kOk;
}

int check_max_len(const char *fn, int max_len, int stride, int page) {
    if (max_len < 0 || max_len > (long long)stride * page)
        QG_REFUSE(kEInval, "%s: max_len = %d must be in 0..%lld (the table's pages)", fn, max_len,
                  (long long)stride * page);
    if (max_len > (1 << 30)) QG_REFUSE(kEInval, "%s: max_len = %d, must be <= 2^30", fn, max_len);
    return kOk;
}

// Rows of all sequences, and cost units of one sequence, must be counted in 31
// bits (a launch takes as many sequences as have their units counted so).
int check_attn_sizes(const char *fn, const KvView &c, int n_seq, int max_len, int S, int n_q_heads) {
    if (S < 1 || S > 8) QG_REFUSE(kEInval, "%s: S = %d new tokens, must be in 1..8", fn, S);
    if (n_seq < 0) QG_REFUSE(kEInval, "%s: n_seq = %d, must be >= 0", fn, n_seq);
    const int rc = check_heads(fn, n_q_heads, c.n_heads);
    if (rc) return rc;
    if ((double)n_seq * S * n_q_heads > (double)INT_MAX / 2 || attn_units(c, max_len, S, n_q_heads) > kAttnMaxUnits)
        QG_REFUSE(kEInval, "%s: sizes overflow", fn);
    return kOk;
}

}  // namespace

extern "C" {

int qg_rope_append(const qg_kv_cache *cache, const int *table, int table_stride, int n_seq, const int *seq,
                   const int *slot, int T, void *q, int q_type, const void *qkv, int qkv_type, size_t qkv_stride,
                   int n_q_heads, const int *pos, int n_axes, const unsigned char *axis, const float *inv_freq,
                   int rotary_dim, int style, qg_stream_t stream) {
    const char *fn = "qg_rope_append";
    RopeArgs a = {};
    int rc = check_cache(fn, cache, &a.c);
    if (rc) return rc;
    if (T < 0) QG_REFUSE(kEInval, "%s: T = %d, must be >= 0", fn, T);
    if ((rc = check_heads(fn, n_q_heads, a.c.n_heads))) return rc;
    if (!is_16bit(q_type)) QG_REFUSE(kEInval, "%s: q type %d is not QG_BF16 or QG_F16", fn, q_type);
    if (qkv_type != QG_F32 && !is_16bit(qkv_type))
        QG_REFUSE(kEInval, "%s: qkv type %d is not QG_F32, QG_BF16 or QG_F16", fn, qkv_type);
    const size_t row = ((size_t)n_q_heads + 2 * (size_t)a.c.n_heads) * a.c.dim;
    if (qkv_stride < row) QG_REFUSE(kEInval, "%s: qkv_stride = %zu is below a row's %zu", fn, qkv_stride, row);
    if (qkv_stride > ((size_t)1 << 40)) QG_REFUSE(kEInval, "%s: sizes overflow", fn);
    if (rotary_dim < 0 || rotary_dim > a.c.dim || (rotary_dim & 1))
        QG_REFUSE(kEInval, "%s: rotary_dim = %d must be even and in 0..%d", fn, rotary_dim, a.c.dim);
    if (style != QG_ROPE_HALF && style != QG_ROPE_INTERLEAVED) QG_REFUSE(kEInval, "%s: unknown style %d", fn, style);
    if (n_axes < 1 || n_axes > 255) QG_REFUSE(kEInval, "%s: n_axes = %d, must be in 1..255", fn, n_axes);
    if (axis)
        for (int j = 0; j < rotary_dim / 2; ++j)
            if (axis[j] >= n_axes)
                QG_REFUSE(kEInval, "%s: axis[%d] = %d, must be below n_axes = %d", fn, j, (int)axis[j], n_axes);
    if (n_seq < 0 || (n_seq == 0 && T > 0)) QG_REFUSE(kEInval, "%s: n_seq = %d, must be >= 1 (0 without tokens)", fn, n_seq);
    if (T == 0) return kOk;
    if ((rc = check_table(fn, "table", table, table_stride))) return rc;
    if (!seq || !slot || !q || !qkv) QG_REFUSE(kEInval, "%s: seq, slot, q and qkv must be non-NULL", fn);
    if (rotary_dim > 0 && (!pos || !inv_freq)) QG_REFUSE(kEInval, "%s: pos and inv_freq must be non-NULL", fn);
    if (!aligned(seq, 4) || !aligned(slot, 4) || !aligned(pos, 4) || !aligned(inv_freq, 4))
        QG_REFUSE(kEAlign, "%s: seq, slot, pos and inv_freq must be 4-byte aligned", fn);
    if (!aligned(q, 2) || !aligned(qkv, qkv_type == QG_F32 ? 4 : 2))
        QG_REFUSE(kEAlign, "%s: q and qkv must be aligned to their elements", fn);
    a.table = table;
    a.table_stride = table_stride;
    a.n_seq = n_seq;
    a.seq = seq;
    a.slot = slot;
    a.T = T;
    a.q = q;
    a.q_type = q_type;
    a.qkv = qkv;
    a.qkv_stride = qkv_stride;
    a.n_q_heads = n_q_heads;
    a.pos = pos;
    a.n_axes = n_axes;
    a.inv_freq = inv_freq;
    a.rotary = rotary_dim;
    a.interleaved = style == QG_ROPE_INTERLEAVED;
    if (axis) memcpy(a.axis, axis, (size_t)rotary_dim / 2);
    cudaGetLastError();
    a.err = device_error_word();
    return run_rope_append(a, qkv_type, reinterpret_cast<cudaStream_t>(stream));
}

size_t qattn_workspace_bytes(const qg_kv_cache *cache, int n_seq, int max_len, int S, int n_q_heads,
                             int accumulate) {
    const char *fn = "qattn_workspace_bytes";
    KvView c;
    if (check_cache(fn, cache, &c) || max_len < 0 || check_attn_sizes(fn, c, n_seq, max_len, S, n_q_heads) ||
        n_seq == 0)
        return 0;
    return ws_attn_paged_most(c, n_seq, max_len, S, n_q_heads, accumulate != 0);
}

int qattn_paged(const qg_kv_cache *cache, const int *table, int table_stride, const int *lens, int n_seq,
                int max_len, void *o, int o_type, float *lse, const void *q, int q_type, size_t q_stride, int S,
                int n_q_heads, float scale, int accumulate, void *ws, size_t ws_bytes, qg_stream_t stream) {
    const char *fn = "qattn_paged";
    AttnArgs a = {};
    int rc = check_cache(fn, cache, &a.c);
    if (rc) return rc;
    if (max_len < 0) QG_REFUSE(kEInval, "%s: max_len = %d, must be >= 0", fn, max_len);
    if ((rc = check_attn_sizes(fn, a.c, n_seq, max_len, S, n_q_heads))) return rc;
    if (o_type != QG_F32 && !is_16bit(o_type))
        QG_REFUSE(kEInval, "%s: o type %d is not QG_F32, QG_BF16 or QG_F16", fn, o_type);
    if (!is_16bit(q_type) || (a.c.type != QG_E4M3 && q_type != a.c.type))
        QG_REFUSE(kEInval, "%s: q type %d does not go with a cache of type %d", fn, q_type, a.c.type);
    if (!isfinite(scale)) QG_REFUSE(kEInval, "%s: scale must be finite", fn);
    if (q_stride < (size_t)n_q_heads * a.c.dim || q_stride > ((size_t)1 << 40))
        QG_REFUSE(kEInval, "%s: q_stride = %zu must hold a row's %zu elements", fn, q_stride,
                  (size_t)n_q_heads * a.c.dim);
    if (accumulate && !a.c.weight) QG_REFUSE(kEInval, "%s: accumulate needs the cache's weight", fn);
    if (n_seq == 0) return kOk;
    if ((rc = check_table(fn, "table", table, table_stride))) return rc;
    if ((rc = check_max_len(fn, max_len, table_stride, a.c.page))) return rc;
    if (!lens || !o || !q) QG_REFUSE(kEInval, "%s: lens, o and q must be non-NULL", fn);
    if (!aligned(lens, 4) || !aligned(lse, 4)) QG_REFUSE(kEAlign, "%s: lens and lse must be 4-byte aligned", fn);
    if (!aligned(q, 16) || q_stride % 8 || !aligned(o, 16))
        QG_REFUSE(kEAlign, "%s: q, its rows and o must be 16-byte aligned", fn);
    const size_t need = ws_attn_paged(a.c, n_seq, max_len, S, n_q_heads, accumulate != 0);
    if (need > 0 && (ws == nullptr || ws_bytes < need))
        QG_REFUSE(kEWorkspace, "%s: needs a workspace of %zu bytes (qattn_workspace_bytes; got %zu)", fn, need,
                  ws == nullptr ? (size_t)0 : ws_bytes);
    if (ws && !aligned(ws, 256)) QG_REFUSE(kEAlign, "%s: workspace must be 256-byte aligned", fn);
    a.table = table;
    a.table_stride = table_stride;
    a.lens = lens;
    a.n_seq = n_seq;
    a.max_len = max_len;
    a.o = o;
    a.o_type = o_type;
    a.lse = lse;
    a.q = q;
    a.q_type = q_type;
    a.q_stride = q_stride;
    a.S = S;
    a.n_q_heads = n_q_heads;
    a.group = n_q_heads / a.c.n_heads;
    a.scale = scale;
    a.accumulate = accumulate != 0;
    cudaGetLastError();
    a.err = device_error_word();
    return run_attn_paged(a, ws, reinterpret_cast<cudaStream_t>(stream));
}

int qg_kv_evict(const qg_kv_cache *cache, const int *table, int table_stride, const int *dst_table, int dst_stride,
                const int *lens, int n_seq, int max_len, int budget, int sinks, int recent, int *kept,
                int *new_lens, qg_stream_t stream) {
    const char *fn = "qg_kv_evict";
    EvictArgs a = {};
    int rc = check_cache(fn, cache, &a.c);
    if (rc) return rc;
    if (!a.c.weight) QG_REFUSE(kEInval, "%s: the cache has no weight", fn);
    if (n_seq < 0) QG_REFUSE(kEInval, "%s: n_seq = %d, must be >= 0", fn, n_seq);
    if (budget < 1) QG_REFUSE(kEInval, "%s: budget = %d, must be >= 1", fn, budget);
    if (sinks < 0 || recent < 0 || (long long)sinks + recent > budget)
        QG_REFUSE(kEInval, "%s: sinks = %d and recent = %d must be >= 0 and together at most budget = %d", fn, sinks,
                  recent, budget);
    if ((double)n_seq * a.c.n_heads > (double)INT_MAX / 16) QG_REFUSE(kEInval, "%s: sizes overflow", fn);
    if (n_seq == 0) return kOk;
    if ((rc = check_table(fn, "table", table, table_stride))) return rc;
    if ((rc = check_table(fn, "dst_table", dst_table, dst_stride))) return rc;
    if ((rc = check_max_len(fn, max_len, table_stride, a.c.page))) return rc;
    if ((long long)dst_stride * a.c.page < (budget < max_len ? budget : max_len))
        QG_REFUSE(kEInval, "%s: a row of dst_table holds %lld slots, min(budget, max_len) = %d are needed", fn,
                  (long long)dst_stride * a.c.page, budget < max_len ? budget : max_len);
    if (!lens || !kept || !new_lens) QG_REFUSE(kEInval, "%s: lens, kept and new_lens must be non-NULL", fn);
    if (lens == new_lens) QG_REFUSE(kEInval, "%s: new_lens must not be lens", fn);
    if (!aligned(lens, 4) || !aligned(kept, 4) || !aligned(new_lens, 4))
        QG_REFUSE(kEAlign, "%s: lens, kept and new_lens must be 4-byte aligned", fn);
    a.table = table;
    a.table_stride = table_stride;
    a.dst_table = dst_table;
    a.dst_stride = dst_stride;
    a.lens = lens;
    a.n_seq = n_seq;
    a.max_len = max_len;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.kept = kept;
    a.new_lens = new_lens;
    cudaGetLastError();
    a.err = device_error_word();
    return run_kv_evict(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
